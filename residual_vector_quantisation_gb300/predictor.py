"""Operators of a code predictor over torch tensors: differentiable norms,
dropout, log probabilities and distillation loss, and a beam search over a
quantiser's codes.

They sit on the C ABI of include/rvq.h (the rvq_* functions of the package) and
own what those leave to the caller: outputs, statistics and workspaces.
"""

from __future__ import annotations

from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

import residual_vector_quantisation_gb300 as _rq


def _as_rows(t: torch.Tensor) -> torch.Tensor:
    """t as [rows][last axis] with contiguous rows (a view where that is possible)."""
    r = t if t.dim() == 2 else t.reshape(-1, t.shape[-1])
    if r.shape[0] > 1 and r.stride(0) < r.shape[1] or r.shape[1] > 1 and r.stride(1) != 1:
        r = r.contiguous()
    return r


def _result(x: torch.Tensor, rows: torch.Tensor):
    """A new tensor like x, and it as rows for the kernels.  An autograd function gives back the first: a view that it
    made could not be changed in place."""
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    return y, y.view(rows.shape)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        rows = _as_rows(x)
        y, y_rows = _result(x, rows)
        mean, rstd = torch.empty((2, rows.shape[0]), dtype=torch.float32, device=x.device).unbind(0)
        _rq.rvq_layer_norm(rows, weight, bias, eps, y_rows, mean, rstd)
        ctx.save_for_backward(rows, weight, bias, mean, rstd)
        ctx.shape = x.shape
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        rows, weight, bias, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx = torch.empty(rows.shape, dtype=rows.dtype, device=rows.device) if need[0] else None
        dweight = torch.empty_like(weight) if weight is not None and need[1] else None
        dbias = torch.empty_like(bias) if bias is not None and need[2] else None
        workspace = None
        if dweight is not None or dbias is not None:
            nbytes = _rq.rvq_layer_norm_workspace_bytes(*rows.shape)
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=rows.device)
        _rq.rvq_layer_norm_backward(_as_rows(dy.to(rows.dtype)), rows, weight, mean, rstd, dx, dweight, dbias,
                                    workspace)
        return None if dx is None else dx.view(ctx.shape), dweight, dbias, None


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5) -> torch.Tensor:
    """Layer norm over the last axis of x (float32, bfloat16 or float16), differentiable in x, weight and bias.
    weight and bias: float32, or x's dtype, both the same.  Runs on the current stream."""
    for p in (weight, bias):
        if p is not None and not p.is_contiguous():
            raise ValueError("weight and bias must be contiguous")
    return _LayerNorm.apply(x, weight, bias, eps)


def _same_kind(x: torch.Tensor, residual: Optional[torch.Tensor]) -> None:
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype):
        raise ValueError("residual must have x's shape and dtype")


def _beside(x: torch.Tensor, residual: Optional[torch.Tensor]):
    """x and residual as rows."""
    _same_kind(x, residual)
    return _as_rows(x), None if residual is None else _as_rows(residual)


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, mask, step):
        rows, add = _beside(x, residual)
        y, y_rows = _result(x, rows)
        _rq.rvq_dropout(rows, mask, y_rows, add)
        ctx.save_for_backward(step)  # counted up before the backward pass, it would give another mask
        ctx.mask = mask.copy()  # its fields may be another place's by then
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        ctx.saved_tensors  # raises where the step has been counted up
        dx = None
        if ctx.needs_input_grad[0]:
            rows = _as_rows(dy)
            dx = torch.empty(rows.shape, dtype=rows.dtype, device=rows.device)
            _rq.rvq_dropout(rows, ctx.mask, dx)
            dx = dx.view(dy.shape)
        return dx, dy if ctx.needs_input_grad[1] else None, None, None


def dropout(x: torch.Tensor, mask: Optional[_rq.rvq_dropout_mask],
            residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x where the mask has it stay, times the factor that keeps its mean, and 0 elsewhere; plus residual: a new tensor.
    Differentiable in x and residual (x's shape and dtype).  The mask is made anew in the backward pass and never
    stored: mask = rvq_dropout_mask(p, seed, offset, step) says which one, element by element of x in its order
    (whatever its strides); None: nothing is dropped.  A step on the GPU has to be counted up after the backward pass.
    Runs on the current stream."""
    if mask is None:
        mask = _rq.rvq_dropout_mask(0.0, 0)
    if x.numel() == 0:
        _same_kind(x, residual)
        return x.clone() if residual is None else x + residual
    return _Dropout.apply(x, residual, mask, mask.tensor)


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps, mask, step):
        rows, add = _beside(x, residual)
        y, y_rows = _result(x, rows)
        total, total_rows = (None, None) if add is None and mask is None else _result(x, rows)
        rstd = torch.empty(rows.shape[0], dtype=torch.float32, device=x.device)
        _rq.rvq_rms_norm(rows, weight, eps, y_rows, rstd, add, mask, total_rows)
        ctx.save_for_backward(rows if total is None else total, weight, rstd, step)
        ctx.set_materialize_grads(False)
        ctx.shape, ctx.mask = x.shape, None if mask is None else mask.copy()
        return y if total is None else (y, total)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dtotal=None):
        total, weight, rstd, _ = ctx.saved_tensors
        total = total.view(-1, total.shape[-1])  # (a result of the forward pass, or rows)
        need, mask = ctx.needs_input_grad, ctx.mask
        if dy is None and dtotal is None:
            return (None,) * 6
        like = dict(dtype=total.dtype, device=total.device)
        if dy is None:  # the sum's gradient passes the norm by, whatever its rows hold, as the tensor that it is
            dx = dtotal
            if need[0] and mask is not None:
                dx = torch.empty(ctx.shape, **like)
                _rq.rvq_dropout(_as_rows(dtotal), mask, dx.view(total.shape))
            return (dx if need[0] else None, dtotal if need[1] else None,
                    torch.zeros_like(weight) if need[2] else None, None, None, None)
        dtotal = None if dtotal is None else _as_rows(dtotal.to(total.dtype))
        dy = _as_rows(dy.to(total.dtype))
        dresidual = torch.empty(total.shape, **like) if need[1] or (need[0] and mask is None) else None
        dx = torch.empty(total.shape, **like) if need[0] and mask is not None else None
        dweight = workspace = None
        if weight is not None and need[2]:
            dweight = torch.empty_like(weight)
            nbytes = _rq.rvq_rms_norm_workspace_bytes(*total.shape)
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=total.device)
        _rq.rvq_rms_norm_backward(dy, total, weight, rstd, dresidual, dweight, workspace, dtotal, mask, dx)
        dresidual = None if dresidual is None else dresidual.view(ctx.shape)
        # without a mask x's gradient is the residual's, and the same tensor: autograd gives a leaf a gradient that
        # nothing else holds as it is, and two views of one memory would each be such a one
        dx = dresidual if mask is None else None if dx is None else dx.view(ctx.shape)
        return dx if need[0] else None, dresidual if need[1] else None, dweight, None, None, None


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
             residual: Optional[torch.Tensor] = None, mask: Optional[_rq.rvq_dropout_mask] = None):
    """Root-mean-square norm over the last axis of x (float32, bfloat16 or float16), or of total = residual + drop(x):
    y, or (y, total) where a residual or a mask is given, total being the residual of the next sublayer (the backward pass
    reads it: changed in place before, it is an error there).
    Differentiable in x, weight (float32, or x's dtype) and residual (x's shape and dtype), from both results.  mask: as
    in dropout.  Runs on the current stream."""
    if weight is not None and not weight.is_contiguous():
        raise ValueError("weight must be contiguous")
    return _RmsNorm.apply(x, residual, weight, eps, mask, None if mask is None else mask.tensor)


def rms_norm_8bit(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  residual: Optional[torch.Tensor] = None, block: int = 0, powers: bool = False):
    """The same norm with its result in 8 bits: (q, scales), or (q, scales, total) with a residual.  q: float8_e4m3fn,
    x's shape; scales [...][n]: one for each `block` columns (32, 64 or 128), or (0) one a row; float32, or, with powers,
    powers of two (float8_e8m0fnu).  q * scales is the norm's result.  For inference: it has no gradient."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, weight, residual)):
        raise ValueError("rms_norm_8bit has no gradient: call it under torch.no_grad(), or on tensors that need none")
    if block not in (0, 32, 64, 128):
        raise ValueError("block must be 0, 32, 64 or 128")
    if weight is not None and not weight.is_contiguous():
        raise ValueError("weight must be contiguous")
    rows, add = _beside(x, residual)
    count = 1 if block == 0 else -(-x.shape[-1] // block)
    q = torch.empty(rows.shape, dtype=torch.float8_e4m3fn, device=x.device)
    scales = torch.empty((rows.shape[0], count), dtype=torch.float8_e8m0fnu if powers else torch.float32, device=x.device)
    total = None if add is None else torch.empty(rows.shape, dtype=x.dtype, device=x.device)
    _rq.rvq_rms_norm(rows, weight, eps, None, residual=add, total=total, q=q, scales=scales, block=block)
    out = q.view(x.shape), scales.view(x.shape[:-1] + (count,))
    return out if total is None else out + (total.view(x.shape),)


class LogProbs(NamedTuple):
    """What log_probs gives; None where it was not asked for."""
    log_probs: Optional[torch.Tensor]
    entropy: Optional[torch.Tensor]
    lse: torch.Tensor
    top_log_probs: Optional[torch.Tensor]
    top_codes: Optional[torch.Tensor]


class _LogProbs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, codes, entropy, top, temperature):
        rows = _as_rows(logits)
        n, lead = rows.shape[0], logits.shape[:-1]
        if codes is not None:
            if codes.shape != lead:
                raise ValueError("codes must have the logits' leading axes")
            codes = _int32(codes).reshape(-1).contiguous()

        def one(*shape, dtype=torch.float32):
            return torch.empty(lead + shape, dtype=dtype, device=rows.device)

        log_p, h = None if codes is None else one(), one() if entropy else None
        lse = one()
        best = (one(top), one(top, dtype=torch.int32)) if top else (None, None)
        out = log_p, h, lse, *best
        stats = torch.empty((n, 2), dtype=torch.float32, device=rows.device)
        flat = [None if t is None else t.view((n,) + t.shape[len(lead):]) for t in out]
        _rq.rvq_log_probs(rows, codes, temperature, *flat[:3], stats, *flat[3:])
        ctx.save_for_backward(rows, codes, stats, h)
        ctx.set_materialize_grads(False)
        ctx.shape, ctx.temperature = logits.shape, temperature
        ctx.mark_non_differentiable(*(t for t in out[3:] if t is not None))
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_log_probs, grad_entropy, grad_lse, *_):
        rows, codes, stats, entropy = ctx.saved_tensors
        entropy = None if entropy is None else entropy.view(-1)
        grads = [None if g is None else g.to(torch.float32).reshape(-1).contiguous()
                 for g in (grad_log_probs, grad_entropy, grad_lse)]
        dlogits = torch.empty(rows.shape, dtype=rows.dtype, device=rows.device)
        _rq.rvq_log_probs_backward(*grads, rows, codes, ctx.temperature, stats, entropy, dlogits)
        return dlogits.view(ctx.shape), None, None, None, None


def log_probs(logits: torch.Tensor, codes: Optional[torch.Tensor] = None, entropy: bool = False, top: int = 0,
              temperature: float = 1.0) -> LogProbs:
    """Log probabilities of codes [...] (integers; -1: none, 0 then) under softmax(logits [...][vocab] / temperature),
    the distributions' entropy where asked for, their log sum exp, and the `top` best codes (at most 64) with their log
    probabilities.  Differentiable in logits through log_probs, entropy and lse; top_log_probs are constants.

    The lists are a teacher's for distill_loss: at the same temperature T,
    distill_loss(student, T * top_log_probs, top_codes, torch.zeros_like(lse), temperature=T).  Runs on the current
    stream."""
    return LogProbs(*_LogProbs.apply(logits, codes, bool(entropy), int(top), float(temperature)))


def _int32(codes: torch.Tensor) -> torch.Tensor:
    if codes.dtype != torch.int32:  # a code past 32 bits stays out of range
        codes = codes.to(torch.int64).clamp(-2, 2 ** 31 - 1).to(torch.int32)
    return codes


def _teacher(logits, top_logits, top_codes, teacher_lse, weights):
    """The loss's arguments as rows."""
    vocab, top = logits.shape[-1], top_logits.shape[-1]
    rows = _as_rows(logits)
    if top_logits.shape[:-1] != logits.shape[:-1] or top_codes.shape != top_logits.shape:
        raise ValueError("top_logits and top_codes must have the logits' leading axes")
    flat = []
    for t, name in ((teacher_lse, "teacher_lse"), (weights, "weights")):
        if t is not None:
            if t.shape != logits.shape[:-1]:
                raise ValueError(f"{name} must have the logits' leading axes")
            t = t.to(torch.float32).reshape(-1).contiguous()
        flat.append(t)
    top_codes = _int32(top_codes)
    return rows, (top_logits.reshape(-1, top).contiguous(), top_codes.reshape(-1, top).contiguous(), *flat)


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_logits, top_codes, teacher_lse, weights, temperature):
        rows, teacher = _teacher(logits, top_logits, top_codes, teacher_lse, weights)
        loss = torch.empty(logits.shape[:-1], dtype=torch.float32, device=rows.device)
        lse = torch.empty((rows.shape[0], 2), dtype=torch.float32, device=rows.device)
        _rq.rvq_distill(rows, *teacher, temperature, loss.view(-1), lse=lse)
        ctx.save_for_backward(rows, *teacher, lse)
        ctx.shape, ctx.temperature = logits.shape, temperature
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        rows, *teacher, lse = ctx.saved_tensors
        dlogits = torch.empty(rows.shape, dtype=rows.dtype, device=rows.device)
        grad = grad.to(torch.float32).reshape(-1).contiguous()
        _rq.rvq_distill_backward(grad, rows, *teacher, ctx.temperature, lse, dlogits)
        return dlogits.view(ctx.shape), None, None, None, None, None


def distill_loss(logits, top_logits, top_codes, teacher_lse=None, weights=None, temperature: float = 1.0):
    """Distillation loss of each row of logits [...][vocab], of shape [...], differentiable in logits.

    top_logits, top_codes [...][top]: the teacher's largest logits and their codes (-1: empty); teacher_lse [...]:
    the log sum exp of all the teacher's logits / temperature, where the mass that the list leaves out is to count
    (rvq_distill in include/rvq.h); weights [...]: a factor per row, 0 for padding.  The teacher and the weights are
    constants: no gradient goes to them.  Runs on the current stream."""
    return _Distill.apply(logits, top_logits, top_codes, teacher_lse, weights, float(temperature))


def distill_loss_and_grad(logits, top_logits, top_codes, teacher_lse=None, weights=None, temperature: float = 1.0,
                          out=None):
    """(loss [...], d sum(loss) / d logits) from one read of the logits; scale the gradient through `weights`.
    out: where the gradient goes (logits itself, where it is not needed any more)."""
    rows, teacher = _teacher(logits, top_logits, top_codes, teacher_lse, weights)
    if out is None:
        dlogits = torch.empty(rows.shape, dtype=rows.dtype, device=rows.device)
        out = dlogits.view(logits.shape)
    else:
        if out.shape != logits.shape or out.dtype != logits.dtype:
            raise ValueError("out must have the logits' shape and dtype")
        dlogits = out if out.dim() == 2 else out.view(-1, out.shape[-1])
    loss = torch.empty(rows.shape[0], dtype=torch.float32, device=rows.device)
    _rq.rvq_distill(rows, *teacher, float(temperature), loss, dlogits=dlogits)
    increment_version(out)  # written behind autograd's back: a backward pass that saved it has to notice
    return loss.view(logits.shape[:-1]), out


class BeamSearch:
    """Steps of `groups` beam searches over `vocab` codes.

    mode "logits": beams are scored by their sums of log probabilities; "raw": by the sums of the values given.
    end_code: the code that finishes a beam (None: none does).  The object owns a workspace; one object serves one
    stream at a time."""

    def __init__(self, groups: int, beams: int, vocab: int, select: Optional[int] = None, mode: str = "logits",
                 dtype: torch.dtype = torch.float32, end_code: Optional[int] = None, device="cuda"):
        modes = {"logits": _rq.RVQ_BEAM_LOGITS, "raw": _rq.RVQ_BEAM_RAW}
        self.dims = _rq.rvq_beam_dims(groups, beams, vocab, beams if select is None else select, modes[mode],
                                      _rq.DTYPES[dtype])
        self.end_code = -1 if end_code is None else int(end_code)
        nbytes = _rq.rvq_beam_workspace_bytes(self.dims)
        if nbytes == 0:
            raise ValueError("unsupported beam search arguments")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.device = self.workspace.device

    def first_scores(self) -> torch.Tensor:
        """Scores before the first step: one live beam per group."""
        scores = torch.full((self.dims.groups, self.dims.beams), float("-inf"), device=self.device)
        scores[:, 0] = 0.0
        return scores

    def select(self, logits, scores, finished=None, stream=None):
        """(scores, parents, codes, finished), each [groups][select], best first; finished is None where no code
        ends a beam.  stream: where the step runs (None: the current stream); the inputs have to be ready there, and
        the results are."""
        return _rq._run_on(stream, self.device, lambda: self._select(logits, scores, finished, stream),
                           lambda: (logits, scores, finished, self.workspace))

    def _select(self, logits, scores, finished, stream):
        kept = (self.dims.groups, self.dims.select)
        out = torch.empty(kept, dtype=torch.float32, device=self.device)
        parents, codes = torch.empty((2,) + kept, dtype=torch.int32, device=self.device).unbind(0)
        done = torch.empty(kept, dtype=torch.bool, device=self.device) if self.end_code >= 0 else None
        _rq.rvq_beam_select(self.dims, logits, scores, finished, self.end_code, out, parents, codes, done,
                            self.workspace, stream)
        return out, parents, codes, done

    def reorder(self, parents, state, out=None, layered: bool = False, stream=None):
        """state [groups][beams][...] (or [layers][groups][beams][...]) by the beams' parents: a new tensor, `out`,
        or in place where out is state.  stream: as in select."""
        return _rq._run_on(stream, self.device, lambda: self._reorder(parents, state, out, layered, stream),
                           lambda: (parents, state, out))

    def _reorder(self, parents, state, out, layered, stream):
        if out is None:
            lead = 1 if layered else 0
            shape = list(state.shape)
            shape[lead + 1] = self.dims.select
            out = torch.empty(shape, dtype=state.dtype, device=state.device)
        _rq.rvq_beam_reorder(self.dims, parents, _rq.rvq_beam_states([(state, out)], layered), stream)
        increment_version(out)
        return out
