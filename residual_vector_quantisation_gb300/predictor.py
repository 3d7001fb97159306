"""Operators of a code predictor over torch tensors: differentiable layer norm
and distillation loss, and a beam search over a quantiser's codes.

They sit on the C ABI of include/rvq.h (the rvq_* functions of the package) and
own what those leave to the caller: outputs, statistics and workspaces.
"""

from __future__ import annotations

from typing import Optional

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


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        rows = _as_rows(x)
        y = torch.empty(rows.shape, dtype=x.dtype, device=x.device)
        mean, rstd = torch.empty((2, rows.shape[0]), dtype=torch.float32, device=x.device).unbind(0)
        _rq.rvq_layer_norm(rows, weight, bias, eps, y, mean, rstd)
        ctx.save_for_backward(rows, weight, bias, mean, rstd)
        ctx.shape = x.shape
        return y.view(x.shape)

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
    if top_codes.dtype != torch.int32:  # a code past 32 bits stays out of range
        top_codes = top_codes.to(torch.int64).clamp(-2, 2 ** 31 - 1).to(torch.int32)
    return rows, (top_logits.reshape(-1, top).contiguous(), top_codes.reshape(-1, top).contiguous(), *flat)


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_logits, top_codes, teacher_lse, weights, temperature):
        rows, teacher = _teacher(logits, top_logits, top_codes, teacher_lse, weights)
        loss = torch.empty(rows.shape[0], dtype=torch.float32, device=rows.device)
        lse = torch.empty((rows.shape[0], 2), dtype=torch.float32, device=rows.device)
        _rq.rvq_distill(rows, *teacher, temperature, loss, lse=lse)
        ctx.save_for_backward(rows, *teacher, lse)
        ctx.shape, ctx.temperature = logits.shape, temperature
        return loss.view(logits.shape[:-1])

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
