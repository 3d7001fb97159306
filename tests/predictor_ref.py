"""Plain 64-bit statements of the code predictor's operators, and how far a
32-bit computation of them may be off.

U is half a unit in the last place of float32 relative to its value.  Each
`*_tol` sums the rounding that a straightforward 32-bit evaluation may make:
STEPS * U times the size of the terms that are added (rows are summed in
pieces, so that no sum has more than STEPS roundings on a path, and each term
carries a few), plus one rounding of the output type.
"""

import torch

U = 2.0 ** -24
STEPS = 64
OUT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24}


def out_tol(ref, inner, dtype):
    return OUT[dtype] * ref.abs() + (1 + OUT[dtype]) * inner + TINY[dtype]


def check(got, ref, inner, what):
    """got equals ref (64 bits) within its type's rounding and `inner`; infinities (values past the type's range
    among them) and NaN in the same places."""
    g, r = got.double().cpu(), ref.cpu()
    r = torch.where(torch.isinf(r.to(got.dtype)), r.to(got.dtype).double(), r)
    inner = inner.cpu() if torch.is_tensor(inner) else torch.full_like(r, inner)
    assert g.shape == r.shape, (what, g.shape, r.shape)
    fine = torch.isfinite(r)
    assert torch.equal(torch.isnan(g), torch.isnan(r)), f"{what}: NaN in other places"
    same = (g == r) | torch.isnan(r)
    assert bool(same[~fine].all()), f"{what}: infinities in other places"
    off = ((g - r).abs() / out_tol(r, inner.expand_as(r), got.dtype))[fine]
    assert off.numel() == 0 or bool((off <= 1).all()), f"{what}: {off.max().item():.3g} times the tolerance"


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------

def norm(x, weight, bias, eps, dy=None):
    """({name: value}, {name: inner tolerance}) of y and, with dy, dx, dweight, dbias."""
    x = x.double()
    rows, width = x.shape
    w = torch.ones(width, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    b = torch.zeros_like(w) if bias is None else bias.double()
    mu = x.mean(1, keepdim=True)
    var = ((x - mu) ** 2).mean(1, keepdim=True)
    r = 1 / torch.sqrt(var + eps)
    h = (x - mu) * r
    size = (x.abs() + x.abs().amax(1, keepdim=True)) * r + h.abs()   # what cancels in x - mu
    val = {"y": h * w + b}
    tol = {"y": STEPS * U * (size * w.abs() + b.abs())}
    if dy is not None:
        dy = dy.double()
        g = dy * w
        val["dx"] = r * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
        inner = g.abs() + g.abs().mean(1, keepdim=True) + 2 * size * (g.abs() * size).mean(1, keepdim=True)
        tol["dx"] = STEPS * U * r * inner
        val["dweight"], val["dbias"] = (dy * h).sum(0), dy.sum(0)
        tol["dweight"], tol["dbias"] = STEPS * U * (dy.abs() * size).sum(0), STEPS * U * dy.abs().sum(0)
    return val, tol


# ---------------------------------------------------------------------------
# distillation
# ---------------------------------------------------------------------------

def distill(logits, top_logits, top_codes, teacher_lse, weights, temperature, grad_loss=None):
    """Row by row, from the definition: ({"loss", "dlogits"}, tolerances, bad codes)."""
    z = logits.double().cpu() / temperature
    t = top_logits.double().cpu() / temperature
    codes = top_codes.cpu().tolist()
    rows, vocab = z.shape
    loss, grad = torch.zeros(rows, dtype=torch.float64), torch.zeros((rows, vocab), dtype=torch.float64)
    loss_tol, grad_tol = torch.zeros_like(loss), torch.zeros_like(grad)
    bad = 0
    for i in range(rows):
        w = 1.0 if weights is None else weights[i].item()
        up = (1.0 if grad_loss is None else grad_loss[i].item()) * w / temperature
        if w == 0.0:
            continue
        at, code = [], []
        for j, c in enumerate(codes[i]):
            if 0 <= c < vocab and c not in code:
                at.append(j)
                code.append(c)
            elif c != -1:
                bad += 1
        if not code:
            continue
        tt, index = t[i, at], torch.tensor(code)
        if teacher_lse is None and bool((tt == -torch.inf).all()):
            continue
        given = None if teacher_lse is None else teacher_lse[i].double().cpu()
        log_q = tt - (torch.logsumexp(tt, 0) if given is None else given)
        q = log_q.exp()
        if bool((z[i] == -torch.inf).all()):
            log_p = torch.full((vocab,), -torch.inf, dtype=torch.float64)
        else:
            log_p = torch.log_softmax(z[i], 0)
        p = log_p.exp()
        lp = log_p[index]
        terms = torch.where(q == 0, 0.0, q * (log_q - lp))
        value, g = terms.sum(), p.clone()
        # the exponents' rounding goes with their size
        size = z[i][torch.isfinite(z[i]) & (z[i] > -1e30)].abs()
        size = size.max().item() if size.numel() else 0.0
        ts = tt[torch.isfinite(tt) & (tt > -1e30)].abs()
        size_t = max(ts.max().item() if ts.numel() else 0.0, 0.0 if given is None else abs(given.item()))
        c, ct = (STEPS + 8 * size) * U, (STEPS + 8 * size_t) * U
        inner = torch.where(q == 0, 0.0, q * (ct * (1 + (log_q - lp).abs()) + c)).sum()
        g_tol = c * p
        if given is not None:
            rest = torch.ones(vocab, dtype=torch.bool)
            rest[index] = False
            q_rest = 1 - q.sum()
            q_rest = torch.where(q_rest <= 2.0 ** -20, 0.0, q_rest)
            log_rest = torch.logsumexp(log_p[rest], 0) if bool((log_p[rest] > -torch.inf).any()) or \
                bool(torch.isnan(log_p).any()) else torch.tensor(-torch.inf, dtype=torch.float64)
            share = torch.where(log_p[rest] == -torch.inf, 0.0, (log_p[rest] - log_rest).exp())
            g[rest] = p[rest] - q_rest * share
            g_tol[rest] += (ct + c * q_rest) * share
            if q_rest != 0:
                value = value + q_rest * (q_rest.log() - log_rest)
                inner = inner + ct * (1 + (q_rest.log() - log_rest).abs()) + c * q_rest
        g[index] = p[index] - q
        g_tol[index] = c * p[index] + ct * q
        loss[i], grad[i] = value * w, g * up
        loss_tol[i] = (inner * abs(w)) if bool(torch.isfinite(inner)) else 0.0
        grad_tol[i] = g_tol * abs(up)
    return {"loss": loss, "dlogits": grad}, {"loss": loss_tol, "dlogits": grad_tol}, bad


# ---------------------------------------------------------------------------
# the beam step
# ---------------------------------------------------------------------------

def beam(logits, scores, finished, end_code, select, raw):
    """(scores, parents, codes, finished) of [groups][beams][vocab] logits; raw totals in float32 (one sum, so
    that ties are the kernel's), else in 64 bits."""
    groups, beams, vocab = logits.shape
    logits, scores = logits.cpu(), scores.cpu()
    out = [], [], [], []
    for g in range(groups):
        best = []
        for b in range(beams):
            s = scores[g, b]
            if not bool(s > -torch.inf):
                continue
            if finished is not None and bool(finished[g, b]):
                best.append((-s.item(), b, 0.0, end_code))
                continue
            x = logits[g, b].float() if raw else logits[g, b].double()
            total = s + x if raw else s.double() + torch.log_softmax(x, 0)
            ok = (total > -torch.inf).nonzero()[:, 0].tolist()
            values, z = total.tolist(), x.tolist()
            best += [(-values[v], b, 0.0 if raw else -z[v], v) for v in ok]
        best.sort()
        best = best[:select] + [(torch.inf, -1, 0.0, -1)] * (select - len(best))
        out[0].append([-c[0] for c in best])
        out[1].append([c[1] for c in best])
        out[2].append([c[3] for c in best])
        out[3].append([c[1] < 0 or bool(finished is not None and finished[g, c[1]]) or c[3] == end_code for c in best])
    return (torch.tensor(out[0], dtype=torch.float64), torch.tensor(out[1]), torch.tensor(out[2]),
            torch.tensor(out[3]))
