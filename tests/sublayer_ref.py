"""Plain 64-bit statements of the operators at the end of a sublayer (dropout,
root-mean-square norm) and of log probabilities, and how far a 32-bit
computation of them may be off (U, STEPS, OUT, check: predictor_ref)."""

import numpy as np
import torch

from predictor_ref import OUT, STEPS, TINY, U, check, out_tol  # noqa: F401

# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------


def philox(counter, key, rounds=10):
    """Philox4x32 of one counter (four words) under one key (two words), in Python's whole numbers."""
    x, k = list(counter), list(key)
    for _ in range(rounds):
        p, q = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
        x = [(q >> 32) ^ x[1] ^ k[0], q & 0xFFFFFFFF, (p >> 32) ^ x[3] ^ k[1], p & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return x


def stays(n, p, seed, offset=0, step=0, first=0):
    """Whether elements first .. first + n - 1 stay (numpy), and the factor of those that do."""
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    upper = (offset + (step << 32)) % (1 << 64)
    g = np.arange(first // 8, (first + n + 7) // 8, dtype=np.uint64)
    x = [g & low, g >> half, np.full_like(g, upper & 0xFFFFFFFF), np.full_like(g, upper >> 32)]
    for i in range(10):
        k0 = np.uint64((seed + i * 0x9E3779B9) & 0xFFFFFFFF)
        k1 = np.uint64(((seed >> 32) + i * 0xBB67AE85) & 0xFFFFFFFF)
        a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(b >> half) ^ x[1] ^ k0, b & low, (a >> half) ^ x[3] ^ k1, a & low]
    bits = np.stack([w.astype("<u4") for w in x], 1).view("<u2").reshape(-1)[first % 8:][:n]
    drop = int(float(np.float32(p)) * 65536 + 0.5)
    return bits.astype(np.int64) >= drop, 65536 / (65536 - drop) if drop < 65536 else 0.0


def dropout(x, mask, residual=None):
    """(value, inner tolerance) of dropout with mask = (p, seed, offset, step) on x [rows][width]."""
    keep, factor = stays(x.numel(), *mask)
    keep = torch.from_numpy(keep).view(x.shape).to(x.device)
    v = torch.where(keep, x.double() * factor, 0.0)
    # the factor is a float32; the product and the sum are rounded once each
    tol = 2 * U * v.abs()
    if residual is not None:
        v = v + residual.double()
        tol = tol + U * v.abs()
    return v, tol


# ---------------------------------------------------------------------------
# root-mean-square norm
# ---------------------------------------------------------------------------

def total_of(x, mask=None, residual=None):
    """What is normalised: the sum in 32 bits, rounded to the type (the definition of the operator's `total`)."""
    h = x.float()
    if mask is not None:
        keep, factor = stays(x.numel(), *mask)
        keep = torch.from_numpy(keep).view(x.shape).to(x.device)
        h = torch.where(keep, h * torch.tensor(factor, dtype=torch.float32, device=x.device), 0.0)
    if residual is not None:
        h = h + residual.float()
    return h.to(x.dtype)


def rms(h, weight, eps, dy=None, dtotal=None, mask=None):
    """({name: value}, {name: inner tolerance}) of y and, with dy, dresidual, dx (with a mask) and dweight, from h.

    Sums over a row are taken in pieces, a thread's at most 40 terms one after the other and the rest in trees, so that
    no more than STEPS roundings lie on a path; the rows' sum of dweight likewise (a block's rows one after the other,
    the blocks in a tree): its terms' roundings are counted with their number where that is more."""
    h = h.double()
    rows, width = h.shape
    w = torch.ones(width, dtype=torch.float64, device=h.device) if weight is None else weight.double()
    r = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    u = h * r
    val = {"y": u * w}
    tol = {"y": STEPS * U * (u * w).abs()}
    if dy is not None:
        dy = dy.double()
        g = dy * w
        m = (g * u).mean(1, keepdim=True)
        size = (g * u).abs().mean(1, keepdim=True)
        dh = r * (g - u * m)
        inner = STEPS * U * r * (g.abs() + u.abs() * (size + m.abs()))
        if dtotal is not None:
            dh = dh + dtotal.double()
            inner = inner + U * (dh.abs() + dtotal.double().abs())
        val["dresidual"], tol["dresidual"] = dh, inner
        if mask is not None:
            keep, factor = stays(h.numel(), *mask)
            keep = torch.from_numpy(keep).view(h.shape).to(h.device)
            val["dx"] = torch.where(keep, dh * factor, 0.0)
            tol["dx"] = torch.where(keep, inner * factor + 2 * U * val["dx"].abs(), 0.0)
        val["dweight"] = (dy * u).sum(0)
        tol["dweight"] = (STEPS + rows / 152) * U * (dy * u).abs().sum(0)
    return val, tol


def e4m3_grid():
    """The values of e4m3 that are not negative, in order."""
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:-1], dtype=torch.float64)       # the last code is NaN


def check_8bit(q, scales, y, tol, block, powers):
    """q * scales is y (64 bits, off by at most tol) to half a step of e4m3 at its place; the scales are the blocks'
    largest magnitudes / 448, at least 2^-126, and, with powers, the next power of two."""
    y, tol = y.cpu(), tol.cpu()
    rows, width = y.shape
    size = block or width
    count = -(-width // size)
    s, got = scales.float().double().cpu(), q.float().double().cpu()
    assert s.shape == (rows, count) and bool(torch.isfinite(got).all())
    grid = e4m3_grid()
    step = torch.cat([grid[1:] - grid[:-1], grid[-1:] - grid[-2:-1]])
    for i in range(count):
        a, b = i * size, min(width, (i + 1) * size)
        most, off = y[:, a:b].abs().amax(1), tol[:, a:b].amax(1)
        low, high = (torch.clamp(v / 448, min=2.0 ** -126) for v in (most - off, most + off))
        if powers:
            low, high = (2.0 ** torch.ceil(torch.log2(v)) for v in (low, high))
            assert bool(((s[:, i] == low) | (s[:, i] == high)).all())
        else:   # the division is rounded once
            assert bool((s[:, i] >= low * (1 - 2 * U)).all()) and bool((s[:, i] <= high * (1 + 2 * U)).all())
        # a value is at most half a step from y / scale (its quotient is rounded twice); the step at its place is the
        # larger of those on its two sides
        t = got[:, a:b].abs()
        at = torch.searchsorted(grid, t.contiguous())
        assert bool((grid[at] == t).all())
        off = (y[:, a:b] / s[:, i:i + 1] - got[:, a:b]).abs()
        assert bool((off <= step[at] / 2 + 4 * U * t + tol[:, a:b] / s[:, i:i + 1]).all())


# ---------------------------------------------------------------------------
# log probabilities
# ---------------------------------------------------------------------------

def log_probs(logits, codes, temperature, top=0, grads=(None, None, None)):
    """({name: value}, {name: inner tolerance}) of log_probs, entropy, lse, top_log_probs, top_codes and, with the
    gradients of the first three, dlogits; on the CPU.

    z / T is a difference from the largest logit, rounded before and after its product with 1 / T (a float32 itself):
    4 roundings of |z - m| / T in all, which are a relative error of each exponential, with 2 units of the exponential
    itself; the sums' paths and what else is done are STEPS roundings of what is added."""
    z, inv = logits.double().cpu(), 1.0 / temperature
    rows, vocab = z.shape
    m = z.amax(1, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    d = (z - m) * inv
    lse0 = torch.logsumexp(d, 1, keepdim=True)
    alive = torch.isfinite(lse0)
    lp = torch.where(alive, d - lse0, -torch.inf)
    p = lp.exp()
    near = torch.where(p > 0, d.abs(), 0.0)
    rel = STEPS * U + 4 * U * (p * near).sum(1, keepdim=True)       # of a sum of exponentials
    off = 4 * U * near + rel + 4 * U * lse0.abs().nan_to_num(0.0, 0.0, 0.0)
    entropy = -torch.where(p > 0, p * lp, 0.0).sum(1, keepdim=True)
    # H = ln S - sum p d: its terms' sizes, each with the relative errors above
    size = (p * near).sum(1, keepdim=True)
    h_off = 2 * (STEPS * U + rel) * (1 + size) + 4 * U * (p * near * near).sum(1, keepdim=True)
    c = codes.cpu().long()
    there = (c >= 0) & (c < vocab)
    at = torch.where(there, c, 0)[:, None]
    val = {"log_probs": torch.where(there, lp.gather(1, at)[:, 0], 0.0), "entropy": entropy[:, 0],
           "lse": torch.where(alive, m * inv + lse0, -torch.inf)[:, 0]}
    at_off = 4 * U * (z.gather(1, at) - m).abs().nan_to_num(0.0, 0.0, 0.0) * inv + off.amin(1, keepdim=True)
    tol = {"log_probs": at_off[:, 0], "entropy": h_off[:, 0],
           "lse": (rel + 4 * U * ((m * inv).abs() + lse0.abs().nan_to_num(0.0, 0.0, 0.0)))[:, 0]}
    if top:
        order = torch.sort(z, stable=True, dim=1, descending=True)
        best, place = order.values[:, :top], order.indices[:, :top]
        real = best > -torch.inf
        fill = top - best.shape[1]
        val["top_codes"] = torch.nn.functional.pad(torch.where(real, place, -1), (0, max(0, fill)), value=-1)
        val["top_log_probs"] = torch.nn.functional.pad(torch.where(real, lp.gather(1, place), -torch.inf),
                                                       (0, max(0, fill)), value=-torch.inf)
        reach = torch.where(real, (best - m).abs() * inv, 0.0)
        tol["top_log_probs"] = torch.nn.functional.pad(4 * U * reach + off.amin(1, keepdim=True), (0, max(0, fill)))
    if any(g is not None for g in grads):
        gp, gh, gl = (torch.zeros(rows, 1, dtype=torch.float64) if g is None else g.double().cpu()[:, None] for g in grads)
        gp = torch.where(there[:, None], gp, 0.0)
        dead = ~alive | ((gp == 0) & (gh == 0) & (gl == 0))
        lp0 = torch.where(p > 0, lp, 0.0)
        one = torch.zeros_like(z).scatter_(1, at, 1.0)
        grad = gp * (one - p) + gl * p - gh * p * (lp0 + entropy)
        val["dlogits"] = torch.where(dead, 0.0, grad * inv)
        e_rel = 4 * U * near + rel
        size = p * (gp.abs() + gl.abs() + gh.abs() * (lp0.abs() + entropy))
        inner = size * (e_rel + STEPS * U) + gh.abs() * p * (off + h_off) + 4 * U * one * gp.abs()
        tol["dlogits"] = torch.where(dead, 0.0, inner * inv)
    return val, tol
