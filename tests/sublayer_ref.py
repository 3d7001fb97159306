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
