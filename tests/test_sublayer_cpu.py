"""The sublayer's operators and log probabilities without a GPU: the generator's
numbers, and refusals, all of which come before the CUDA runtime is touched."""

import ctypes

import numpy as np
import pytest
import torch

import residual_vector_quantisation_gb300 as rq
import sublayer_ref as ref
from residual_vector_quantisation_gb300 import build as rqb

INVALID, UNSUPPORTED = -1, -2
AT = 1 << 24


def ptr(at):
    return ctypes.c_void_p(at)                # never dereferenced


ODD = ptr(AT + 1)


@pytest.fixture(scope="module")
def lib():
    rqb.build_library()
    return rq.load_library()


def test_generator_known_answers():
    """The published answers of Philox4x32-10, and the two statements of it against one another."""
    full = 0xFFFFFFFF
    assert ref.philox([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ref.philox([full] * 4, [full] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert ref.philox([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]
    seed, offset, step, first = 0x123456789ABCDEF0, (3 << 40) + 5, 77, 8 * ((1 << 33) + 5) + 3
    upper = offset + (step << 32)
    for p in (0.1, 0.5, 0.999):
        keep, factor = ref.stays(40, p, seed, offset, step, first)
        drop = round(p * 65536)
        assert factor == 65536 / (65536 - drop)
        for i in range(40):
            g = (first + i) // 8
            words = ref.philox([g & full, g >> 32, upper & full, upper >> 32], [seed & full, seed >> 32])
            assert bool(keep[i]) == ((words[(first + i) % 8 // 2] >> 16 * ((first + i) % 2)) & 0xFFFF >= drop)


def test_masks_have_their_probability_and_are_their_own():
    n = 200000
    first, _ = ref.stays(n, 0.25, 1)
    assert abs(first.mean() - 0.75) < 6 * (0.25 * 0.75 / n) ** 0.5
    for other in (dict(seed=2), dict(seed=1, offset=1), dict(seed=1, step=1)):
        second, _ = ref.stays(n, 0.25, **other)
        both = np.mean(first & second)
        assert abs(both - 0.75 ** 2) < 6 * (0.75 ** 2 * (1 - 0.75 ** 2) / n) ** 0.5


def mask(p=0.1, seed=1, offset=0, step=None):
    m = rq.rvq_dropout_mask(p, seed, offset)
    m.step = step
    return m


def test_mask_refusals():
    for kw in (dict(seed=-1), dict(seed=1 << 64), dict(seed=1, offset=-1), dict(seed=1, offset=1 << 64)):
        with pytest.raises(ValueError):
            rq.rvq_dropout_mask(0.1, **kw)
    for step in (torch.zeros(1, dtype=torch.int64), 7):
        with pytest.raises((ValueError, AttributeError)):
            rq.rvq_dropout_mask(0.1, 1, 0, step)


def test_dropout_refusals(lib):
    def run(rows=4, width=64, dtype=1, x=AT, xs=64, r=None, rs=64, m=mask(), y=2 * AT, ys=64):
        return lib.rvq_dropout(rq.rvq_dropout_dims(rows, width, dtype), ptr(x), xs, ptr(r), rs,
                               None if m is None else ctypes.byref(m), ptr(y), ys, None)

    for kw in (dict(rows=-1), dict(width=-1), dict(dtype=3), dict(dtype=-1), dict(x=None), dict(y=None), dict(m=None),
               dict(x=AT + 1), dict(y=AT + 1), dict(r=AT + 1), dict(xs=63), dict(ys=63), dict(r=3 * AT, rs=63),
               dict(m=mask(-0.1)), dict(m=mask(1.1)), dict(m=mask(float("nan"))), dict(m=mask(step=AT + 4))):
        assert run(**kw) == INVALID, kw
    assert run(rows=1 << 40, width=1 << 40, xs=1 << 40, ys=1 << 40) == UNSUPPORTED
    assert run(rows=0, x=None, y=None) == 0 and run(width=0, x=None, y=None) == 0
    # outputs that meet their inputs anywhere but row by row
    for kw in (dict(y=AT + 2), dict(y=AT, ys=65), dict(y=AT - 128), dict(x=3 * AT, r=AT, y=AT + 2), dict(r=2 * AT, rs=65),
               dict(m=mask(step=2 * AT + 8))):
        assert run(**kw) == INVALID, kw
