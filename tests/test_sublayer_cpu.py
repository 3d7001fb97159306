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


RMS = (4, 64, 1, 0, 1e-6)


def rms_call(lib, dims=RMS, x=AT, xs=64, r=None, rs=64, m=None, w=2 * AT, t=None, ts=64, y=3 * AT, ys=64, rstd=None, q=None):
    return lib.rvq_rms_norm(rq.rvq_norm_dims(*dims), ptr(x), xs, ptr(r), rs, None if m is None else ctypes.byref(m), ptr(w),
                            ptr(t), ts, ptr(y), ys, ptr(rstd), None if q is None else ctypes.byref(q), None)


def eight(values=5 * AT, stride=64, scales=6 * AT, block=32, kind=0):
    return rq.rvq_rms_8bit(values, stride, scales, block, kind)


def test_rms_norm_refusals(lib):
    for dims in ((-1, 64, 1, 0, 1e-5), (4, 0, 1, 0, 1e-5), (4, 64, 3, 0, 1e-5), (4, 64, -1, 0, 1e-5), (4, 64, 1, 2, 1e-5),
                 (4, 64, 0, 1, 1e-5), (4, 64, 1, 0, -1.0), (4, 64, 1, 0, float("nan"))):
        assert rms_call(lib, dims) == INVALID, dims
    assert rms_call(lib, (4, 16385, 1, 0, 1e-5), xs=20000, ys=20000) == UNSUPPORTED
    for kw in (dict(x=None), dict(y=None), dict(xs=63), dict(ys=63), dict(x=AT + 1), dict(y=AT + 1), dict(w=AT + 2),
               dict(rstd=AT + 2), dict(r=4 * AT, rs=63), dict(r=4 * AT + 1), dict(r=4 * AT, t=7 * AT, ts=63),
               dict(r=4 * AT, t=7 * AT + 1), dict(t=7 * AT),                       # nothing is added: the sum is x
               dict(m=mask(2.0)), dict(q=eight(values=None)), dict(q=eight(scales=None)), dict(q=eight(scales=AT + 2)),
               dict(q=eight(stride=63)), dict(q=eight(block=16)), dict(q=eight(block=-1)), dict(q=eight(kind=2))):
        assert rms_call(lib, **kw) == INVALID, kw
    assert rms_call(lib, (0, 64, 1, 0, 1e-5), x=None, y=None) == 0


def test_rms_norm_refuses_overlaps(lib):
    """Rows of 128 bytes; refused on the host."""
    far = dict(r=4 * AT, t=7 * AT)
    for kw in (dict(y=AT + 2), dict(y=AT, ys=65), dict(y=AT - 128), dict(r=4 * AT, y=4 * AT + 2), dict(far, t=AT + 2),
               dict(far, t=3 * AT), dict(far, t=4 * AT, ts=72), dict(y=2 * AT), dict(y=2 * AT + 128), dict(rstd=AT),
               dict(rstd=3 * AT + 8), dict(far, rstd=7 * AT), dict(q=eight(values=AT)), dict(q=eight(values=3 * AT + 500)),
               dict(q=eight(scales=AT + 8)), dict(q=eight(scales=5 * AT + 8)), dict(q=eight(scales=2 * AT)),
               dict(rstd=6 * AT, q=eight()), dict(far, m=mask(step=7 * AT + 8)), dict(m=mask(step=3 * AT))):
        assert rms_call(lib, **kw) == INVALID, kw


def test_rms_norm_backward_refusals(lib):
    need = lib.rvq_rms_norm_workspace_bytes(4, 64)
    assert need >= 4 * 64 * 4
    assert lib.rvq_rms_norm_workspace_bytes(-1, 64) == 0 and lib.rvq_rms_norm_workspace_bytes(4, 16385) == 0
    assert lib.rvq_rms_norm_workspace_bytes(4, 0) == 0 and lib.rvq_rms_norm_workspace_bytes(0, 64) > 0
    assert lib.rvq_rms_norm_workspace_bytes(10 ** 9, 16384) < 1 << 25

    def back(dims=RMS, dy=AT, dys=64, dt=None, dts=64, t=2 * AT, ts=64, m=None, w=3 * AT, rstd=4 * AT, dr=5 * AT, drs=64,
             dx=None, dxs=64, dw=6 * AT, ws=7 * AT, nb=need):
        return lib.rvq_rms_norm_backward(rq.rvq_norm_dims(*dims), ptr(dy), dys, ptr(dt), dts, ptr(t), ts,
                                         None if m is None else ctypes.byref(m), ptr(w), ptr(rstd), ptr(dr), drs, ptr(dx),
                                         dxs, ptr(dw), ptr(ws), nb, None)

    for kw in (dict(dy=None), dict(t=None), dict(rstd=None), dict(dys=63), dict(ts=63), dict(dt=8 * AT, dts=63), dict(drs=63),
               dict(dy=AT + 1), dict(t=AT + 1), dict(dt=AT + 1), dict(dr=AT + 1), dict(w=AT + 2), dict(dw=AT + 2),
               dict(rstd=AT + 2), dict(ws=None), dict(ws=7 * AT + 8), dict(nb=need - 1), dict(dx=8 * AT),
               dict(dx=8 * AT, m=mask(), dxs=63), dict(dx=8 * AT + 1, m=mask()), dict(m=mask(-1.0)),
               # overlaps
               dict(dr=AT + 2), dict(dr=2 * AT, drs=65), dict(dt=8 * AT, dr=8 * AT + 128), dict(dr=3 * AT), dict(dr=4 * AT),
               dict(dx=5 * AT, m=mask()), dict(dx=AT + 2, m=mask()), dict(dw=AT), dict(dw=5 * AT), dict(ws=AT), dict(ws=6 * AT),
               dict(dr=7 * AT + need - 128), dict(dx=8 * AT, m=mask(step=8 * AT))):
        assert back(**kw) == INVALID, kw
    assert back(dr=None, dw=None, ws=None, nb=0) == 0                  # nothing asked for


def test_log_probs_refusals(lib):
    ok = (4, 100, 0, 2, 1.0)

    def run(dims=ok, z=AT, zs=100, c=2 * AT, lp=3 * AT, h=None, lse=None, st=None, tl=None, tc=None, bad=None):
        return lib.rvq_log_probs(rq.rvq_log_probs_dims(*dims), ptr(z), zs, ptr(c), ptr(lp), ptr(h), ptr(lse), ptr(st), ptr(tl),
                                 ptr(tc), ptr(bad), None)

    for dims in ((-1, 100, 0, 2, 1.0), (4, 0, 0, 2, 1.0), (4, 100, -1, 2, 1.0), (4, 100, 0, 5, 1.0), (4, 100, 0, 2, 0.0),
                 (4, 100, 0, 2, -1.0), (4, 100, 0, 2, float("nan")), (4, 100, 0, 2, float("inf")), (4, 100, 0, 2, 1e-39)):
        assert run(dims) == INVALID, dims
    assert run((4, (1 << 20) + 1, 0, 2, 1.0), zs=1 << 21) == UNSUPPORTED
    assert run((4, 100, 65, 2, 1.0), tl=5 * AT, tc=6 * AT) == UNSUPPORTED
    top = dict(dims=(4, 100, 3, 2, 1.0), tl=5 * AT, tc=6 * AT)
    for kw in (dict(z=None), dict(z=AT + 1), dict(zs=99), dict(c=None), dict(lp=None), dict(c=None, lp=None), dict(c=AT + 2),
               dict(lp=3 * AT + 2), dict(h=AT + 2), dict(lse=AT + 2), dict(st=AT + 2), dict(bad=7 * AT + 4), dict(tl=5 * AT),
               dict(tc=5 * AT), dict(top, tl=None), dict(top, tc=None), dict(top, tl=5 * AT + 2), dict(top, tc=5 * AT + 2),
               # overlaps
               dict(lp=AT), dict(lp=AT + 796), dict(lp=2 * AT + 12), dict(h=3 * AT + 4), dict(lse=3 * AT - 12),
               dict(st=3 * AT - 28), dict(top, tc=5 * AT + 44), dict(top, tl=3 * AT - 44), dict(bad=3 * AT + 8), dict(bad=AT)):
        assert run(**kw) == INVALID, kw
    assert run((0, 100, 0, 2, 1.0), z=None, c=None, lp=None) == 0


def test_log_probs_backward_refusals(lib):
    def run(dims=(4, 100, 0, 2, 1.0), g=2 * AT, gh=None, gl=None, z=AT, zs=100, c=3 * AT, st=4 * AT, h=None, d=5 * AT, ds=100):
        return lib.rvq_log_probs_backward(rq.rvq_log_probs_dims(*dims), ptr(g), ptr(gh), ptr(gl), ptr(z), zs, ptr(c), ptr(st),
                                          ptr(h), ptr(d), ds, None)

    for kw in (dict(z=None), dict(st=None), dict(d=None), dict(c=None), dict(gh=6 * AT), dict(zs=99), dict(ds=99),
               dict(d=5 * AT + 1), dict(g=AT + 2), dict(gh=AT + 2, h=7 * AT), dict(gl=AT + 2), dict(st=AT + 2),
               dict(d=AT + 2), dict(d=AT, ds=101), dict(d=AT - 200), dict(d=2 * AT), dict(d=3 * AT), dict(d=4 * AT - 790),
               dict(gl=6 * AT, d=6 * AT), dict(gh=6 * AT, h=7 * AT, d=7 * AT)):
        assert run(**kw) == INVALID, kw
    assert run((0, 100, 0, 2, 1.0), z=None, st=None, d=None, c=None, g=None) == 0


# ---------------------------------------------------------------------------
# the device of a call
# ---------------------------------------------------------------------------

from test_predictor_edges_cpu import F32, I32, U8, OnGpu, Stream, gpus, kernels  # noqa: E402, F401


def operators(t):
    rows, one, w = (lambda: t(4, 8)), (lambda: t(4)), (lambda: t(8))
    step = lambda: t(1, dtype=torch.int64)  # noqa: E731

    def masked(call):
        """The mask's step is one of the tensors (a mask takes those that are on a GPU)."""
        def run(*tensors, **kw):
            m = rq.rvq_dropout_mask(0.1, 1)
            m.tensor = tensors[-1]
            return call(*tensors[:-1], m, **kw)
        return run

    return {
        "rvq_dropout": (masked(lambda x, y, r, m, **kw: rq.rvq_dropout(x, m, y, r, **kw)), [rows(), rows(), rows(), step()]),
        "rvq_rms_norm": (masked(lambda x, w, y, s, r, t, q, sc, m, **kw: rq.rvq_rms_norm(
            x, w, 1e-6, y, s, r, m, t, q, sc, 32, **kw)),
            [rows(), w(), rows(), one(), rows(), rows(), t(4, 8, dtype=torch.float8_e4m3fn), t(4, 1), step()]),
        "rvq_rms_norm_backward": (masked(lambda dy, t, w, s, dr, dw, ws, dt, dx, m, **kw: rq.rvq_rms_norm_backward(
            dy, t, w, s, dr, dw, ws, dt, m, dx, **kw)),
            [rows(), rows(), w(), one(), rows(), w(), t(64, dtype=U8), rows(), rows(), step()]),
        "rvq_log_probs": (lambda z, c, *out, **kw: rq.rvq_log_probs(z, c, 1.0, *out, **kw),
                          [rows(), t(4, dtype=I32), one(), one(), one(), t(4, 2), t(4, 3), t(4, 3, dtype=I32), step()]),
        "rvq_log_probs_backward": (lambda a, b, c, z, codes, s, h, d, **kw: rq.rvq_log_probs_backward(
            a, b, c, z, codes, 1.0, s, h, d, **kw),
            [one(), one(), one(), rows(), t(4, dtype=I32), t(4, 2), one(), rows()]),
    }


NAMES = sorted(operators(lambda *shape, dtype=F32: None))


@pytest.mark.parametrize("name", NAMES)
def test_calls_run_on_their_tensors_device(name, gpus):  # noqa: F811
    for index in (0, 1):
        call, tensors = operators(lambda *shape, dtype=F32: OnGpu(index, *shape, dtype=dtype))[name]
        call(*tensors)
        assert gpus.pop() == (name, index, 100 + index)
        call(*tensors, stream=Stream(index, 7))
        assert gpus.pop() == (name, index, 7)
        with pytest.raises(ValueError):
            call(*tensors, stream=Stream(1 - index, 7))
    assert not gpus


@pytest.mark.parametrize("name", NAMES)
def test_calls_refuse_tensors_of_two_devices(name, gpus):  # noqa: F811
    call, tensors = operators(lambda *shape, dtype=F32: OnGpu(0, *shape, dtype=dtype))[name]
    for i, t in enumerate(tensors):
        for other in (OnGpu(1, *t.shape, dtype=t.dtype), t.t):
            with pytest.raises(ValueError):
                call(*tensors[:i], other, *tensors[i + 1:])
    assert not gpus


@pytest.mark.parametrize("name", ["rvq_rms_backward.cu"])
def test_overlapping_kernels_take_no_read_only_pointers(name):
    """As for the other kernels that start while the one before them runs."""
    waiting = [(kernel, parameters, body) for kernel, parameters, body in kernels(name) if "griddep_wait" in body]
    assert waiting
    for kernel, parameters, body in waiting:
        assert "__restrict__" not in parameters and "__ldg(" not in body, kernel
