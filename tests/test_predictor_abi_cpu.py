"""The code predictor's entry points without a GPU: every refusal comes before
the CUDA runtime is touched, and workspace sizes are what the calls need."""

import ctypes

import pytest
import torch

import residual_vector_quantisation_gb300 as rq
from residual_vector_quantisation_gb300 import build as rqb

INVALID, UNSUPPORTED = -1, -2
P = ctypes.c_void_p(1 << 20)          # never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 1)


@pytest.fixture(scope="module")
def lib():
    rqb.build_library()
    return rq.load_library()


def test_layer_norm_refusals(lib):
    ok = rq.rvq_norm_dims(4, 64, 1, 0, 1e-5)

    def norm(dims=ok, x=P, xs=64, w=P, b=P, y=P, ys=64, mean=None, rstd=None):
        return lib.rvq_layer_norm(dims, x, xs, w, b, y, ys, mean, rstd, None)

    for dims in ((-1, 64, 1, 0, 1e-5), (4, 0, 1, 0, 1e-5), (4, 64, 3, 0, 1e-5), (4, 64, -1, 0, 1e-5),
                 (4, 64, 1, 2, 1e-5), (4, 64, 0, 1, 1e-5), (4, 64, 1, 0, -1.0), (4, 64, 1, 0, float("nan"))):
        assert norm(rq.rvq_norm_dims(*dims)) == INVALID, dims
    assert norm(rq.rvq_norm_dims(4, 16385, 1, 0, 1e-5), xs=20000, ys=20000) == UNSUPPORTED
    for kw in ({"x": None}, {"y": None}, {"xs": 63}, {"ys": 63}, {"x": ODD}, {"y": ODD}, {"w": ODD}, {"b": ODD},
               {"mean": ODD}, {"rstd": ODD}):
        assert norm(**kw) == INVALID, kw
    assert norm(rq.rvq_norm_dims(0, 64, 1, 0, 1e-5), x=None, y=None) == 0

    need = lib.rvq_layer_norm_workspace_bytes(4, 64)
    assert need >= 4 * 2 * 64 * 4
    assert lib.rvq_layer_norm_workspace_bytes(-1, 64) == 0
    assert lib.rvq_layer_norm_workspace_bytes(4, 16385) == 0
    assert lib.rvq_layer_norm_workspace_bytes(10 ** 9, 16384) < 1 << 27

    def back(dims=ok, dy=P, dys=64, x=P, xs=64, w=P, mean=P, rstd=P, dx=P, dxs=64, dw=P, db=P, ws=P, nb=need):
        return lib.rvq_layer_norm_backward(dims, dy, dys, x, xs, w, mean, rstd, dx, dxs, dw, db, ws, nb, None)

    for kw in ({"dy": None}, {"x": None}, {"mean": None}, {"rstd": None}, {"dys": 1}, {"xs": 1}, {"dxs": 1},
               {"dx": ODD}, {"dw": ODD}, {"db": ODD}, {"ws": None}, {"ws": ODD}, {"nb": need - 1}):
        assert back(**kw) == INVALID, kw
    assert back(dx=None, dw=None, db=None, ws=None, nb=0) == 0     # nothing asked for


def test_distill_refusals(lib):
    ok = rq.rvq_distill_dims(4, 100, 8, 2, 0, 1.0)

    def run(dims=ok, z=P, zs=100, t=P, c=P, lse=None, w=None, loss=P, out=None, d=P, ds=100, bad=None):
        return lib.rvq_distill(dims, z, zs, t, c, lse, w, loss, out, d, ds, bad, None)

    for dims in ((-1, 100, 8, 2, 0, 1.0), (4, 0, 8, 2, 0, 1.0), (4, 100, 0, 2, 0, 1.0), (4, 100, 8, 5, 0, 1.0),
                 (4, 100, 8, 2, 3, 1.0), (4, 100, 8, 2, 0, 0.0), (4, 100, 8, 2, 0, -1.0),
                 (4, 100, 8, 2, 0, float("nan")), (4, 100, 8, 2, 0, float("inf"))):
        assert run(rq.rvq_distill_dims(*dims)) == INVALID, dims
    assert run(rq.rvq_distill_dims(4, (1 << 20) + 1, 8, 2, 0, 1.0), zs=1 << 21, ds=1 << 21) == UNSUPPORTED
    assert run(rq.rvq_distill_dims(4, 100, 257, 2, 0, 1.0)) == UNSUPPORTED
    for kw in ({"z": None}, {"t": None}, {"c": None}, {"loss": None}, {"zs": 99}, {"ds": 99}, {"z": ODD}, {"t": ODD},
               {"c": ODD}, {"lse": ODD}, {"w": ODD}, {"loss": ODD}, {"out": ODD}, {"d": ODD}, {"bad": ODD}):
        assert run(**kw) == INVALID, kw
    assert run(rq.rvq_distill_dims(0, 100, 8, 2, 0, 1.0), z=None, t=None, c=None, loss=None, d=None) == 0

    def back(dims=ok, g=P, z=P, t=P, c=P, lse=P, d=P, ds=100):
        return lib.rvq_distill_backward(dims, g, z, 100, t, c, None, None, lse, d, ds, None)

    for kw in ({"g": ODD}, {"z": None}, {"t": None}, {"c": None}, {"lse": None}, {"lse": ODD}, {"d": None},
               {"ds": 99}):
        assert back(**kw) == INVALID, kw


def test_beam_refusals(lib):
    ok = rq.rvq_beam_dims(3, 4, 100, 4, 0, 1)
    need = lib.rvq_beam_workspace_bytes(ok)
    assert need > 0

    def run(dims=ok, z=P, zs=100, s=P, f=None, end=-1, o=P, p=P, c=P, of=None, ws=P, nb=need):
        return lib.rvq_beam_select(dims, z, zs, s, f, end, o, p, c, of, ws, nb, None)

    for dims in ((-1, 4, 100, 4, 0, 1), (3, 0, 100, 4, 0, 1), (3, 4, 0, 4, 0, 1), (3, 4, 100, 0, 0, 1),
                 (3, 4, 100, 4, 2, 1), (3, 4, 100, 4, 0, 3)):
        assert run(rq.rvq_beam_dims(*dims)) == INVALID, dims
        assert lib.rvq_beam_workspace_bytes(rq.rvq_beam_dims(*dims)) == 0
    for dims in ((3, 65, 100, 4, 0, 1), (3, 4, 100, 65, 0, 1), (3, 4, (1 << 24) + 1, 4, 0, 1),
                 (1 << 40, 4, 100, 4, 0, 1)):
        assert run(rq.rvq_beam_dims(*dims)) == UNSUPPORTED, dims
        assert lib.rvq_beam_workspace_bytes(rq.rvq_beam_dims(*dims)) == 0
    for kw in ({"z": None}, {"s": None}, {"o": None}, {"p": None}, {"c": None}, {"ws": None}, {"z": ODD}, {"s": ODD},
               {"o": ODD}, {"p": ODD}, {"c": ODD}, {"ws": ODD}, {"zs": 99}, {"nb": need - 1}, {"end": 100},
               {"end": -2}, {"f": P, "end": -1}):
        assert run(**kw) == INVALID, kw
    assert run(rq.rvq_beam_dims(0, 4, 100, 4, 0, 1), z=None, s=None, ws=None) == 0


def test_reorder_refusals(lib):
    ok = rq.rvq_beam_dims(3, 4, 100, 4, 0, 1)

    def state(src=1 << 20, dst=2 << 20, layers=1, row=16, gs=64, bs=16, dgs=64, dbs=16):
        return rq.rvq_beam_state(src, dst, layers, row, 0, gs, bs, 0, dgs, dbs)

    def run(*states, dims=ok, parents=P, n=None):
        array = (rq.rvq_beam_state * max(1, len(states)))(*states)
        return lib.rvq_beam_reorder(dims, parents, array, len(states) if n is None else n, None)

    assert run(state(), n=-1) == INVALID
    assert run(state(), n=rq.RVQ_BEAM_MAX_STATES + 1) == INVALID
    assert lib.rvq_beam_reorder(ok, P, None, 1, None) == INVALID
    assert run(state(), parents=None) == INVALID
    assert run(state(), parents=ODD) == INVALID
    assert run(state(src=None)) == INVALID
    assert run(state(dst=None)) == INVALID
    assert run(state(layers=-1)) == INVALID
    assert run(state(row=-1)) == INVALID
    assert run(state(dst=1 << 20, dgs=128)) == INVALID                        # in place, other strides
    assert run(state(dst=1 << 20), dims=rq.rvq_beam_dims(3, 4, 100, 5, 0, 1)) == INVALID
    assert run() == 0 and run(state(row=0)) == 0 and run(state(layers=0)) == 0


def test_python_side_refuses_cpu_tensors():
    x = torch.zeros((2, 8))
    with pytest.raises(ValueError):
        rq.rvq_layer_norm(x, None, None, 1e-5, x)
    with pytest.raises(ValueError):
        rq.rvq_distill(x, x, torch.zeros((2, 8), dtype=torch.int32), None, None, 1.0, torch.zeros(2))
    with pytest.raises(ValueError):
        rq.rvq_beam_states([(x.view(1, 2, 8), x.view(1, 2, 8))])
