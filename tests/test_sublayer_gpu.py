"""The sublayer's operators (dropout, root-mean-square norm) on the GPU against
plain 64-bit statements of them (sublayer_ref)."""

import math

import pytest
import torch

import sublayer_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import residual_vector_quantisation_gb300 as rq  # noqa: E402
from residual_vector_quantisation_gb300 import build as rqb  # noqa: E402

DEV = torch.device("cuda:0")
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def library():
    rqb.build_library()
    rq.load_library()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def rows_in(t, pad, shift):
    """The same rows, `pad` elements of NaN after each, the first `shift` elements into a buffer of NaN."""
    rows, width = t.shape
    buffer = torch.full((rows * (width + pad) + shift + 16,), NAN, dtype=t.dtype, device=t.device)
    view = buffer.as_strided((rows, width), (width + pad, 1), shift)
    view.copy_(t)
    return view


def untouched(view):
    """What lies beside the rows of rows_in is NaN as before."""
    buffer = torch.empty(0, dtype=view.dtype, device=DEV).set_(view.untyped_storage())
    held = buffer.clone()
    held.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(NAN)
    return bool(torch.isnan(held).all())


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------

def step_of(n):
    return torch.tensor([n], dtype=torch.int64, device=DEV)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width,pad,shift", [(1, 1, 0, 0), (1, 7, 0, 0), (1, 8, 0, 0), (3, 5, 0, 1), (5, 64, 0, 0),
                                                  (5, 64, 8, 0), (7, 40, 3, 0), (9, 33, 7, 5), (2, 4096, 0, 3),
                                                  (300, 1000, 0, 0), (300, 1000, 24, 8), (41, 1025, 6, 0)])
def test_dropout_sizes(rows, width, pad, shift, dtype):
    g = gen(rows + width)
    x, r = randn(g, rows, width).to(dtype), randn(g, rows, width).to(dtype)
    for p, seed, offset, step, res in ((0.1, 5, 3, None, False), (0.5, (1 << 63) + 9, 1 << 35, 12345, True),
                                       (0.0, 1, 0, None, True), (0.9, 3, 0, -1, False)):
        mask = rq.rvq_dropout_mask(p, seed, offset, None if step is None else step_of(step))
        val, tol = ref.dropout(x, (p, seed, offset, step or 0), r if res else None)
        y = rows_in(torch.zeros_like(x), pad, shift)
        rq.rvq_dropout(rows_in(x, pad, shift), mask, y, rows_in(r, pad, shift) if res else None)
        ref.check(y, val, tol, (p, res))
        assert untouched(y)
        assert bool((y[val == 0] == 0).all())
        # tensors that lie differently get the same mask
        other = rows_in(torch.zeros_like(x), pad + 1, shift + 1)
        rq.rvq_dropout(x, mask, other, rows_in(r, 1, 0) if res else None)
        assert torch.equal(other, y) and untouched(other)


@pytest.mark.parametrize("dtype", TYPES)
def test_dropout_in_place_and_what_is_dropped(dtype):
    g = gen(3)
    x, r = randn(g, 50, 96).to(dtype), randn(g, 50, 96).to(dtype)
    mask = rq.rvq_dropout_mask(0.3, 8)
    keep = torch.from_numpy(ref.stays(x.numel(), 0.3, 8)[0]).view(x.shape).to(DEV)
    want, with_r = torch.empty_like(x), torch.empty_like(x)
    rq.rvq_dropout(x, mask, want)
    rq.rvq_dropout(x, mask, with_r, r)
    # infinities and NaN in dropped places are gone
    bad = torch.where(keep, x, torch.where(randn(g, 50, 96) > 0, INF, NAN).to(dtype))
    rq.rvq_dropout(bad, mask, bad)
    assert torch.equal(bad, want)
    y = r.clone()
    rq.rvq_dropout(x, mask, y, y)
    assert torch.equal(y, with_r)
    # where all is dropped the residual is left, whatever x holds
    rq.rvq_dropout(torch.full_like(x, NAN), rq.rvq_dropout_mask(1.0, 8), y, r)
    assert torch.equal(y, r)
    rq.rvq_dropout(x, rq.rvq_dropout_mask(0.0, 8), y)
    assert torch.equal(y, x)


def test_dropout_past_32_bits():
    """More than 2^31 elements, and counters past 32 bits of groups are looked at through the offsets of a long row."""
    n = (1 << 31) + 4099
    x = torch.ones((1, n), dtype=BF16, device=DEV)
    mask = rq.rvq_dropout_mask(0.5, 77, 5)
    for res in (None, x):
        y = torch.empty_like(x)
        rq.rvq_dropout(x, mask, y, res)
        for first in (0, (1 << 31) - 64, n - 5000):
            keep, factor = ref.stays(min(5000, n - first), 0.5, 77, 5, 0, first)
            got = y[0, first:first + len(keep)].float().cpu() - (0 if res is None else 1)
            assert torch.equal(got, torch.from_numpy(keep).float() * factor)
    # rows that lie apart, elements one by one
    rows = torch.ones((3, (1 << 30) + 3), dtype=BF16, device=DEV)[:, 1:]
    y = torch.zeros_like(rows)
    rq.rvq_dropout(rows, mask, y)
    width = rows.shape[1]
    for at in (0, width - 50, width * 2 - 50, width * 3 - 50):
        keep, factor = ref.stays(50, 0.5, 77, 5, 0, at)
        assert torch.equal(y.reshape(-1)[at:at + 50].float().cpu(), torch.from_numpy(keep).float() * factor)


def test_dropout_gradients_and_steps():
    """The gradient is the forward pass's mask; a step counted up between the passes is an error and not another mask."""
    g = gen(4)
    x, r = (randn(g, 6, 5, 40).requires_grad_() for _ in range(2))
    step = step_of(3)
    mask = rq.rvq_dropout_mask(0.2, 9, 1, step)
    up = randn(g, 6, 5, 40)
    y = rq.dropout(x, mask, r)
    val, tol = ref.dropout(x.detach().view(30, 40), (0.2, 9, 1, 3), r.detach().view(30, 40))
    ref.check(y.detach().view(30, 40), val, tol, "y")
    y.backward(up)
    val, tol = ref.dropout(up.view(30, 40), (0.2, 9, 1, 3))
    ref.check(x.grad.view(30, 40), val, tol, "dx")
    assert torch.equal(r.grad, up)
    # tensors whose last axis is not contiguous: the mask goes by the elements' order
    t = x.detach().transpose(0, 2)
    assert torch.equal(rq.dropout(t, mask), rq.dropout(t.contiguous(), mask))
    y = rq.dropout(x, mask)
    step.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward(up)
    assert not torch.equal(rq.dropout(x, mask), y)
    assert rq.dropout(x[:0], mask, r[:0]).shape == (0, 5, 40)
    with pytest.raises(ValueError):
        rq.dropout(x, mask, r[:1])


def test_dropout_graph_counts_its_steps():
    """A captured training step: forward, backward and the count, a new mask at each replay."""
    x = torch.ones((30, 64), device=DEV)
    step, dy = step_of(0), torch.full((30, 64), 2.0, device=DEV)
    mask = rq.rvq_dropout_mask(0.5, 11, 2, step)
    y, dx = torch.empty_like(x), torch.empty_like(x)

    def both():
        rq.rvq_dropout(x, mask, y)
        rq.rvq_dropout(dy, mask, dx)
        step.add_(1)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    seen = []
    for k in range(1, 4):
        graph.replay()
        torch.cuda.synchronize()
        assert step.item() == k + 1
        val, _ = ref.dropout(x, (0.5, 11, 2, k))
        assert torch.equal(y.double(), val) and torch.equal(dx.double(), 2 * val)
        seen.append(y.clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


# ---------------------------------------------------------------------------
# root-mean-square norm
# ---------------------------------------------------------------------------

MASK = (0.2, 17, 4, 2)


def mask_of(m):
    return None if m is None else rq.rvq_dropout_mask(m[0], m[1], m[2], step_of(m[3]))


def run_rms(x, w, eps, dy, r=None, m=None, dt=None, place=lambda t: t.clone()):
    """Both passes, every tensor where `place` puts it; outputs hold NaN before."""
    rows, width = x.shape
    mask = mask_of(m)
    out = {"y": place(torch.full_like(x, NAN))}
    if r is not None or mask is not None:
        out["total"] = place(torch.full_like(x, NAN))
    rstd = torch.full((rows,), NAN, device=DEV)
    xv, rv = place(x), None if r is None else place(r)
    rq.rvq_rms_norm(xv, w, eps, out["y"], rstd, rv, mask, out.get("total"))
    total = out.get("total", xv)
    out["dresidual"] = place(torch.full_like(x, NAN))
    if mask is not None:
        out["dx"] = place(torch.full_like(x, NAN))
    out["dweight"] = None if w is None else torch.full_like(w, NAN)
    need = rq.rvq_rms_norm_workspace_bytes(rows, width)
    buffer = torch.full((need + (1 << 16),), 0xFF, dtype=torch.uint8, device=DEV)
    rq.rvq_rms_norm_backward(place(dy), total, w, rstd, out["dresidual"], out["dweight"], buffer[:need],
                             None if dt is None else place(dt), mask, out.get("dx"))
    assert bool((buffer[need:] == 0xFF).all())
    return out


def check_rms(got, x, w, eps, dy, r=None, m=None, dt=None):
    total = ref.total_of(x, m, r)
    if "total" in got:
        assert torch.equal(got["total"], total)
    val, tol = ref.rms(total, w, eps, dy, dt, m)
    for k in val:
        if got[k] is not None:
            ref.check(got[k], val[k], tol[k], k)


def make_rms(rows, width, dtype, pdtype):
    g = gen(rows * 31 + width)
    x, r, dy, dt = (randn(g, rows, width).to(dtype) for _ in range(4))
    return x, r, dy, dt, (1 + 0.2 * randn(g, width)).to(pdtype)


@pytest.mark.parametrize("dtype,pdtype", [(F32, F32), (BF16, F32), (BF16, BF16), (F16, F32), (F16, F16)])
@pytest.mark.parametrize("rows,width", [(1, 1), (1, 1024), (3, 7), (5, 33), (130, 256), (700, 768), (9, 1000), (33, 1024),
                                        (6, 1025), (17, 1032), (4, 2048), (3, 4097), (200, 1500), (2, 8200), (5, 12288),
                                        (3, 13400), (2, 16384), (2, 16383)])
def test_rms_sizes(rows, width, dtype, pdtype):
    x, r, dy, dt, w = make_rms(rows, width, dtype, pdtype)
    check_rms(run_rms(x, w, 1e-6, dy), x, w, 1e-6, dy)
    check_rms(run_rms(x, w, 1e-6, dy, r, None, dt), x, w, 1e-6, dy, r, None, dt)
    check_rms(run_rms(x, w, 1e-6, dy, r, MASK, dt), x, w, 1e-6, dy, r, MASK, dt)
    check_rms(run_rms(x, w, 1e-6, dy, None, MASK), x, w, 1e-6, dy, None, MASK)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (5, 7)])
@pytest.mark.parametrize("width", [1, 9, 40, 250, 500, 1024, 1500, 9000])
def test_rms_strides_and_alignment(width, pad, shift, dtype):
    rows = 37 if width < 5000 else 9
    x, r, dy, dt, w = make_rms(rows, width, dtype, F32)
    placed = []

    def place(t):
        placed.append(rows_in(t, pad, shift))
        return placed[-1]

    check_rms(run_rms(x, w, 1e-6, dy, r, MASK, dt, place), x, w, 1e-6, dy, r, MASK, dt)
    check_rms(run_rms(x, w, 1e-6, dy, r, None, dt, place), x, w, 1e-6, dy, r, None, dt)
    assert all(untouched(t) for t in placed)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [5, 100, 768, 1025, 5000])
def test_rms_tensors_that_lie_differently(width, dtype):
    x, r, dy, dt, w = make_rms(21, width, dtype, F32)
    placed = []

    def place(t):
        placed.append(rows_in(t, len(placed) % 5, 3 * len(placed) % 8))
        return placed[-1]

    check_rms(run_rms(x, w, 1e-6, dy, r, MASK, dt, place), x, w, 1e-6, dy, r, MASK, dt)
    assert all(untouched(t) for t in placed)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [1, 8, 48, 96, 130, 248, 256, 257, 352, 512, 519])
def test_rms_narrow_rows_share_a_warp(width, dtype):
    """Row counts that leave a warp's last rows, and a block's, without work."""
    for rows in (1, 7, 153, 1219, 5003):
        x, r, dy, dt, w = make_rms(rows, width, dtype, F32)
        check_rms(run_rms(x, w, 1e-6, dy, r, MASK, dt), x, w, 1e-6, dy, r, MASK, dt)
        check_rms(run_rms(x, w, 1e-6, dy), x, w, 1e-6, dy)


@pytest.mark.parametrize("width", [96, 1024, 3000])
def test_rms_without_weight_in_place_and_parts(width):
    x, r, dy, dt, w = make_rms(41, width, F32, F32)
    check_rms(run_rms(x, None, 1e-6, dy, r, MASK, dt), x, None, 1e-6, dy, r, MASK, dt)
    want = run_rms(x, w, 1e-6, dy, r, MASK, dt)
    mask = mask_of(MASK)
    # the sum over the residual and the result over x, and the other way round
    for swap in (False, True):
        xx, rr = x.clone(), r.clone()
        y, total = (rr, xx) if swap else (xx, rr)
        rstd = torch.empty(41, device=DEV)
        rq.rvq_rms_norm(xx, w, 1e-6, y, rstd, rr, mask, total)
        assert torch.equal(y, want["y"]) and torch.equal(total, want["total"])
    # gradients over what they are made from, and each of them alone
    for over in range(3):
        t = [dy.clone(), want["total"].clone(), dt.clone()]
        dx = t[(over + 1) % 3]
        rq.rvq_rms_norm_backward(t[0], t[1], w, rstd, t[over], None, None, t[2], mask, dx)
        assert torch.equal(t[over], want["dresidual"]) and torch.equal(dx, want["dx"])
    ws = torch.empty(rq.rvq_rms_norm_workspace_bytes(41, width), dtype=torch.uint8, device=DEV)
    for k in ("dresidual", "dx", "dweight"):
        out = {n: None for n in ("dresidual", "dx", "dweight")}
        out[k] = torch.empty_like(want[k])
        rq.rvq_rms_norm_backward(dy, want["total"], w, rstd, out["dresidual"], out["dweight"], ws, dt, mask, out["dx"])
        assert torch.equal(out[k], want[k]), k


def test_rms_odd_values_and_no_rows():
    x, _, dy, _, w = make_rms(7, 512, F32, F32)
    x[1] = 0.0                      # the norm of zeros: eps alone
    x[2] = 1e-30
    x[3] *= 1e15
    x[4, 17] = NAN
    x[5, 3] = INF
    x[6] = 3e19                     # its square is past float32: infinite, and the result zero
    got = run_rms(x, w, 1e-6, dy)
    val, tol = ref.rms(x[:4], w, 1e-6, dy[:4])
    ref.check(got["y"][:4], val["y"], tol["y"] + 1e-38, "y")
    ref.check(got["dresidual"][:4], val["dresidual"], tol["dresidual"], "dresidual")
    assert bool(torch.isnan(got["y"][4]).all()) and bool(torch.isnan(got["dresidual"][4:6]).all())
    assert bool(torch.isnan(got["y"][5, 3])) and bool((got["y"][5, :3] == 0).all()) and bool((got["y"][6] == 0).all())
    empty = torch.empty((0, 64), device=DEV)
    w = torch.ones(64, device=DEV)
    assert bool((run_rms(empty, w, 1e-6, empty)["dweight"] == 0).all())


def test_rms_many_rows_and_repeats():
    x, r, dy, dt, w = make_rms(20011, 192, BF16, F32)
    one = run_rms(x, w, 1e-6, dy, r, MASK, dt)
    check_rms(one, x, w, 1e-6, dy, r, MASK, dt)
    two = run_rms(x, w, 1e-6, dy, r, MASK, dt)
    for k in one:
        assert torch.equal(one[k], two[k]), k


def run_8bit(x, w, r, block, powers, pad=0, shift=0, m=None):
    rows, width = x.shape
    count = -(-width // block) if block else 1
    buffer = torch.full((rows * (width + pad) + shift + 16,), 0x5A, dtype=torch.uint8, device=DEV)
    q = buffer.as_strided((rows, width), (width + pad, 1), shift).view(torch.float8_e4m3fn)
    scales = torch.full((rows, count), NAN, device=DEV).to(torch.float8_e8m0fnu if powers else F32)
    total = None if r is None else torch.empty_like(x)
    xv = rows_in(x, pad, shift)
    rq.rvq_rms_norm(xv, w, 1e-6, None, None, None if r is None else rows_in(r, pad, shift), mask_of(m),
                    None if total is None else rows_in(total, pad, shift), q, scales, block)
    held = buffer.clone()
    held.as_strided((rows, width), (width + pad, 1), shift).fill_(0x5A)
    assert bool((held == 0x5A).all())
    return q, scales


@pytest.mark.parametrize("powers", [False, True])
@pytest.mark.parametrize("block", [0, 32, 64, 128])
@pytest.mark.parametrize("dtype", TYPES)
def test_rms_8bit(dtype, block, powers):
    for rows, width, pad, shift in ((1, 1, 0, 0), (3, 31, 0, 0), (5, 64, 0, 0), (700, 200, 0, 0), (9, 768, 16, 0),
                                    (33, 1024, 0, 0), (5, 1025, 6, 0), (6, 1100, 0, 0), (7, 1100, 3, 5), (4, 520, 2, 1),
                                    (3, 5000, 0, 0), (2, 5003, 1, 3), (2, 16384, 0, 0), (2, 16383, 0, 0), (1200, 40, 1, 1)):
        g = gen(rows + width)
        x, r = (randn(g, rows, width).to(dtype) for _ in range(2))
        x *= torch.exp(randn(g, rows, width)).to(dtype)
        w = 1 + 0.2 * randn(g, width)
        for res in (None, r):
            val, tol = ref.rms(ref.total_of(x, None, res), w, 1e-6)
            q, s = run_8bit(x, w, res, block, powers, pad, shift)
            ref.check_8bit(q, s, val["y"], tol["y"], block, powers)


def test_rms_8bit_beside_y_with_a_mask_and_odd_values():
    g = gen(5)
    x, r = randn(g, 6, 256).to(BF16), randn(g, 6, 256).to(BF16)
    w = 1 + 0.2 * randn(g, 256)
    val, tol = ref.rms(ref.total_of(x, MASK, r), w, 1e-6)
    q, s = run_8bit(x, w, r, 64, True, m=MASK)
    ref.check_8bit(q, s, val["y"], tol["y"], 64, True)
    y, q2, s2 = torch.empty_like(x), torch.empty_like(q), torch.empty_like(s)
    rq.rvq_rms_norm(x, w, 1e-6, y, None, r, mask_of(MASK), None, q2, s2, 64)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s.view(torch.uint8), s2.view(torch.uint8))
    ref.check(y, val["y"], tol["y"], "y")
    # a block of zeros, a NaN in one row, and a weight that makes one block's values overflow
    x = randn(g, 4, 256)
    x[1] = 0.0
    x[2, 7] = NAN
    w = torch.ones(256, device=DEV)
    w[64:128] = INF
    for powers in (False, True):
        q, s = run_8bit(x, w, None, 64, powers)
        q, s = q.float(), s.float()
        assert bool((s[1, [0, 2, 3]] == 2.0 ** -126).all()) and bool((q[1, 128:] == 0).all())
        assert bool(torch.isnan(s[2]).all()) and bool(torch.isnan(q[2]).all())
        assert bool(torch.isnan(s[0, 1]) if powers else torch.isinf(s[0, 1])) and bool(torch.isnan(q[0, 64:128]).all())
        assert bool(torch.isfinite(q[0, :64]).all()) and bool(torch.isfinite(q[0, 128:]).all())


def test_rms_8bit_scales_at_their_borders():
    """Largest magnitudes of 448 * 2^k and its neighbours: the next power of two, no value past the type's largest."""
    eps = 1e-6                                 # run_8bit's
    for k in (-9, -1, 0, 3):
        for ulps in (-1, 0, 1):
            x = torch.zeros((1, 64), device=DEV)
            w = torch.zeros(64, device=DEV)
            x[0, 0] = 1.0                      # rstd is about 8
            rstd = torch.empty(1, device=DEV)
            y = torch.empty_like(x)
            rq.rvq_rms_norm(x, torch.ones(64, device=DEV), eps, y, rstd)
            target = torch.tensor(448.0 * 2.0 ** k)
            for _ in range(abs(ulps)):
                target = torch.nextafter(target, torch.tensor(INF if ulps > 0 else 0.0))
            # a weight whose product with y is the target, where there is one
            w0 = (target.double() / y[0, 0].double().cpu()).float()
            for d in range(-2, 3):
                c = w0
                for _ in range(abs(d)):
                    c = torch.nextafter(c, torch.tensor(INF if d > 0 else 0.0))
                w[0] = c
                q, s = run_8bit(x, w, None, 32, True)
                most = (y[0, 0] * w[0]).double().item()
                want = 2.0 ** math.ceil(math.log2(most / 448))
                assert s[0, 0].float().item() == want and abs(q[0, 0].float().item()) <= 448.0


def test_rms_autograd():
    g = gen(9)
    x, r, up, ut = (randn(g, 2, 9, 64) for _ in range(4))
    w = 1 + 0.2 * randn(g, 64)
    flat = [t.view(18, 64) for t in (x, r, up, ut)]
    for res, m in ((False, None), (True, None), (False, MASK), (True, MASK)):
        xs, rs, ws = (t.clone().requires_grad_() for t in (x, r, w))
        out = rq.rms_norm(xs, ws, 1e-6, rs if res else None, mask_of(m))
        both = isinstance(out, tuple)
        assert both == (res or m is not None)
        torch.autograd.backward(out, (up, ut) if both else (up,))
        val, tol = ref.rms(ref.total_of(flat[0], m, flat[1] if res else None), w, 1e-6, flat[2], flat[3] if both else None, m)
        ref.check(xs.grad.view(18, 64), val["dx" if m else "dresidual"], tol["dx" if m else "dresidual"], "dx")
        ref.check(ws.grad, val["dweight"], tol["dweight"], "dweight")
        if res:
            ref.check(rs.grad.view(18, 64), val["dresidual"], tol["dresidual"], "dresidual")
    # the sum alone is used, or the result alone
    xs, rs = x.clone().requires_grad_(), r.clone().requires_grad_()
    rq.rms_norm(xs, w, 1e-6, rs)[1].backward(ut)
    assert torch.equal(xs.grad, ut) and torch.equal(rs.grad, ut)
    xs.grad = None
    rq.rms_norm(xs, w, 1e-6, r)[0].backward(up)
    val, tol = ref.rms(ref.total_of(flat[0], None, flat[1]), w, 1e-6, flat[2])
    ref.check(xs.grad.view(18, 64), val["dresidual"], tol["dresidual"], "dx")
    with pytest.raises(ValueError):
        rq.rms_norm_8bit(xs, w)
    with torch.no_grad():
        q, s, total = rq.rms_norm_8bit(xs, w, 1e-6, r, 32, True)
    assert q.shape == x.shape and s.shape == (2, 9, 2) and torch.equal(total, x + r)
    val, tol = ref.rms(total.view(18, 64), w, 1e-6)
    ref.check_8bit(q.view(18, 64), s.view(18, 2), val["y"], tol["y"], 32, True)


def test_rms_gradient_against_differences():
    """d sum(c * y + d * total) along a direction, by differences of the 64-bit statement."""
    g = gen(10)
    x, r, up, ut, dx, dr = (randn(g, 5, 40).double() for _ in range(6))
    w, dw = 1 + 0.2 * randn(g, 40).double(), randn(g, 40).double()
    keep, factor = ref.stays(200, *MASK)
    keep = torch.from_numpy(keep).view(5, 40).to(DEV)

    def value(t):
        h = torch.where(keep, (x + t * dx) * factor, 0.0) + r + t * dr
        return (h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * (w + t * dw) * up + h * ut).sum().item()

    step = 1e-5
    want = (value(step) - value(-step)) / (2 * step)
    xs, rs, ws = (t.float().requires_grad_() for t in (x, r, w))
    torch.autograd.backward(rq.rms_norm(xs, ws, 1e-6, rs, mask_of(MASK)), (up.float(), ut.float()))
    terms = [(xs.grad.double() * dx), (rs.grad.double() * dr), (ws.grad.double() * dw)]
    got, size = sum(t.sum().item() for t in terms), sum(t.abs().sum().item() for t in terms)
    # the inputs' rounding and the gradient's (64 roundings of 2^-24 each), and the differences' own error of about step^2
    assert abs(got - want) <= size * (128 * ref.U + 1e-8), (got, want)


def test_rms_two_streams_at_once_and_a_graph():
    x, r, dy, dt, w = make_rms(3000, 520, BF16, F32)
    want = run_rms(x, w, 1e-6, dy, r, MASK, dt)
    q_want = run_8bit(x, w, r, 32, True)
    torch.cuda.synchronize()
    got = []
    for s in [torch.cuda.Stream() for _ in range(2)]:
        with torch.cuda.stream(s):
            got.append((run_rms(x, w, 1e-6, dy, r, MASK, dt), run_8bit(x, w, r, 32, True)))
    torch.cuda.synchronize()
    for a, q in got:
        for k in want:
            assert torch.equal(a[k], want[k]), k
        for u, v in zip(q, q_want):
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))
    # a training step through autograd, captured: a new mask at each replay, the gradients those of its own
    step, grads = step_of(0), []
    leaves = [t.float().clone().requires_grad_() for t in (x[:40], r[:40], w)]
    mask = rq.rvq_dropout_mask(0.2, 3, 1, step)

    def train():
        y, total = rq.rms_norm(leaves[0], leaves[2], 1e-6, leaves[1], mask)
        out = torch.autograd.grad((y.square().sum() + total.sum()), leaves)
        step.add_(1)
        return [y, total, *out]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = train()
    for k in (1, 2):
        graph.replay()
        torch.cuda.synchronize()
        total = ref.total_of(leaves[0].detach(), (0.2, 3, 1, k), leaves[1].detach())
        assert torch.equal(captured[1], total)
        grads.append([t.clone() for t in captured])
        step.fill_(k)
        for a, b in zip(train(), grads[-1]):
            assert torch.equal(a, b)
    assert not torch.equal(grads[0][1], grads[1][1])


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def test_a_predictor_is_trained_scored_and_distilled():
    """Two sublayers (drop, add, norm), a head, log probabilities with entropy, one step of a policy's loss, the lists of
    a teacher, a distillation step and a beam step on the scores; the gradients against the same in 64 bits."""
    g = gen(21)
    rows, width, vocab = 60, 64, 90
    x0, f0, f1 = (randn(g, rows, width) for _ in range(3))
    w = [(1 + 0.2 * randn(g, width)) for _ in range(2)]
    head = randn(g, vocab, width) / 8
    codes = torch.randint(-1, vocab, (rows,), generator=g, device=DEV)
    gain = randn(g, rows)
    step = step_of(5)
    masks = [rq.rvq_dropout_mask(0.1, 33, place, step) for place in range(2)]
    keeps = [tuple(torch.as_tensor(v, device=DEV) for v in ref.stays(rows * width, 0.1, 33, place, 5)) for place in range(2)]

    def model(x, f, g2, wa, wb, ours):
        if ours:
            y, total = rq.rms_norm(f, wa, 1e-6, x, masks[0])
            y, total = rq.rms_norm(g2 + y, wb, 1e-6, total, masks[1])
        else:
            total = torch.where(keeps[0][0].view(rows, width), f * keeps[0][1], 0.0) + x
            y = total / torch.sqrt((total * total).mean(1, keepdim=True) + 1e-6) * wa
            total = torch.where(keeps[1][0].view(rows, width), (g2 + y) * keeps[1][1], 0.0) + total
            y = total / torch.sqrt((total * total).mean(1, keepdim=True) + 1e-6) * wb
        return y

    def loss_of(leaves, ours):
        logits = model(*leaves[:5], ours) @ leaves[5].t()
        if ours:
            out = rq.log_probs(logits, codes, entropy=True)
            return -(gain * out.log_probs).sum() - 0.1 * out.entropy.sum() + 0.01 * (out.lse ** 2).sum(), logits
        lp = torch.log_softmax(logits, 1)
        at = torch.where(codes >= 0, lp.gather(1, codes.clamp(min=0)[:, None])[:, 0], 0.0)
        entropy = -(lp.exp() * lp).sum(1)
        return -(gain * at).sum() - 0.1 * entropy.sum() + 0.01 * (torch.logsumexp(logits, 1) ** 2).sum(), logits

    plain = [t.double().requires_grad_() for t in (x0, f0, f1, *w, head)]
    leaves = [t.clone().requires_grad_() for t in (x0, f0, f1, *w, head)]
    loss, logits = loss_of(leaves, True)
    loss.backward()
    loss_of(plain, False)[0].backward()
    for a, b in zip(leaves, plain):
        # a product of 64, one of 90, four norms and two sums over 64: each STEPS roundings of what it adds, which the
        # largest gradients bound
        assert (a.grad.double() - b.grad).abs().max() <= 16 * ref.STEPS * ref.U * b.grad.abs().max() * width ** 0.5
    step.add_(1)

    # the trained model as the teacher of a student, by its lists; and its answers' scores in a beam step
    logits = logits.detach()
    top = rq.log_probs(logits, top=8, temperature=2.0)
    student = randn(g, rows, vocab).requires_grad_()
    rq.distill_loss(student, 2.0 * top.top_log_probs, top.top_codes, torch.zeros_like(top.lse), temperature=2.0).sum().backward()
    assert bool(torch.isfinite(student.grad).all()) and bool((student.grad != 0).any())
    best = rq.log_probs(logits, top=4)
    search = rq.BeamSearch(rows, 1, vocab, 4)
    scores, _, chosen, _ = search.select(logits.view(rows, 1, vocab), torch.zeros((rows, 1), device=DEV))
    assert torch.equal(chosen, best.top_codes)
    ref.check(scores, best.top_log_probs.double().cpu(), 64 * ref.U * best.top_log_probs.abs().double().cpu() + 64 * ref.U, "scores")
