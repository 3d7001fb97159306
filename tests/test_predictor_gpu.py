"""The code predictor's operators on the GPU against plain 64-bit statements of
them (predictor_ref): sizes, types, strides and masks where they can go wrong."""

import math

import pytest
import torch

import predictor_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import residual_vector_quantisation_gb300 as rq  # noqa: E402
from residual_vector_quantisation_gb300 import build as rqb  # noqa: E402

DEV = torch.device("cuda:0")
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
INF = math.inf


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


def rows_of(t, pad, shift):
    """The same rows, `pad` elements of NaN after each and the first `shift` elements into its buffer."""
    rows, width = t.shape
    buffer = torch.full((rows * (width + pad) + shift + 8,), math.nan, dtype=t.dtype, device=t.device)
    view = buffer[shift:shift + rows * (width + pad)].view(rows, width + pad)[:, :width]
    view.copy_(t)
    return view


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------

def run_norm(x, weight, bias, eps, dy, out=None, params=True, stream=None):
    rows, width = x.shape
    y = torch.empty((rows, width), dtype=x.dtype, device=DEV) if out is None else out[0]
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    rq.rvq_layer_norm(x, weight, bias, eps, y, mean, rstd, stream)
    dx = torch.empty((rows, width), dtype=x.dtype, device=DEV) if out is None else out[1]
    pd = F32 if weight is None else weight.dtype
    dw, db = (torch.full((width,), math.nan, dtype=pd, device=DEV) for _ in range(2)) if params else (None, None)
    ws = torch.empty(rq.rvq_layer_norm_workspace_bytes(rows, width), dtype=torch.uint8, device=DEV)
    rq.rvq_layer_norm_backward(dy, x, weight, mean, rstd, dx, dw, db, ws, stream)
    return {"y": y, "dx": dx, "dweight": dw, "dbias": db}


def check_norm(got, x, weight, bias, eps, dy):
    val, tol = ref.norm(x, weight, bias, eps, dy)
    for k in val:
        if got[k] is not None:
            ref.check(got[k], val[k], tol[k], k)


@pytest.mark.parametrize("dtype,pdtype", [(F32, F32), (BF16, F32), (BF16, BF16), (F16, F32), (F16, F16)])
@pytest.mark.parametrize("rows,width", [(1, 1), (1, 1024), (3, 7), (5, 33), (130, 256), (700, 768), (9, 1000),
                                        (33, 1024), (6, 1025), (17, 1032), (4, 2048), (3, 4097), (2, 8200),
                                        (5, 12288), (2, 16384)])
def test_norm_sizes(rows, width, dtype, pdtype):
    g = gen(rows * 31 + width)
    x = (randn(g, rows, width) + 0.5 * randn(g, rows, 1)).to(dtype)
    w, b = (1 + 0.2 * randn(g, width)).to(pdtype), (0.3 * randn(g, width)).to(pdtype)
    dy = randn(g, rows, width).to(dtype)
    check_norm(run_norm(x, w, b, 1e-5, dy), x, w, b, 1e-5, dy)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (5, 7)])
@pytest.mark.parametrize("width", [40, 1024, 1500])
def test_norm_strides_and_alignment(width, pad, shift, dtype):
    g = gen(width + pad)
    x, dy = randn(g, 37, width).to(dtype), randn(g, 37, width).to(dtype)
    w, b = 1 + 0.2 * randn(g, width), 0.3 * randn(g, width)
    xv, dyv = rows_of(x, pad, shift), rows_of(dy, pad, shift)
    out = [rows_of(torch.zeros_like(x), pad, shift) for _ in range(2)]
    check_norm(run_norm(xv, w, b, 1e-5, dyv, out), x, w, b, 1e-5, dy)
    # what lies between the rows is untouched
    for t in out:
        buffer = torch.empty(0, dtype=dtype, device=DEV).set_(t.untyped_storage())
        assert int(torch.isnan(buffer).sum()) == buffer.numel() - t.numel()


@pytest.mark.parametrize("width", [96, 1024, 3000])
def test_norm_without_parameters_and_in_place(width):
    g = gen(5)
    x, dy = randn(g, 41, width), randn(g, 41, width)
    val, tol = ref.norm(x, None, None, 1e-5, dy)
    got = run_norm(x, None, None, 1e-5, dy, params=False)
    for k in ("y", "dx"):
        ref.check(got[k], val[k], tol[k], k)
    y, mean, rstd = x.clone(), torch.empty(41, device=DEV), torch.empty(41, device=DEV)
    rq.rvq_layer_norm(y, None, None, 1e-5, y, mean, rstd)
    assert torch.equal(y, got["y"])
    for same in (0, 1):
        d, xx = dy.clone(), x.clone()
        rq.rvq_layer_norm_backward(d, xx, None, mean, rstd, (d, xx)[same], None, None, None)
        assert torch.equal((d, xx)[same], got["dx"])


def test_norm_constant_rows_large_means_and_nan():
    g = gen(6)
    x = randn(g, 6, 512)
    x[1] = 3.0                      # no variance: y is the bias
    x[2] += 4000.0                  # the mean cancels
    x[3] = 0.0
    x[4, 17] = math.nan
    x[5, 3] = INF
    w, b, dy = 1 + 0.1 * randn(g, 512), randn(g, 512), randn(g, 6, 512)
    got = run_norm(x, w, b, 1e-5, dy)
    val, tol = ref.norm(x[:4], w, b, 1e-5, dy[:4])
    for k in ("y", "dx"):
        ref.check(got[k][:4], val[k], tol[k], k)
        assert bool(torch.isnan(got[k][4:]).all())
    assert torch.equal(got["y"][1], b)


def test_norm_no_rows_and_parts():
    empty = torch.empty((0, 64), device=DEV)
    w = torch.ones(64, device=DEV)
    got = run_norm(empty, w, w, 1e-5, empty)
    assert bool((got["dweight"] == 0).all()) and bool((got["dbias"] == 0).all())
    # each gradient alone is the one that all together give
    g = gen(8)
    x, dy = randn(g, 333, 200), randn(g, 333, 200)
    w = 1 + 0.1 * randn(g, 200)
    every = run_norm(x, w, None, 1e-5, dy)
    mean, rstd = torch.empty(333, device=DEV), torch.empty(333, device=DEV)
    rq.rvq_layer_norm(x, w, None, 1e-5, torch.empty_like(x), mean, rstd)
    ws = torch.empty(rq.rvq_layer_norm_workspace_bytes(333, 200), dtype=torch.uint8, device=DEV)
    for k in ("dx", "dweight", "dbias"):
        out = {n: None for n in ("dx", "dweight", "dbias")}
        out[k] = torch.empty_like(every[k])
        rq.rvq_layer_norm_backward(dy, x, w, mean, rstd, out["dx"], out["dweight"], out["dbias"], ws)
        assert torch.equal(out[k], every[k]), k


@pytest.mark.parametrize("rows", [1, 3, 9, 150, 700])
@pytest.mark.parametrize("width,shift", [(64, 0), (200, 1), (1500, 0), (9000, 0), (9000, 1)])
def test_norm_stays_in_its_workspace(rows, width, shift):
    g = gen(rows)
    x, dy = (rows_of(randn(g, rows, width), 3, shift) for _ in range(2))
    w = 1 + 0.1 * randn(g, width)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    rq.rvq_layer_norm(x, w, None, 1e-5, torch.empty((rows, width), device=DEV), mean, rstd)
    need = rq.rvq_layer_norm_workspace_bytes(rows, width)
    buffer = torch.full((need + (1 << 22),), 0xA5, dtype=torch.uint8, device=DEV)
    dw, db = torch.empty_like(w), torch.empty_like(w)
    rq.rvq_layer_norm_backward(dy, x, w, mean, rstd, rows_of(torch.zeros((rows, width), device=DEV), 3, shift), dw, db,
                               buffer[:need])
    assert bool((buffer[need:] == 0xA5).all())
    val, tol = ref.norm(x, w, None, 1e-5, dy)
    ref.check(dw, val["dweight"], tol["dweight"], "dweight")
    ref.check(db, val["dbias"], tol["dbias"], "dbias")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("width", [1, 5, 8, 31, 48, 64, 96, 130, 248, 256, 257, 300, 352, 500, 512, 519])
def test_norm_narrow_rows_share_a_warp(width, dtype):
    """Row counts that leave a warp's last rows, and a block's, without work; rows that start inside a vector."""
    g = gen(width)
    w, b = 1 + 0.2 * randn(g, width), 0.3 * randn(g, width)
    for rows, pad, shift in ((1, 0, 0), (7, 0, 0), (153, 3, 1), (1219, 8, 0), (5003, 1, 2)):
        x, dy = randn(g, rows, width).to(dtype), randn(g, rows, width).to(dtype)
        xv, dyv = rows_of(x, pad, shift), rows_of(dy, pad, shift)
        out = [rows_of(torch.zeros_like(x), pad, shift) for _ in range(2)]
        check_norm(run_norm(xv, w, b, 1e-5, dyv, out), x, w, b, 1e-5, dy)
        for t in out:
            buffer = torch.empty(0, dtype=dtype, device=DEV).set_(t.untyped_storage())
            assert int(torch.isnan(buffer).sum()) == buffer.numel() - t.numel()


def test_norm_many_rows_and_repeats():
    g = gen(9)
    x, dy = randn(g, 20011, 192).to(BF16), randn(g, 20011, 192).to(BF16)
    w, b = 1 + 0.2 * randn(g, 192), 0.3 * randn(g, 192)
    one = run_norm(x, w, b, 1e-5, dy)
    check_norm(one, x, w, b, 1e-5, dy)
    two = run_norm(x, w, b, 1e-5, dy)
    for k in one:
        assert torch.equal(one[k], two[k]), k


@pytest.mark.parametrize("width,stride", [(640, 1 << 30), (1031, (1 << 30) + 1)])
def test_norm_offsets_past_32_bits(width, stride):
    g = gen(10)
    buffer = torch.zeros(4 * stride, dtype=F16, device=DEV)
    x = buffer.as_strided((4, width), (stride, 1))
    x.copy_(randn(g, 4, width))
    dy = randn(g, 4, width).to(F16)
    w = 1 + 0.1 * randn(g, width)
    plain = x.contiguous()
    got = run_norm(x, w, None, 1e-5, dy, [torch.empty_like(dy), x])   # dx over x
    check_norm(got, plain, w, None, 1e-5, dy)


def test_norm_differences_and_autograd():
    g = gen(11)
    x, w, b = randn(g, 8, 3, 160), 1 + 0.2 * randn(g, 160), 0.3 * randn(g, 160)
    dy = randn(g, 3, 8, 160).transpose(0, 1)          # a gradient in another order
    leaf = [t.clone().requires_grad_() for t in (x, w, b)]
    rq.layer_norm(*leaf).backward(dy)
    # central differences of sum(y * dy) in 64 bits; what a step of 1e-3 leaves out is below 1e-6 of its size
    for k, t in enumerate((x, w, b)):
        d = randn(g, *t.shape)
        total = []
        for side in (1, -1):
            a = [v.double() for v in (x, w, b)]
            a[k] = a[k] + side * 1e-3 * d.double()
            val, _ = ref.norm(a[0].reshape(24, 160), a[1], a[2], 1e-5)
            total.append((val["y"].reshape(8, 3, 160) * dy.double()).sum())
        want = (total[0] - total[1]).item() / 2e-3
        got = (leaf[k].grad.double() * d.double()).sum().item()
        scale = (leaf[k].grad.double() * d.double()).abs().sum().item()
        assert abs(got - want) <= 2e-5 * scale, (k, got, want)


# ---------------------------------------------------------------------------
# distillation
# ---------------------------------------------------------------------------

def make_distill(seed, rows, vocab, top, dtype, tail, temperature=1.0, top_dtype=F32):
    g = gen(seed)
    z = (randn(g, rows, vocab) * 2.5).to(dtype)
    teacher = 0.7 * z.float() + 2.0 * randn(g, rows, vocab)
    t, codes = torch.topk(teacher, min(top, vocab), dim=1)
    if top > vocab:
        t = torch.cat([t, t.new_zeros((rows, top - vocab))], 1)
        codes = torch.cat([codes, codes.new_full((rows, top - vocab), -1)], 1)
    lse = torch.logsumexp(teacher.double() / temperature, 1).float() if tail else None
    weights = torch.rand(rows, generator=g, device=DEV) + 0.5
    return z, t.to(top_dtype), codes.to(torch.int32), lse, weights


def run_distill(z, t, codes, lse, weights, temperature, grad_loss=None, out=None, bad=None):
    """Fused, and as two passes; both have to be right."""
    rows = z.shape[0]
    loss = torch.full((rows,), math.nan, device=DEV)
    d = torch.full(z.shape, math.nan, dtype=z.dtype, device=DEV) if out is None else out
    rq.rvq_distill(z, t, codes, lse, weights, temperature, loss, dlogits=d, bad_codes=bad)
    loss2, stats, d2 = torch.empty_like(loss), torch.empty((rows, 2), device=DEV), torch.empty(z.shape, dtype=z.dtype,
                                                                                                device=DEV)
    rq.rvq_distill(z, t, codes, lse, weights, temperature, loss2, lse=stats)
    rq.rvq_distill_backward(grad_loss, z, t, codes, lse, weights, temperature, stats, d2)
    return {"loss": loss, "dlogits": d}, {"loss": loss2, "dlogits": d2}


def check_distill(z, t, codes, lse, weights, temperature=1.0, grad_loss=None, out=None):
    bad = torch.zeros(1, dtype=torch.int64, device=DEV)
    plain = z.clone()
    fused, split = run_distill(z, t, codes, lse, weights, temperature, grad_loss, out, bad)
    val, tol, n_bad = ref.distill(plain, t, codes, lse, weights, temperature)
    for k in val:
        ref.check(fused[k], val[k], tol[k], "fused " + k)
    if grad_loss is not None:
        val, tol, _ = ref.distill(plain, t, codes, lse, weights, temperature, grad_loss)
        ref.check(split["dlogits"], val["dlogits"], tol["dlogits"], "split dlogits")
    else:
        for k in val:
            ref.check(split[k], val[k], tol[k], "split " + k)
    assert rq.rvq_read_error_count(bad) == n_bad
    return val


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (1, 2, 5), (3, 31, 4), (5, 64, 64), (7, 130, 33), (40, 1024, 16),
                                            (33, 1025, 32), (9, 1281, 50), (3, 4100, 64), (2, 5121, 256),
                                            (2, 20481, 8), (2, 32768, 64), (1, 70001, 100), (2, 131072, 40)])
def test_distill_sizes(rows, vocab, top, tail, dtype):
    check_distill(*make_distill(rows + vocab, rows, vocab, top, dtype, tail))


@pytest.mark.parametrize("temperature", [0.25, 3.0])
@pytest.mark.parametrize("top_dtype", [F32, BF16, F16])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_temperature_types_and_upstream(tail, top_dtype, temperature):
    a = make_distill(3, 21, 1025, 20, BF16, tail, temperature, top_dtype)
    grad = torch.randn(21, device=DEV)
    check_distill(*a, temperature, grad)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad,shift,vocab", [(7, 0, 1025), (8, 0, 1024), (1, 3, 200), (3, 1, 6000), (5, 2, 40000)])
def test_distill_strides_alignment_and_in_place(pad, shift, vocab, dtype):
    z, t, codes, lse, w = make_distill(pad, 6, vocab, 9, dtype, True)
    zv = rows_of(z, pad, shift)
    check_distill(zv, t, codes, lse, w, out=rows_of(torch.zeros_like(z), pad, shift))
    other = rows_of(torch.zeros_like(z), pad + 1, shift + 1)          # rows that start elsewhere than the logits'
    check_distill(zv, t, codes, lse, w, out=other)
    buffer = torch.empty(0, dtype=dtype, device=DEV).set_(other.untyped_storage())
    assert int(torch.isnan(buffer).sum()) == buffer.numel() - z.numel()
    loss = torch.empty(6, device=DEV)
    want = torch.empty_like(zv)
    rq.rvq_distill(zv, t, codes, lse, w, 1.0, loss, dlogits=want)
    rq.rvq_distill(zv, t, codes, lse, w, 1.0, loss, dlogits=zv)
    assert torch.equal(zv, want)


@pytest.mark.parametrize("vocab", [64, 1025, 6000, 30000, 100000])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_masks(tail, vocab):
    z, t, codes, lse, w = make_distill(17, 12, vocab, 8, F32, tail)
    low = torch.finfo(F32).min
    z[0, vocab // 2:] = -INF                       # masked codes
    z[1, vocab // 2:] = low
    w[2] = 0.0
    z[2, 5] = math.nan                             # a row without weight: nothing in it matters
    t[2, 0] = INF
    codes[3] = -1                                  # no entries
    z[3, 1] = math.nan
    t[4] = -INF                                    # entries without a share
    t[5, 3:] = -INF
    codes[6, 4:] = -1                              # a list that ends early
    z[7, int(codes[7, 0])] = -INF                  # the student gives the teacher's best code nothing
    z[8] = -INF                                    # the mask leaves nothing
    z[9] = low
    codes[10, 2] = codes[10, 0]                    # a code twice
    codes[10, 3] = vocab                           # not a code
    codes[10, 4] = -7
    keep = torch.zeros(vocab, dtype=torch.bool, device=DEV)
    keep[codes[11].long()] = True
    z[11, ~keep] = -INF                            # nothing off the list
    val = check_distill(z, t, codes, lse, w)
    assert val["loss"][7] == INF and val["loss"][2] == 0 and val["loss"][3] == 0


@pytest.mark.parametrize("tail", [False, True])
def test_distill_nan_stays_in_its_row(tail):
    z, t, codes, lse, w = make_distill(23, 6, 1500, 8, F32, tail)
    z[1, 700] = math.nan
    z[3, 20] = INF
    t[4, 2] = math.nan
    loss, d = torch.empty(6, device=DEV), torch.empty_like(z)
    rq.rvq_distill(z, t, codes, lse, w, 1.0, loss, dlogits=d)
    assert torch.isnan(loss).tolist() == [False, True, False, True, True, False]
    assert bool(torch.isnan(d[1]).all()) and bool(torch.isnan(d[3]).all())
    for r in (0, 2, 5):
        assert bool(torch.isfinite(d[r]).all())


def test_distill_list_with_nearly_everything():
    """p off the list is 1e-12 of the row: the tail's gradient keeps its digits."""
    z, t, codes, lse, w = make_distill(29, 4, 1025, 16, F32, True)
    z -= 0.5 * z.amax(1, keepdim=True)
    z.scatter_add_(1, codes.long(), torch.full((4, 16), 30.0, device=DEV))
    check_distill(z, t, codes, lse, w)


def test_distill_codes_past_32_bits_are_not_codes():
    z, t, codes, lse, w = make_distill(33, 4, 300, 6, F32, False)
    wide = codes.long()
    wide[:, 2] += 1 << 32
    bad = codes.clone()
    bad[:, 2] = -7
    want = torch.empty(4, device=DEV)
    rq.rvq_distill(z, t, bad, None, w, 1.0, want)
    assert torch.equal(rq.distill_loss(z, t, wide, None, w), want)


def test_distill_no_rows_weights_and_repeats():
    z, t, codes, lse, _ = make_distill(31, 0, 100, 4, F32, True)
    run_distill(z, t, codes, lse, None, 1.0)
    a = make_distill(37, 3000, 1025, 32, BF16, True)
    one, _ = run_distill(*a, 2.0)
    two, _ = run_distill(*a, 2.0)
    assert torch.equal(one["loss"], two["loss"]) and torch.equal(one["dlogits"], two["dlogits"])
    check_distill(*make_distill(41, 5, 300, 4, F32, False)[:4], None)


def test_distill_offsets_past_32_bits():
    vocab, rows = 1025, 5
    stride = (1 << 30) + 3
    z, t, codes, lse, w = make_distill(43, rows, vocab, 12, F16, True)
    buffer = torch.zeros((rows - 1) * stride + vocab, dtype=F16, device=DEV)
    zv = buffer.as_strided((rows, vocab), (stride, 1))
    zv.copy_(z)
    loss, d = torch.empty(rows, device=DEV), torch.empty_like(z)
    rq.rvq_distill(zv, t, codes, lse, w, 1.0, loss, dlogits=d)
    rq.rvq_distill(zv, t, codes, lse, w, 1.0, loss, dlogits=zv)
    val, tol, _ = ref.distill(z, t, codes, lse, w, 1.0)
    ref.check(loss, val["loss"], tol["loss"], "loss")
    ref.check(d, val["dlogits"], tol["dlogits"], "dlogits")
    assert torch.equal(zv, d)


@pytest.mark.parametrize("tail", [False, True])
def test_distill_differences_and_autograd(tail):
    temperature = 1.5
    z, t, codes, lse, w = make_distill(47, 10, 257, 12, F32, tail, temperature)
    shape = (2, 5)
    leaf = z.view(*shape, 257).clone().requires_grad_()
    args = (t.view(*shape, 12), codes.view(*shape, 12).long(), None if lse is None else lse.view(shape))
    loss = rq.distill_loss(leaf, *args, w.view(shape), temperature)
    loss.sum().backward()                          # an upstream gradient that is one broadcast value
    both = rq.distill_loss_and_grad(leaf.detach(), *args, w.view(shape), temperature)
    assert torch.equal(both[0], loss.detach())
    assert torch.allclose(both[1], leaf.grad, rtol=1e-5, atol=1e-7)
    # central differences of the loss in 64 bits: a step of 1e-3 leaves out less than 1e-6 of each row
    g = gen(2)
    d = randn(g, 10, 257)
    side = [ref.distill(z.double() + s * 1e-3 * d.double(), t, codes, lse, w, temperature)[0]["loss"] for s in (1, -1)]
    want = (side[0] - side[1]) / 2e-3
    got = (leaf.grad.view(10, 257).double() * d.double()).sum(1).cpu()
    scale = (leaf.grad.view(10, 257).double() * d.double()).abs().sum(1).cpu()
    assert bool(((got - want).abs() <= 2e-5 * scale + 1e-6).all())


# ---------------------------------------------------------------------------
# the beam step
# ---------------------------------------------------------------------------

def run_beam(logits, scores, finished, end_code, select, raw=False, stream=None):
    groups, beams, vocab = logits.shape
    search = rq.BeamSearch(groups, beams, vocab, select, "raw" if raw else "logits", logits.dtype,
                           None if end_code < 0 else end_code)
    return search, search.select(logits, scores, finished, stream)


def check_beam(logits, scores, finished, end_code, select, raw=False):
    search, (out, parents, codes, done) = run_beam(logits, scores, finished, end_code, select, raw)
    want = ref.beam(logits, scores, finished, end_code, select, raw)
    assert torch.equal(parents.cpu().long(), want[1]), (parents, want[1])
    assert torch.equal(codes.cpu().long(), want[2])
    if done is not None:
        assert torch.equal(done.cpu(), want[3])
    live = torch.isfinite(logits.float())
    size = torch.where(live, logits.float(), 0.0).abs().clamp(max=1e4).max().item() + math.log(logits.shape[2])
    bound = torch.where(torch.isfinite(want[0]), want[0].abs() + size, torch.zeros_like(want[0]))
    ref.check(out, want[0], 0.0 if raw else 16 * ref.U * bound, "scores")
    return out, parents, codes


def make_beam(seed, groups, beams, vocab, dtype):
    """Logits on a grid of 1/16 and scores on one of 1/8 plus a beam's own offset: totals of different beams are
    at least 1e-4 apart unless chance brings two sums of the rows' exponentials that near (checked by the caller's
    comparison, with seeds fixed here)."""
    g = gen(seed)
    logits = ((randn(g, groups, beams, vocab) * 48).round() / 16).to(dtype)
    scores = -(randn(g, groups, beams) * 24).round().abs() / 8
    return logits, scores


BEAM_SIZES = [(1, 1, 1, 1), (1, 1, 2, 4), (2, 3, 5, 15), (1, 4, 1025, 4), (5, 4, 1024, 8), (3, 8, 4096, 16),
              (2, 5, 4099, 1), (1, 2, 20000, 64), (40, 2, 300, 3), (1, 64, 257, 64), (1, 1, 70000, 32),
              (2, 3, 65536, 6)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("groups,beams,vocab,select", BEAM_SIZES)
def test_beam_sizes(groups, beams, vocab, select, dtype):
    logits, scores = make_beam(groups + beams + vocab, groups, beams, vocab, dtype)
    check_beam(logits, scores, None, -1, select)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("groups,beams,vocab,select", BEAM_SIZES)
def test_beam_raw_with_ties(groups, beams, vocab, select, dtype):
    logits, scores = make_beam(groups * beams + vocab, groups, beams, vocab, dtype)
    check_beam((logits * 0.25).round(), scores, None, -1, select, raw=True)     # many equal totals
    check_beam(torch.zeros_like(logits), torch.zeros_like(scores), None, -1, select, raw=True)
    check_beam(-torch.zeros_like(logits), torch.zeros_like(scores), None, -1, select, raw=True)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("vocab", [37, 1025, 9000])
def test_beam_masks_and_finished(vocab, raw):
    logits, scores = make_beam(vocab, 9, 4, vocab, F32)
    low = torch.finfo(F32).min
    finished = torch.zeros((9, 4), dtype=torch.bool, device=DEV)
    finished[0, 1] = True
    finished[1] = True                             # every beam done
    scores[2] = -INF                               # no beam left
    scores[3, 1:] = -INF                           # the first step
    logits[3, 1:] = math.nan                       # rows that nothing reads
    logits[4, 0] = -INF                            # a beam whose mask leaves nothing
    logits[4, 1, 3:] = -INF
    logits[4, 2:] = -INF                           # three candidates in all
    logits[5, :, 2:] = low                         # the type's lowest value in masked places
    logits[6, 1, 7] = math.nan
    logits[7, 2] = math.nan
    scores[8, 0] = math.nan
    finished[8, 3] = True
    if not raw:
        logits[6, 1] = -INF                        # a NaN takes its whole row: stated by the row's absence
    check_beam(logits, scores, finished, vocab - 1, 6, raw)
    if not raw:
        logits[6, 1, 7] = math.nan
        _, (out, parents, codes, _) = run_beam(logits, scores, finished, vocab - 1, 6)
        assert not bool((parents[6] == 1).any()) and not bool(torch.isnan(out).any())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("order", ["rising", "falling", "last", "first"])
def test_beam_orders(order, dtype):
    """Rows in which every step brings a better entry, or none does, or the best ones stand together."""
    vocab = 30000
    ramp = torch.arange(vocab, device=DEV, dtype=F32)
    row = {"rising": ramp, "falling": -ramp, "last": (ramp > vocab - 50) * ramp, "first": (ramp < 50) * (50 - ramp)}
    logits = (row[order] / 64).to(dtype).expand(1, 2, vocab).contiguous()
    scores = torch.tensor([[-0.25, 0.0]], device=DEV)
    check_beam(logits, scores, None, -1, 64, raw=True)
    check_beam(logits, scores, None, -1, 5, raw=True)


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("pad,shift", [(7, 0), (0, 3), (8, 8)])
def test_beam_strides(pad, shift, dtype):
    logits, scores = make_beam(3, 3, 4, 1025, dtype)
    want = check_beam(logits, scores, None, -1, 8)
    rows = rows_of(logits.view(12, 1025), pad, shift)
    for view in (rows, rows.as_strided((3, 4, 1025), (4 * rows.stride(0), rows.stride(0), 1))):
        search = rq.BeamSearch(3, 4, 1025, 8, dtype=dtype)
        got = search.select(view, scores)
        for a, b in zip(got[1:3], want[1:]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("groups,beams,vocab,select", [(3, 4, 1025, 4), (2, 8, 4096, 8), (1, 4, 70000, 4),
                                                       (5, 12, 9000, 12), (1, 64, 40000, 64)])
def test_beam_workspace_and_outputs_over_inputs(groups, beams, vocab, select):
    logits, scores = make_beam(vocab, groups, beams, vocab, F32)
    finished = torch.zeros((groups, beams), dtype=torch.bool, device=DEV)
    finished[0, 1] = True
    search = rq.BeamSearch(groups, beams, vocab, select, end_code=3)
    want = search.select(logits, scores, finished)
    need = search.workspace.numel()
    buffer = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device=DEV)
    parents, codes = (torch.empty((groups, select), dtype=torch.int32, device=DEV) for _ in range(2))
    held, done = scores.clone(), finished.clone()
    rq.rvq_beam_select(search.dims, logits, held, done, 3, held, parents, codes, done, buffer[:need])
    for a, b in zip((held, parents, codes, done), want):
        assert torch.equal(a, b)
    assert bool((buffer[need:] == 0xA5).all())


def test_beam_offsets_past_32_bits():
    stride = (1 << 30) + 5
    logits, scores = make_beam(4, 1, 5, 1025, F16)
    buffer = torch.zeros(4 * stride + 1025, dtype=F16, device=DEV)
    view = buffer.as_strided((5, 1025), (stride, 1))
    view.copy_(logits[0])
    want = check_beam(logits, scores, None, -1, 10)
    got = rq.BeamSearch(1, 5, 1025, 10, dtype=F16).select(view, scores)
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


def reordered(state, parents, layered):
    s = state if layered else state[None]
    groups = torch.arange(s.shape[1], device=s.device)[:, None]
    p = parents.long()
    there = (p >= 0) & (p < s.shape[2])
    out = s[:, groups, torch.where(there, p, 0)]
    out = torch.where(there.view(1, *p.shape, *[1] * (s.dim() - 3)), out, torch.zeros_like(out))
    return out if layered else out[0]


@pytest.mark.parametrize("dtype,row", [(F32, (1024,)), (BF16, (25, 64)), (torch.int32, (7,)), (torch.uint8, (13,)),
                                       (F16, (3, 5)), (torch.int64, (1,)), (F32, (100, 1000))])
@pytest.mark.parametrize("layered", [False, True])
def test_reorder(layered, dtype, row):
    g = gen(1)
    groups, beams, select = 5, 4, 6
    shape = ((3,) if layered else ()) + (groups, beams) + row
    state = torch.randint(0, 100, shape, generator=g, device=DEV).to(dtype)
    parents = torch.randint(0, beams, (groups, select), generator=g, device=DEV, dtype=torch.int32)
    parents[1, 2], parents[3, 0] = -1, beams
    search = rq.BeamSearch(groups, beams, 100, select)
    assert torch.equal(search.reorder(parents, state, layered=layered), reordered(state, parents, layered))
    # in place, and a slice of a longer cache
    square = rq.BeamSearch(groups, beams, 100)
    parents = parents[:, :beams].contiguous()
    parents[0] = torch.arange(beams)               # nothing moves
    parents[2] = torch.tensor([1, 0, 3, 2])        # everything moves
    held = state.clone()
    square.reorder(parents, held, held, layered)
    assert torch.equal(held, reordered(state, parents, layered))
    if len(row) > 1:
        part = state[..., :row[0] - 1, :]
        held = state.clone()
        square.reorder(parents, held[..., :row[0] - 1, :], held[..., :row[0] - 1, :], layered)
        assert torch.equal(held[..., :row[0] - 1, :], reordered(part, parents, layered))
        assert torch.equal(held[..., row[0] - 1:, :], state[..., row[0] - 1:, :])


def test_reorder_several_states_at_once():
    g = gen(2)
    a, b = randn(g, 6, 3, 50), randn(g, 6, 3, 4, 8).to(BF16)
    parents = torch.randint(0, 3, (6, 3), generator=g, device=DEV, dtype=torch.int32)
    out = torch.empty_like(a)
    held = b.clone()
    states = rq.rvq_beam_states([(a, out), (held, held)])
    rq.rvq_beam_reorder(rq.rvq_beam_dims(6, 3, 10, 3, rq.RVQ_BEAM_RAW, 0), parents, states)
    assert torch.equal(out, reordered(a, parents, False)) and torch.equal(held, reordered(b, parents, False))


def test_reorder_offsets_past_32_bits():
    state = torch.zeros((1, 3, (1 << 31) + 16), dtype=torch.uint8, device=DEV)
    state[0, :, -5:] = torch.arange(15, device=DEV, dtype=torch.uint8).view(3, 5) + 1
    want = state[0, :, -16:].clone()
    search = rq.BeamSearch(1, 3, 10)
    parents = torch.tensor([[2, 0, 1]], device=DEV, dtype=torch.int32)
    out = search.reorder(parents, state)
    assert torch.equal(out[0, :, -16:], want[[2, 0, 1]])
    search.reorder(parents, state, state)
    assert torch.equal(state[0, :, -16:], want[[2, 0, 1]])


# ---------------------------------------------------------------------------
# streams, graphs, refusals
# ---------------------------------------------------------------------------

def test_other_streams_and_graphs():
    """On a stream of their own behind work that is still running, and replayed from a graph on new inputs."""
    g = gen(12)
    x, dy, w = randn(g, 4000, 512), randn(g, 4000, 512), 1 + 0.1 * randn(g, 512)
    z, t, codes, lse, weights = make_distill(53, 500, 1025, 16, F32, True)
    logits, scores = make_beam(6, 4, 4, 1025, F32)
    state = randn(g, 4, 4, 256)
    search = rq.BeamSearch(4, 4, 1025)

    def everything():
        n = run_norm(x, w, w, 1e-5, dy)
        loss, d = torch.empty(500, device=DEV), torch.empty_like(z)
        rq.rvq_distill(z, t, codes, lse, weights, 1.0, loss, dlogits=d)
        out, parents, chosen, _ = search.select(logits, scores)
        return [*n.values(), loss, d, out, parents, chosen, search.reorder(parents, state)]

    want = [v.clone() for v in everything()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device=DEV)
        held = x.clone()
        x.zero_()
        for _ in range(20):
            big = big @ big * 1e-3
        x.copy_(held)                              # the inputs are ready on this stream only
        got = everything()
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = everything()
    x.mul_(0.5)
    logits.copy_(logits.flip(2))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(captured, everything()):
        assert torch.equal(a, b)


def test_python_refusals():
    x = torch.zeros((4, 64), device=DEV)
    w = torch.ones(64, device=DEV)
    with pytest.raises(ValueError):
        rq.rvq_layer_norm(x, w, None, 1e-5, torch.zeros((4, 63), device=DEV))
    with pytest.raises(ValueError):
        rq.rvq_layer_norm(x, w[:32], None, 1e-5, torch.zeros_like(x))
    with pytest.raises(ValueError):
        rq.rvq_layer_norm(x.t(), w[:4], None, 1e-5, torch.zeros((64, 4), device=DEV))
    with pytest.raises(rq.RVQError):
        rq.rvq_layer_norm(x.to(BF16), w.to(F16), None, 1e-5, x.to(BF16))
    with pytest.raises(rq.RVQError):
        rq.rvq_layer_norm(x, w, None, -1.0, torch.zeros_like(x))
    z, t, codes, lse, weights = make_distill(1, 4, 64, 3, F32, True)
    loss = torch.zeros(4, device=DEV)
    with pytest.raises(ValueError):
        rq.rvq_distill(z, t, codes.long(), lse, weights, 1.0, loss)
    with pytest.raises(ValueError):
        rq.rvq_distill(z, t[:, :2], codes, lse, weights, 1.0, loss)
    with pytest.raises(rq.RVQError):
        rq.rvq_distill(z, t, codes, lse, weights, 0.0, loss)
    with pytest.raises(ValueError):
        rq.distill_loss(z.view(2, 2, 64), t, codes)
    with pytest.raises(ValueError):
        rq.BeamSearch(2, 65, 100)
    search = rq.BeamSearch(2, 3, 100)
    with pytest.raises(ValueError):
        search.select(torch.zeros((2, 3, 99), device=DEV), search.first_scores())
    with pytest.raises(ValueError):
        search.select(torch.zeros((2, 3, 100), dtype=BF16, device=DEV), search.first_scores())
    with pytest.raises(ValueError):
        search.reorder(torch.zeros((2, 3), dtype=torch.int32, device=DEV), torch.zeros((2, 4, 8), device=DEV))
