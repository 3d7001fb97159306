"""Log probabilities of given codes on the GPU against the plain 64-bit
statement of them (sublayer_ref)."""

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
    rows, width = t.shape
    buffer = torch.full((rows * (width + pad) + shift + 16,), NAN, dtype=t.dtype, device=t.device)
    view = buffer.as_strided((rows, width), (width + pad, 1), shift)
    view.copy_(t)
    return view


def untouched(view):
    buffer = torch.empty(0, dtype=view.dtype, device=DEV).set_(view.untyped_storage())
    held = buffer.clone()
    held.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(NAN)
    return bool(torch.isnan(held).all())


def run(z, codes, temperature=1.0, top=0, grads=(None, None, None), entropy=True, d=None):
    rows = z.shape[0]
    f = lambda *shape: torch.full((rows,) + shape, NAN, device=DEV)  # noqa: E731
    out = {"log_probs": f(), "entropy": f() if entropy else None, "lse": f()}
    stats = f(2)
    if top:
        out["top_log_probs"], out["top_codes"] = f(top), torch.full((rows, top), -7, dtype=torch.int32, device=DEV)
    rq.rvq_log_probs(z, codes, temperature, out["log_probs"], out["entropy"], out["lse"], stats, out.get("top_log_probs"),
                     out.get("top_codes"))
    if any(g is not None for g in grads):
        out["dlogits"] = torch.full(z.shape, NAN, dtype=z.dtype, device=DEV) if d is None else d
        rq.rvq_log_probs_backward(*grads, z, codes, temperature, stats, out["entropy"], out["dlogits"])
    return out


def check(got, z, codes, temperature=1.0, top=0, grads=(None, None, None)):
    val, tol = ref.log_probs(z, codes, temperature, top, grads)
    for k, v in val.items():
        if got.get(k) is None:
            continue
        if k == "top_codes":
            assert torch.equal(got[k].cpu().long(), v), k
        else:
            ref.check(got[k], v, tol[k], k)


def make(rows, vocab, dtype, seed=0):
    g = gen(seed + rows * 7 + vocab)
    z = (randn(g, rows, vocab) * 2.5 + randn(g, rows, 1) * 10).to(dtype)
    codes = torch.randint(0, vocab, (rows,), generator=g, device=DEV).to(torch.int32)
    codes[1::5] = -1
    return z, codes, [randn(g, rows), randn(g, rows) * 0.1, randn(g, rows) * 0.1]


SIZES = [(1, 1), (3, 2), (5, 7), (9, 8), (4, 31), (6, 100), (300, 256), (33, 1000), (7, 1024), (50, 1025), (3, 1031),
         (2, 1040), (5, 1100), (4, 2048), (40, 4097), (200, 5000), (3, 16384), (2, 16401), (300, 20001), (1, 65536), (6, 65537),
         (40, 65536), (1, 131071), (1, 1 << 20)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_sizes(rows, vocab, dtype):
    z, codes, grads = make(rows, vocab, dtype)
    for temperature in (1.0, 0.7):
        check(run(z, codes, temperature, 0, grads), z, codes, temperature, 0, grads)
    only = [grads[0], None, grads[2]]
    check(run(z, codes, 1.3, 0, only, entropy=False), z, codes, 1.3, 0, only)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("top", [1, 3, 16, 33, 64])
def test_top(top, dtype):
    for rows, vocab in SIZES:
        if rows * vocab > 1 << 20:
            continue
        z, codes, _ = make(rows, vocab, dtype, top)
        check(run(z, codes, 1.0, top), z, codes, 1.0, top)
    z, codes, _ = make(3, 1 << 19, dtype)
    check(run(z, codes, 0.8, top), z, codes, 0.8, top)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (0, 1), (5, 7)])
def test_strides_and_alignment(pad, shift, dtype):
    for rows, vocab in ((1, 5), (37, 40), (9, 1024), (12, 1500), (5, 9000), (2, 70000)):
        z, codes, grads = make(rows, vocab, dtype)
        zv = rows_in(z, pad, shift)
        for d in (rows_in(z, pad, shift), rows_in(z, pad + 1, shift + 2), None):
            got = run(zv, codes, 1.0, 4 if vocab > 4 else 0, grads, d=d)
            check(got, z, codes, 1.0, 4 if vocab > 4 else 0, grads)
            assert d is None or untouched(d)
        # over the logits, row by row
        want = got["dlogits"]
        got = run(zv, codes, 1.0, 4 if vocab > 4 else 0, grads, d=zv)
        assert torch.equal(got["dlogits"], want) and untouched(zv)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [40, 1025, 3000, 70000])
def test_masks(vocab, dtype):
    """-inf, the type's lowest value and -1e9 in masked places, rows of nothing else, codes that are masked."""
    low = torch.finfo(dtype).min
    z, codes, grads = make(9, vocab, dtype)
    z[0, ::3] = -INF
    z[1, 1:] = -INF                       # one code left: no entropy
    z[2] = -INF                           # none
    z[3] = low                            # all alike
    z[4, 5:] = low
    z[5, ::2] = max(low, -1e9)
    z[6] = -INF
    z[6, vocab - 1] = low
    z[7] = 3.0
    for c in (0, vocab - 1):
        codes[:] = c
        got = run(z, codes, 1.0, 3, grads)
        check(got, z, codes, 1.0, 3, grads)
    assert got["entropy"][1].item() == 0.0 and got["entropy"][2].item() == 0.0
    assert got["top_codes"][2].tolist() == [-1, -1, -1] and got["top_codes"][1].tolist() == [0, -1, -1]
    assert got["top_codes"][7].tolist() == [0, 1, 2]
    assert abs(got["entropy"][3].item() - math.log(vocab)) < 1e-5
    assert bool((got["dlogits"][2] == 0).all())


@pytest.mark.parametrize("vocab", [40, 1025, 3000, 70000])
def test_nan_inf_and_rows_without_gradient(vocab):
    z, codes, grads = make(6, vocab, F32)
    clean = run(z, codes, 1.0, 3, grads)
    z[1, 7] = NAN
    z[2, 9] = INF
    z[4, 3] = NAN
    for g in grads:
        g[4] = 0.0
    got = run(z, codes, 1.0, 3, grads)
    codes[1] = codes[2] = 0
    nan = run(z, codes, 1.0, 3, grads)
    for k in ("log_probs", "entropy", "lse"):
        assert bool(torch.isnan(nan[k][[1, 2]]).all())
    assert bool(torch.isnan(got["dlogits"][[1, 2]]).all()) and bool((got["dlogits"][4] == 0).all())
    assert got["top_codes"][2, 0].item() == 9 and 7 not in got["top_codes"][1].tolist()
    for k in got:
        assert torch.equal(got[k][[0, 3, 5]], clean[k][[0, 3, 5]]), k


@pytest.mark.parametrize("vocab", [100, 3000, 20000])
def test_lowest_temperature(vocab):
    """All is on the largest logit: no entropy, and gradients of 0 where that is the code and elsewhere, however large a
    finite one the inverse of the temperature makes of those that are not."""
    z, codes, _ = make(5, vocab, F32)
    codes[:] = z.argmax(1).to(torch.int32)
    grads = [torch.full((5,), 1000.0, device=DEV), torch.full((5,), 2.0, device=DEV), None]
    got = run(z, codes, 4.3e-39, 2, [torch.full((5,), 0.5, device=DEV), grads[1], None])
    assert bool((got["log_probs"] == 0).all()) and bool((got["entropy"] == 0).all()) and bool((got["dlogits"] == 0).all())
    got = run(z, codes, 4.3e-39, 2, grads)          # 1000 / T is past float32
    others = got["dlogits"].scatter(1, codes.long()[:, None], 0.0)
    assert bool((others == 0).all())


def test_codes_out_of_range():
    z, codes, grads = make(6, 100, BF16)
    codes[:] = torch.tensor([-1, 100, -2, 99, 2 ** 31 - 1, 0], device=DEV)
    bad = torch.full((1,), 5, dtype=torch.int64, device=DEV)
    lp = torch.empty(6, device=DEV)
    rq.rvq_log_probs(z, codes, 1.0, lp, bad_codes=bad)
    assert bad.item() == 8 and lp[[0, 1, 2, 4]].tolist() == [0.0] * 4 and bool((lp[[3, 5]] < 0).all())
    check(run(z, codes, 1.0, 0, grads), z, codes, 1.0, 0, grads)


@pytest.mark.parametrize("vocab", [1025, 5000, 65536])
def test_ties_and_repeats(vocab):
    """Few different values: the lower code is first, and equal inputs give equal bits."""
    g = gen(vocab)
    z = (randn(g, 7, vocab) * 2).round().to(F16)
    z[3] = 0.0
    z[4] = -0.0
    z[4, ::2] = 0.0
    codes = torch.zeros(7, dtype=torch.int32, device=DEV)
    one = run(z, codes, 1.0, 64)
    check(one, z, codes, 1.0, 64)
    two = run(z, codes, 1.0, 64)
    for k in one:
        assert torch.equal(one[k], two[k]), k


def test_autograd_and_a_teacher_of_distillation():
    g = gen(3)
    z = (randn(g, 4, 5, 90) * 2).requires_grad_()
    codes = torch.randint(-1, 90, (4, 5), generator=g, device=DEV)          # 64 bits
    up = [randn(g, 4, 5) for _ in range(3)]
    out = rq.log_probs(z, codes, entropy=True, top=6, temperature=1.5)
    assert not out.top_log_probs.requires_grad and out.top_codes.shape == (4, 5, 6)
    torch.autograd.backward(out[:3], up)
    flat, c32 = z.detach().view(20, 90), codes.view(20).to(torch.int32)
    val, tol = ref.log_probs(flat, c32, 1.5, 6, [u.view(20) for u in up])
    for k in ("log_probs", "entropy", "lse", "top_log_probs"):
        t = getattr(out, k).detach()
        ref.check(t.view(val[k].shape), val[k], tol[k], k)
    ref.check(z.grad.view(20, 90), val["dlogits"], tol["dlogits"], "dlogits")
    # one of them alone
    z.grad = None
    rq.log_probs(z, codes).log_probs.sum().backward()
    val, tol = ref.log_probs(flat, c32, 1.0, 0, [torch.ones(20, device=DEV), None, None])
    ref.check(z.grad.view(20, 90), val["dlogits"], tol["dlogits"], "dlogits")
    assert rq.log_probs(z).log_probs is None
    # the lists, all codes of them, as a teacher: a student that is the teacher has no loss, and the loss is the divergence
    with torch.no_grad():
        top = rq.log_probs(z.view(20, 90)[:, :40].contiguous(), top=40, temperature=2.0)
        student = randn(g, 20, 40)
        loss = rq.distill_loss(student, 2.0 * top.top_log_probs, top.top_codes, torch.zeros_like(top.lse), temperature=2.0)
    q = torch.log_softmax(z.detach().view(20, 90)[:, :40].double() / 2, 1)
    p = torch.log_softmax(student.double() / 2, 1)
    want = (q.exp() * (q - p)).sum(1)
    # of both operators: terms q_j (log q_j - log p_j), each off by STEPS roundings of the logarithms' sizes, and the
    # mass beside the list, at most 2^-20 by its rounding, which counts as none
    ref.check(loss, want.cpu(), (2 * ref.STEPS * ref.U * (q.exp() * (1 + q.abs() + p.abs())).sum(1)).cpu(), "loss")


def test_gradient_against_differences():
    g = gen(8)
    z, dz = randn(g, 5, 60).double(), randn(g, 5, 60).double()
    codes = torch.tensor([0, 59, 7, -1, 30], dtype=torch.int32, device=DEV)
    up = [randn(g, 5) for _ in range(3)]

    def value(t):
        x = (z + t * dz) / 0.9
        lp = torch.log_softmax(x, 1)
        at = torch.where(codes >= 0, lp.gather(1, codes.clamp(min=0).long()[:, None])[:, 0], 0.0)
        return (at * up[0] - (lp.exp() * lp).sum(1) * up[1] + torch.logsumexp(x, 1) * up[2]).sum().item()

    step = 1e-5
    want = (value(step) - value(-step)) / (2 * step)
    zs = z.float().requires_grad_()
    out = rq.log_probs(zs, codes, entropy=True, temperature=0.9)
    torch.autograd.backward(out[:3], up)
    terms = zs.grad.double() * dz
    size = terms.abs().sum().item()
    # the inputs' and the gradient's roundings (some hundred of 2^-24), and the differences' own error of about step^2
    assert abs(terms.sum().item() - want) <= size * (256 * ref.U + 1e-8)


def test_other_streams_graphs_and_two_at_once():
    z, codes, grads = make(60, 3000, BF16)
    few, few_codes, _ = make(2, 70000, F32)
    want = run(z, codes, 1.0, 5, grads), run(few, few_codes, 1.0, 5)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append((run(z, codes, 1.0, 5, grads), run(few, few_codes, 1.0, 5)))
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            for k in b:
                assert torch.equal(a[k], b[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run(z, codes, 1.0, 5, grads), run(few, few_codes, 1.0, 5)
    z.copy_(z.flip(1))
    few.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(captured, (run(z, codes, 1.0, 5, grads), run(few, few_codes, 1.0, 5))):
        for k in b:
            assert torch.equal(a[k], b[k]), k


def test_no_rows_and_python_refusals():
    z = torch.zeros((0, 50), device=DEV)
    out = rq.log_probs(z, torch.zeros(0, dtype=torch.int64, device=DEV), True, 3)
    assert out.log_probs.shape == (0,) and out.top_codes.shape == (0, 3)
    z, codes, _ = make(4, 50, F32)
    with pytest.raises(ValueError):
        rq.log_probs(z, codes[:3])
    with pytest.raises(rq.RVQError):
        rq.log_probs(z, codes, top=65)
    with pytest.raises(rq.RVQError):
        rq.log_probs(z, codes, temperature=0.0)
    with pytest.raises(ValueError):
        rq.rvq_log_probs(z, codes.long(), 1.0, torch.empty(4, device=DEV))
    with pytest.raises(ValueError):
        rq.rvq_log_probs(z, codes, 1.0, torch.empty(3, device=DEV))
