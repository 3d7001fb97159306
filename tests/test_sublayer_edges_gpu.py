"""The sublayer's operators, log probabilities and the beam step on the GPU where calls can go wrong."""

import math

import pytest
import torch

import predictor_ref
import sublayer_ref as ref
from test_sublayer_gpu import BF16, DEV, F32, INF, MASK, NAN, TYPES, gen, library, mask_of, randn, rows_in, untouched  # noqa: F401

import residual_vector_quantisation_gb300 as rq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mask", [None, MASK])
@pytest.mark.parametrize("block", [0, 32, 128])
@pytest.mark.parametrize("dtype", TYPES)
def test_the_sum_beside_8_bits(dtype, block, mask):
    """Bit for bit the sum's definition, nothing written beside its rows, and the same 8 bits as without it."""
    for rows, width, pad, shift in ((1, 1, 0, 0), (3, 31, 0, 0), (5, 64, 8, 0), (700, 200, 0, 0), (9, 768, 16, 0), (5, 1025, 6, 0),
                                    (7, 1100, 3, 5), (4, 520, 2, 1), (3, 5000, 0, 0), (2, 5003, 1, 3), (2, 16384, 0, 0),
                                    (2, 16383, 1, 0), (1200, 40, 1, 1)):
        g = gen(rows + width)
        x, r = (randn(g, rows, width).to(dtype) for _ in range(2))
        w = 1 + 0.2 * randn(g, width)
        for place in (lambda t: rows_in(t, pad, shift), lambda t: rows_in(t, pad + 1, shift + 1)):  # alike, and not
            total = place(torch.zeros_like(x))
            got = []
            for out in (total, None):
                q = torch.empty((rows, width), dtype=torch.float8_e4m3fn, device=DEV)
                s = torch.empty((rows, -(-width // block) if block else 1), dtype=F32, device=DEV)
                rq.rvq_rms_norm(rows_in(x, pad, shift), w, 1e-6, None, None, rows_in(r, pad, shift), mask_of(mask), out, q, s, block)
                got.append((q.view(torch.uint8), s))
            assert torch.equal(total, ref.total_of(x, mask, r)) and untouched(total), (rows, width)
            # another layout adds a row's squares in another order: a scale may be another float
            val, tol = ref.rms(ref.total_of(x, mask, r), w, 1e-6)
            for q, s in got:
                ref.check_8bit(q.view(torch.float8_e4m3fn), s, val["y"], tol["y"], block, False)


def test_squares_are_added_up_in_32_bits():
    """Rows whose squares add up past 3.4e38 have rstd 0 and a result of zero; those just below are normalised."""
    for width, size in ((100, 1.8e18), (1024, 5.7e17), (5000, 2.6e17), (16384, 1.4e17)):
        assert width * size ** 2 < 3.4e38 < width * (1.1 * size) ** 2
        x = torch.full((2, width), size, device=DEV)
        x[1] *= 1.1
        y, rstd = torch.empty_like(x), torch.empty(2, device=DEV)
        rq.rvq_rms_norm(x, None, 1e-6, y, rstd)
        assert rstd[1].item() == 0.0 and bool((y[1] == 0).all())
        val, tol = ref.rms(x[:1], None, 1e-6)
        ref.check(y[:1], val["y"], tol["y"], width)


def leaves(*tensors):
    return [t.clone().requires_grad_() for t in tensors]


@pytest.mark.parametrize("mask", [None, MASK])
def test_two_backward_passes_into_the_same_leaves(mask):
    g = gen(41)
    x, r, up, ut = (randn(g, 7, 96) for _ in range(4))
    x, r = leaves(x, r)
    for k in (1, 2):
        torch.autograd.backward(rq.rms_norm(x, None, 1e-6, r, mask_of(mask)), (up, ut))
        if k == 1:
            first = x.grad.clone(), r.grad.clone()
    assert x.grad.data_ptr() != r.grad.data_ptr()
    assert torch.equal(x.grad, 2 * first[0]) and torch.equal(r.grad, 2 * first[1])


@pytest.mark.parametrize("mask", [None, MASK])
def test_the_sum_alone_rows_without_a_norm(mask):
    g = gen(42)
    x, r, ut = (randn(g, 6, 40) for _ in range(3))
    x[0] = r[0] = 0.0
    x[1, 3], r[2, 4] = NAN, INF
    x, r = leaves(x, r)
    y, total = rq.rms_norm(x, None, 0.0, r, mask_of(mask))
    total.backward(ut)
    want = ut
    if mask is not None:
        keep, factor = ref.stays(ut.numel(), *mask)
        want = torch.where(torch.from_numpy(keep).view(ut.shape).to(DEV), ut * torch.tensor(factor, dtype=F32, device=DEV), 0.0)
    assert torch.equal(r.grad, ut) and torch.equal(x.grad, want)


def test_masks_changed_between_the_passes_and_results_in_place():
    g = gen(43)
    x, r, up = (randn(g, 5, 64) for _ in range(3))
    a, b = leaves(x, r)
    mask = mask_of(MASK)
    out = rq.dropout(a, mask, b), rq.rms_norm(a, None, 1e-6, b, mask)[0]
    mask.p, mask.seed, mask.offset = 0.9, 1, 1
    torch.autograd.backward([out[0].mul_(2.0), out[1].mul_(2.0)], (up, up))
    c, d = leaves(x, r)
    mask = mask_of(MASK)
    torch.autograd.backward([2.0 * rq.dropout(c, mask, d), 2.0 * rq.rms_norm(c, None, 1e-6, d, mask)[0]], (up, up))
    assert torch.equal(a.grad, c.grad) and torch.equal(b.grad, d.grad)


@pytest.mark.parametrize("dtype", TYPES)
def test_dropout_without_a_mask(dtype):
    g = gen(44)
    for shape in ((3, 5), (2, 7, 64), (41,)):
        x, r = (randn(g, *shape).to(dtype) for _ in range(2))
        y = rq.dropout(x, None)
        assert torch.equal(y, x) and y.data_ptr() != x.data_ptr()
        assert torch.equal(rq.dropout(x, None, r), (x.float() + r.float()).to(dtype))


@pytest.mark.parametrize("vocab", [40, 1025, 5000, 70000])
def test_confident_rows(vocab):
    """One code far above the others.  The sum of the exponentials holds its 1, so that log p, entropy and lse are right
    to the roundings of numbers near 1, not to their own size: at most STEPS additions on a path, each rounded by U."""
    others = [2.0 ** -k for k in (8, 14, 20, 23, 24, 25, 26, 30, 40, 60, 100)]       # all of them together
    d = torch.tensor([math.log(m / (vocab - 1)) for m in others], dtype=F32, device=DEV)
    z = d[:, None].expand(-1, vocab).contiguous()
    at = vocab // 3
    z[:, at] = 0.0
    codes = torch.full((len(others),), at, dtype=torch.int32, device=DEV)
    out = rq.log_probs(z, codes, entropy=True)
    lp = torch.log_softmax(z.double(), 1)
    entropy = -(lp.exp() * lp).sum(1)
    assert bool((out.log_probs <= 0).all()) and bool((out.entropy >= 0).all()) and bool((out.lse >= 0).all())
    off = ref.STEPS * ref.U
    assert bool(((out.log_probs.double() - lp[:, at]).abs() <= off).all())
    assert bool(((out.lse.double() - torch.logsumexp(z.double(), 1)).abs() <= off).all())
    # the second term of the entropy, sum p d, is relative: its terms carry the exponentials' errors (4 roundings of d, and
    # 2 units of the exponential) and the sum's
    rel = (ref.STEPS + 8 + 4 * d.abs().double()) * ref.U
    assert bool(((out.entropy.double() - entropy).abs() <= off + rel * entropy).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("groups,beams,vocab", [(3, 3, 300), (2, 2, 1025), (3, 8, 4096), (1, 2, 70000)])
def test_beam_step_and_alternatives_around_the_rules_of_the_bar(groups, beams, vocab, dtype):
    """Counts kept on both sides of where the bar comes from other parts of a lane's elements."""
    g = gen(vocab + beams)
    logits = ((randn(g, groups, beams, vocab) * 12).round() / 16).to(dtype)           # many equal ones
    scores = -(randn(g, groups, beams) * 24).round().abs() / 8
    for kept in (8, 9, 16, 17, 18, 19, 20, 31, 32, 33, 34, 47, 63, 64):
        _, parents, codes, _ = rq.BeamSearch(groups, beams, vocab, kept, "raw", dtype).select(logits, scores)
        want = predictor_ref.beam(logits, scores, None, -1, kept, True)
        assert torch.equal(parents.cpu().long(), want[1]) and torch.equal(codes.cpu().long(), want[2]), kept
        rows = logits.view(-1, vocab)
        best = torch.sort(rows.double().cpu(), dim=1, descending=True, stable=True).indices[:, :kept]
        assert torch.equal(rq.log_probs(rows, top=kept).top_codes.cpu().long(), best), kept
