"""The predictor's autograd functions on the CPU: what they do around the kernels, whose calls are replaced by torch
statements of the same."""

import pytest
import torch

import residual_vector_quantisation_gb300 as rq
import sublayer_ref as ref


def stays(rows, mask):
    keep, factor = ref.stays(rows.numel(), mask.p, mask.seed, mask.offset)
    return torch.from_numpy(keep).view(rows.shape), factor


def drop(rows, mask):
    if mask is None:
        return rows
    keep, factor = stays(rows, mask)
    return torch.where(keep, rows * factor, 0.0)


def dropout(x, mask, y, residual=None):
    y.copy_(drop(x, mask) if residual is None else drop(x, mask) + residual)


def rms_norm(x, weight, eps, y, rstd=None, residual=None, mask=None, total=None):
    h = drop(x, mask) if residual is None else drop(x, mask) + residual
    if total is not None:
        total.copy_(h)
    rstd.copy_(1 / torch.sqrt((h * h).mean(1) + eps))
    y.copy_(h * rstd[:, None] * (1 if weight is None else weight))


def rms_norm_backward(dy, total, weight, rstd, dresidual, dweight, workspace, dtotal=None, mask=None, dx=None):
    u, g = total * rstd[:, None], dy * (1 if weight is None else weight)
    dh = rstd[:, None] * (g - u * (g * u).mean(1, keepdim=True))
    if dtotal is not None:
        dh = dh + dtotal
    for out, value in ((dresidual, dh), (dx, None if mask is None else drop(dh, mask)), (dweight, (dy * u).sum(0))):
        if out is not None:
            out.copy_(value)


@pytest.fixture(autouse=True)
def statements(monkeypatch):
    for name, f in (("rvq_dropout", dropout), ("rvq_rms_norm", rms_norm), ("rvq_rms_norm_backward", rms_norm_backward),
                    ("rvq_rms_norm_workspace_bytes", lambda rows, width: 16)):
        monkeypatch.setattr(rq, name, f)


def tensors(n, *shape, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(shape, generator=g, dtype=torch.float64) for _ in range(n)]


def leaves(*values):
    return [v.clone().requires_grad_() for v in values]


@pytest.mark.parametrize("mask", [None, rq.rvq_dropout_mask(0.3, 5)])
def test_rms_norm_gradients_have_memory_of_their_own(mask):
    """A second pass adds to each leaf's gradient once, and a change of one leaves the other's."""
    x, r, up, ut = tensors(4, 3, 4, 8)
    x, r = leaves(x, r)

    def both_passes():
        torch.autograd.backward(rq.rms_norm(x, None, 1e-6, r, mask), (up, ut))

    both_passes()
    first = x.grad.clone(), r.grad.clone()
    both_passes()
    assert torch.equal(x.grad, 2 * first[0]) and torch.equal(r.grad, 2 * first[1])
    x.grad.mul_(0.5)
    assert torch.equal(r.grad, 2 * first[1])


@pytest.mark.parametrize("mask", [None, rq.rvq_dropout_mask(0.3, 5)])
def test_gradient_of_the_sum_alone_passes_by_the_norm(mask):
    """Rows whose norm is not finite (zeros without an eps, infinities, NaN) leave the sum's gradient as it is."""
    x, r, ut = tensors(3, 5, 8)
    x[0] = r[0] = 0.0
    x[1, 2], r[2, 3] = torch.nan, torch.inf
    x, r, w = leaves(x, r, torch.ones(8, dtype=torch.float64))
    y, total = rq.rms_norm(x, w, 0.0, r, mask)
    assert mask is not None or not bool(torch.isfinite(y[:3]).all(1).any())
    total.backward(ut)
    assert torch.equal(r.grad, ut) and torch.equal(x.grad, drop(ut, mask))
    assert bool((w.grad == 0).all())
    # x or residual alone, the sum's gradient as it comes from a sum
    for given in (0, 1):
        a, b = tensors(2, 5, 8)
        one = leaves((a, b)[given])[0]
        rq.rms_norm(*((one, w, 1e-6, b) if given == 0 else (a, w, 1e-6, one)), mask)[1].sum().backward()
        ones = torch.ones_like(a)
        assert torch.equal(one.grad, drop(ones, mask) if given == 0 else ones)


def test_a_mask_changed_between_the_passes():
    """The backward pass is the forward pass's, whatever became of the mask's fields since: one mask that serves one
    place of a model after the other."""
    x, r, up, ut = tensors(4, 6, 8)
    for call in (lambda x, r, m: (rq.dropout(x, m, r),), lambda x, r, m: rq.rms_norm(x, None, 1e-6, r, m)):
        want, got = leaves(x, r), leaves(x, r)
        out = call(*want, rq.rvq_dropout_mask(0.3, 5, 1))
        torch.autograd.backward(out, (up, ut)[:len(out)])
        mask = rq.rvq_dropout_mask(0.3, 5, 1)
        out = call(*got, mask)
        mask.p, mask.seed, mask.offset = 0.9, 6, 2
        torch.autograd.backward(out, (up, ut)[:len(out)])
        for a, b in zip(got, want):
            assert torch.equal(a.grad, b.grad)


def test_dropout_without_a_mask_drops_nothing():
    """As root-mean-square norm takes it: a model in evaluation hands on None."""
    x, r, up = tensors(3, 2, 3, 8)
    x, r = leaves(x, r)
    y = rq.dropout(x, None)
    assert torch.equal(y, x) and y.data_ptr() != x.data_ptr()
    y = rq.dropout(x, None, r)
    assert torch.equal(y, x + r)
    y.backward(up)
    assert torch.equal(x.grad, up) and torch.equal(r.grad, up)
    for empty in (x[:0], x[..., :0]):
        assert rq.dropout(empty, None).shape == empty.shape
        assert rq.dropout(empty, None, empty).shape == empty.shape


def test_dropout_refuses_another_residual_without_elements_too():
    x = torch.zeros(2, 3, 8)
    mask = rq.rvq_dropout_mask(0.1, 1)
    for a, b in ((x, x[:1]), (x[:0], x[:1, :1]), (x[:0], x[:0].double())):
        for m in (mask, None):
            with pytest.raises(ValueError):
                rq.dropout(a, m, b)


def log_probs(logits, codes, temperature, log_p=None, entropy=None, lse=None, stats=None, top_log_probs=None,
              top_codes=None):
    lp = torch.log_softmax(logits / temperature, 1)
    if log_p is not None:
        log_p.copy_(lp.gather(1, codes.long()[:, None])[:, 0])
    if entropy is not None:
        entropy.copy_(-(lp.exp() * lp).sum(1))
    lse.copy_(torch.logsumexp(logits / temperature, 1))
    if top_codes is not None:
        best = torch.sort(lp, dim=1, descending=True, stable=True)
        top_log_probs.copy_(best.values[:, :top_codes.shape[1]])
        top_codes.copy_(best.indices[:, :top_codes.shape[1]])


def log_probs_backward(grad_log_probs, grad_entropy, grad_lse, logits, codes, temperature, stats, entropy, dlogits):
    lp = torch.log_softmax(logits / temperature, 1)
    p, g = lp.exp(), torch.zeros_like(lp)
    if grad_log_probs is not None:
        g += grad_log_probs[:, None] * (torch.nn.functional.one_hot(codes.long(), lp.shape[1]) - p)
    if grad_entropy is not None:
        g -= grad_entropy[:, None] * p * (lp + entropy[:, None])
    if grad_lse is not None:
        g += grad_lse[:, None] * p
    dlogits.copy_(g / temperature)


def layer_norm(x, weight, bias, eps, y, mean=None, rstd=None):
    mean.copy_(x.mean(1))
    rstd.copy_(1 / torch.sqrt(x.var(1, unbiased=False) + eps))
    y.copy_((x - mean[:, None].to(x)) * rstd[:, None].to(x))


def layer_norm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias, workspace):
    r = rstd[:, None].to(x)
    h = (x - mean[:, None].to(x)) * r
    dx.copy_(r * (dy - dy.mean(1, keepdim=True) - h * (dy * h).mean(1, keepdim=True)))


def distill(logits, top_logits, top_codes, teacher_lse, weights, temperature, loss, lse=None):
    loss.copy_(logits.sum(1))


def distill_backward(grad, logits, top_logits, top_codes, teacher_lse, weights, temperature, lse, dlogits):
    dlogits.copy_(grad[:, None].expand_as(logits))


@pytest.fixture
def row_statements(monkeypatch):
    for name, f in (("rvq_log_probs", log_probs), ("rvq_log_probs_backward", log_probs_backward),
                    ("rvq_layer_norm", layer_norm), ("rvq_layer_norm_backward", layer_norm_backward),
                    ("rvq_distill", distill), ("rvq_distill_backward", distill_backward)):
        monkeypatch.setattr(rq, name, f)


RESULTS = {  # call(x, r) and whether each result is one that the backward pass does not read
    "dropout": (lambda x, r: (rq.dropout(x, rq.rvq_dropout_mask(0.3, 5), r),), [True]),
    "rms_norm of x": (lambda x, r: (rq.rms_norm(x),), [True]),
    "rms_norm of a sum": (lambda x, r: rq.rms_norm(x, None, 1e-6, r), [True, False]),
    "log_probs": (lambda x, r: rq.log_probs(x, (r[..., 0] > 0).long(), entropy=True, top=2)[:4], [True, False, True, True]),
    "layer_norm": (lambda x, r: (rq.layer_norm(x),), [True]),
    "distill_loss": (lambda x, r: (rq.distill_loss(x, r[..., :2].detach(), (r[..., :2] > 0).int()),), [True]),
}


@pytest.mark.parametrize("shape", [(6, 8), (2, 3, 8), (8,)])
@pytest.mark.parametrize("name", RESULTS)
def test_results_can_be_changed_in_place(name, shape, row_statements):
    """As those of torch's own operators: scaled by 3, they have 3 times the gradient.  What the backward pass reads (the
    sum that was normalised, the entropy) is guarded as a saved result of torch's is."""
    call, free = RESULTS[name]
    x, r = tensors(2, *shape)
    x, r = x.float(), r.float()
    for i, ours in enumerate(free):
        with torch.no_grad():
            want = call(x, r)[i].clone()
            assert torch.equal(call(x, r)[i].mul_(3.0), 3.0 * want)
        a, b = leaves(x, r)
        result = call(a, b)[i]
        if not result.requires_grad:
            continue
        result.sum().backward()
        c, d = leaves(x, r)
        changed = call(c, d)[i]
        changed.mul_(3.0)
        if ours:
            changed.sum().backward()
            assert torch.allclose(c.grad, 3.0 * a.grad, rtol=1e-5, atol=1e-6)
            assert d.grad is None or torch.allclose(d.grad, 3.0 * b.grad, rtol=1e-5, atol=1e-6)
        else:
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                changed.sum().backward()


@pytest.mark.parametrize("shape", [(6, 8), (2, 3, 8), (8,)])
@pytest.mark.parametrize("mask", [None, rq.rvq_dropout_mask(0.3, 5)])
def test_gradients_that_pass_through_have_memory_of_their_own(mask, shape):
    """What comes from above goes on as it is, as through an addition: no leaf's gradient is another's memory, nor that of
    the gradient given."""
    x, r, o, up = tensors(4, *shape)
    for call in (lambda x, r: rq.rms_norm(x, None, 1e-6, r, mask)[1], lambda x, r: rq.dropout(x, mask, r)):
        a, b, c = leaves(x, r, o)
        given = up.clone()
        for _ in range(2):
            (call(a, b) + c).backward(given)
        call(a, b).backward(given)
        assert torch.equal(given, up)
        for leaf, times in ((a, drop(up.view(-1, 8), mask).view(shape)), (b, up), (c, up * 2 / 3)):
            assert torch.allclose(leaf.grad, 3 * times)
        places = [t.data_ptr() for t in (a.grad, b.grad, c.grad, given)]
        assert len(set(places)) == 4
        a.grad = b.grad = c.grad = None
        call(a, b).backward(given)
        a.grad.zero_(), b.grad.zero_()
        assert torch.equal(given, up)
