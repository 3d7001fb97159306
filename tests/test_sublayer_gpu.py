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
