"""The code predictor's operators on the GPU where calls can go wrong: sizes at
the seams of a layout, tensors that lie differently, ties, streams."""

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


@pytest.mark.parametrize("vocab", [300, 70000])
def test_beam_steps_without_a_pause(vocab):
    """Steps one behind the other, all of a step's small tensors in one cache line: each kernel has to see what the
    one before it wrote, not what the line held earlier."""
    groups, beams, steps = 1, 4, 24
    g = gen(vocab)
    logits = (randn(g, steps, groups, beams, vocab) * 8).round() / 16
    search = rq.BeamSearch(groups, beams, vocab, mode="raw")
    line = torch.zeros(3 * 16, dtype=torch.uint8, device=DEV)
    scores, parents, codes = (line[16 * i:16 * (i + 1)].view(t).view(groups, beams)
                              for i, t in enumerate((F32, torch.int32, torch.int32)))
    state = torch.arange(groups * beams * 64, dtype=torch.int32, device=DEV).view(groups, beams, 64).contiguous()
    first = state.clone()
    other = torch.empty_like(state)

    def walk(wait):
        scores.zero_()
        parents.zero_()
        state.copy_(first)
        kept = []
        for q in range(steps):
            rq.rvq_beam_select(search.dims, logits[q], scores, None, -1, scores, parents, codes, None, search.workspace)
            wait()
            search.reorder(parents, state, other)
            wait()
            search.reorder(parents, other, state)
            search.reorder(parents, state, state)
            wait()
            kept.append((scores.clone(), parents.clone(), codes.clone(), state.clone()))
        return kept

    want = walk(torch.cuda.synchronize)
    got = walk(lambda: None)
    for q, (a, b) in enumerate(zip(want, got)):
        for x, y in zip(a, b):
            assert torch.equal(x, y), q
    p = torch.stack([k[1] for k in want])
    assert bool((p >= 0).all()) and bool((p != p[0]).any())
