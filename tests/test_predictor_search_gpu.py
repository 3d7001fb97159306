"""The example's search by its predictor's log probabilities, against the same
steps in torch."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("code_predictor", os.path.join(ROOT, "examples", "code_predictor.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("beams", [1, 3, 8])
def test_search_by_log_probabilities(example, beams):
    """Every beam's logits are a table's row for its state, on a grid, and the rows of a stage are permutations of one
    row: the sums of their exponentials differ by rounding alone, so the order is that of the logits' own sums."""
    g = torch.Generator(device=DEV)
    g.manual_seed(beams)
    n, width, stages, codes = 40, 16, 5, 37
    frames = torch.arange(n, device=DEV, dtype=torch.float32)[:, None].expand(n, width).contiguous()
    row = torch.arange(codes, device=DEV, dtype=torch.float32) / 4
    # one permutation a stage and state; a state is a number below 64 that the residual's last column carries
    tables = torch.stack([torch.stack([row[torch.randperm(codes, generator=g, device=DEV)] for _ in range(64)])
                          for _ in range(stages)])
    out = torch.zeros(stages, codes, width, device=DEV)
    out[:, :, 0] = -torch.arange(codes, device=DEV, dtype=torch.float32)      # the residual's first column adds codes up

    def logits_of(residual, q):
        return tables[q, residual[:, 0].long() % 64]

    got = example.search(frames, out, beams, logits_of, "logits")
    assert got.shape == (n, stages) and got.dtype == torch.int32
    # the same search with whole numbers: (sum of 4 * logits, lower beam, larger logit, lower code)
    steps = (tables * 4).long().tolist()
    for f in range(n):
        held = [(0, f, [])]
        for q in range(stages):
            offers = sorted((-(score + steps[q][state % 64][c]), b, -steps[q][state % 64][c], c)
                            for b, (score, state, _) in enumerate(held) for c in range(codes))[:beams]
            held = [(-t, held[b][1] + c, held[b][2] + [c]) for t, b, _, c in offers]
        assert got[f].tolist() == held[0][2], f
