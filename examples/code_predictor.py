"""A code predictor trained and used on the quantiser's codes.

    python examples/code_predictor.py [--frames 2000] [--steps 60] [--beams 4]

1. Frames are encoded and decoded as usual (RVQ.encode, RVQ.decode).
2. A small predictor (layer norm, then one linear head per stage) learns to
   give each stage's codes from the stage's residual.  Its teacher is the
   quantiser itself: the nearest entries of a stage and minus their distances,
   as the teacher's top logits (distill_loss).
3. The predictor answers by beam search over the stages: the best candidates of
   all beams (BeamSearch.select), the residuals and the codes so far following
   them (BeamSearch.reorder); the best beam's codes go to RVQ.decode.
4. The same search with the residual's own squared norm as its score
   (mode "raw") encodes frames better than one code a stage at a time does.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import residual_vector_quantisation_gb300 as rq  # noqa: E402
import rvq_inputs as ri  # noqa: E402

TOP = 16
TEMPERATURE = 2.0


class Predictor(torch.nn.Module):
    """Per stage: logits = head[q] . layer_norm(residual)."""

    def __init__(self, stages, width, codes, device):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(width, device=device))
        self.bias = torch.nn.Parameter(torch.zeros(width, device=device))
        self.head = torch.nn.Parameter(torch.randn(stages, codes, width, device=device) / width ** 0.5)

    def forward(self, residual, q):
        return rq.layer_norm(residual, self.weight, self.bias) @ self.head[q].t()


def stage_outputs(w):
    """What each code of each stage takes from the residual: [Q][K][D]."""
    return torch.einsum("qdc,qkc->qkd", w["w_out"], w["codebook"])


def search(frames, out, beams, logits_of, mode):
    """Codes [N][Q] of the best beam, scored by logits_of(residual, q) (mode "logits") or by minus the residual's
    squared norm (mode "raw")."""
    n, width = frames.shape
    stages, codes, _ = out.shape
    step = rq.BeamSearch(n, beams, codes, mode=mode, device=frames.device)
    scores = step.first_scores()
    if mode == "raw":
        scores[:, 0] = -(frames * frames).sum(1)
    residual = frames[:, None].expand(n, beams, width).contiguous()
    history = torch.zeros((n, beams, stages), dtype=torch.int32, device=frames.device)
    for q in range(stages):
        logits = logits_of(residual.view(n * beams, width), q).view(n, beams, codes)
        scores, parents, chosen, _ = step.select(logits, scores)
        residual = step.reorder(parents, residual)
        history = step.reorder(parents, history)
        history[:, :, q] = chosen
        # a beam that found no candidate has code -1 and score -inf: what it takes away does not matter
        residual -= out[q][chosen.clamp(min=0).long()]
    return history[:, 0].contiguous()


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--frames", type=int, default=2000)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--beams", type=int, default=4)
    args = ap.parse_args(argv)
    torch.manual_seed(0)
    dev = torch.device("cuda:0")

    load = ri.WORKLOAD_BY_NAME["tiny"]
    w = ri.weights_to_torch(ri.make_weights(load), dev)
    rvq = rq.RVQ(w["w_in"], w["codebook"], w["w_out"], device=dev)
    frames = torch.randn(args.frames, load.D, device=dev)
    out = stage_outputs(w)

    def error(codes):
        return ((frames - rvq.decode(codes)) ** 2).mean().item()

    codes = rvq.encode(frames)
    print(f"one code a stage at a time: error {error(codes):.4f}")

    # the teacher: minus the distances of a stage's nearest entries, from the quantiser's own residuals
    residuals, teacher = [], []
    r = frames.clone()
    for q in range(load.Q):
        p = r @ w["w_in"][q].t()
        distance = (p * p).sum(1, keepdim=True) - 2 * p @ w["codebook"][q].t() + (w["codebook"][q] ** 2).sum(1)
        top = torch.topk(-distance, TOP, dim=1)
        lse = torch.logsumexp(-distance / TEMPERATURE, 1)
        residuals.append(r.clone())
        teacher.append((top.values.contiguous(), top.indices.to(torch.int32), lse))
        r = r - out[q][codes[:, q].long()]

    model = Predictor(load.Q, load.D, load.K, dev)
    optimizer = torch.optim.Adam(model.parameters(), lr=3e-3)
    losses = []
    for step in range(args.steps):
        optimizer.zero_grad(set_to_none=True)
        loss = sum(rq.distill_loss(model(residuals[q], q), *teacher[q], temperature=TEMPERATURE).mean()
                   for q in range(load.Q)) / load.Q
        loss.backward()
        optimizer.step()
        losses.append(loss.item())
    print(f"distillation loss: {losses[0]:.4f} -> {losses[-1]:.4f} in {args.steps} steps")

    with torch.no_grad():
        predicted = search(frames, out, args.beams, model, "logits")
    print(f"the predictor's codes, {args.beams} beams: error {error(predicted):.4f}")

    norms = (out * out).sum(2)
    searched = search(frames, out, args.beams, lambda r, q: 2 * r @ out[q].t() - norms[q], "raw")
    print(f"the quantiser's codes, {args.beams} beams: error {error(searched):.4f}")
    return losses, error(codes), error(predicted), error(searched)


if __name__ == "__main__":
    main()
