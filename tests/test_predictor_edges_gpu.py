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


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------

def rows_in(t, stride, shift):
    """The same rows, `stride` elements apart, the first `shift` elements into a buffer of NaN."""
    rows, width = t.shape
    buffer = torch.full((rows * stride + shift + 16,), math.nan, dtype=t.dtype, device=t.device)
    view = buffer.as_strided((rows, width), (stride, 1), shift)
    view.copy_(t)
    return view


def untouched(view):
    """What lies beside the rows of rows_in is NaN as before."""
    buffer = torch.empty(0, dtype=view.dtype, device=DEV).set_(view.untyped_storage())
    held = buffer.clone()
    held.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(math.nan)
    return bool(torch.isnan(held).all())


def check_norm(x, dy, w, b, places):
    """places: (stride, shift) of x, dy, y and dx; outputs and workspace hold NaN before."""
    rows, width = x.shape
    xv, dyv = rows_in(x, *places[0]), rows_in(dy, *places[1])
    y, dx = (rows_in(torch.full_like(x, math.nan), *p) for p in places[2:])
    mean, rstd = (torch.full((rows,), math.nan, device=DEV) for _ in range(2))
    rq.rvq_layer_norm(xv, w, b, 1e-5, y, mean, rstd)
    dw, db = torch.full_like(w, math.nan), torch.full_like(b, math.nan)
    ws = torch.full((rq.rvq_layer_norm_workspace_bytes(rows, width),), 0xFF, dtype=torch.uint8, device=DEV)
    rq.rvq_layer_norm_backward(dyv, xv, w, mean, rstd, dx, dw, db, ws)
    val, tol = ref.norm(x, w, b, 1e-5, dy)
    for k, got in (("y", y), ("dx", dx), ("dweight", dw), ("dbias", db)):
        ref.check(got, val[k], tol[k], k)
    assert untouched(y) and untouched(dx)


@pytest.mark.parametrize("dtype,pdtype", [(F32, F32), (BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("width", [8191, 8192, 8193, 8194, 8195, 8199, 8201, 12287, 12289, 12290, 12291, 12295, 12297,
                                   16381, 16383])
def test_norm_last_vector_of_wide_rows(width, dtype, pdtype):
    """Rows on 16-byte boundaries whose width is no multiple of a vector: the last columns count like the others.
    One row (its stride does not matter) and rows some vectors apart."""
    g = gen(width)
    w, b = (1 + 0.2 * randn(g, width)).to(pdtype), (0.3 * randn(g, width)).to(pdtype)
    for rows, stride in ((1, width), (5, (width + 15) // 8 * 8), (160, (width + 7) // 8 * 8)):
        x, dy = randn(g, rows, width).to(dtype), randn(g, rows, width).to(dtype)
        check_norm(x, dy, w, b, [(stride, 0)] * 4)


# ---------------------------------------------------------------------------
# streams
# ---------------------------------------------------------------------------

def busy(n=30):
    big = torch.ones((4096, 4096), device=DEV)
    for _ in range(n):
        big = big @ big * 1e-4
    return big


def test_beam_search_on_a_stream_of_its_own():
    """The caller's stream runs beside a current stream that has freed memory which it still writes, and takes what is
    freed as soon as the calls return."""
    g = gen(3)
    logits, scores = (randn(g, 5, 4, 300) * 48).round() / 16, -(randn(g, 5, 4) * 24).round().abs() / 8
    state = randn(g, 5, 4, 1000)
    finished = torch.zeros((5, 4), dtype=torch.bool, device=DEV)
    search = rq.BeamSearch(5, 4, 300, end_code=7)
    want = search.select(logits, scores, finished)
    moved = search.reorder(want[1], state)
    want, moved = [t.clone() for t in want], moved.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        other = rq.BeamSearch(5, 4, 300, end_code=7)
        held = [t.clone() for t in (logits, scores, finished, state)]
        torch.cuda.synchronize()
        busy()
        for t in [torch.empty_like(t) for t in (*want, moved) for _ in range(4)]:
            t.fill_(1)                           # still to come when the memory is free again
        del t
        with torch.cuda.stream(side):
            busy(10)                             # the step waits while the current stream goes on
        got = other.select(*held[:3], stream=side)
        after = other.reorder(got[1], held[3], stream=side)
        del other, held
        junk = [torch.full((4096,), 3, dtype=torch.uint8, device=DEV) for _ in range(64)]
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip((*want, moved), (*got, after)):
            assert torch.equal(a, b)
        del junk
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# reordering
# ---------------------------------------------------------------------------

def follow(state, parents):
    """[layers][groups][beams][...] by the parents."""
    groups = torch.arange(state.shape[1], device=DEV)[:, None]
    return state[:, groups, parents.long()]


def test_reorder_states_that_lie_between_one_another():
    """The keys and values of one cache in place, and halves of one buffer moved to one another's other halves: their
    address ranges overlap, their rows do not."""
    g = gen(5)
    layers, groups, beams = 3, 6, 4
    parents = torch.randint(0, beams, (groups, beams), generator=g, device=DEV, dtype=torch.int32)
    dims = rq.rvq_beam_dims(groups, beams, 10, beams, rq.RVQ_BEAM_RAW, 0)
    cache = randn(g, layers, groups, beams, 2, 24, 8)
    want = follow(cache, parents)
    both = [(cache[:, :, :, i], cache[:, :, :, i]) for i in range(2)]
    rq.rvq_beam_reorder(dims, parents, rq.rvq_beam_states(both, layered=True))
    assert torch.equal(cache, want)

    buffer = randn(g, layers, groups, beams, 2, 5)
    want = buffer.clone()
    want[..., 1, :] = follow(buffer[..., 0, :], parents)
    rq.rvq_beam_reorder(dims, parents, rq.rvq_beam_states([(buffer[..., 0, :], buffer[..., 1, :])], layered=True))
    assert torch.equal(buffer, want)

    # kept as it was and reordered in place by one call: the move is first
    state, held = randn(g, layers, groups, beams, 40), torch.zeros((layers, groups, beams, 40), device=DEV)
    want = follow(state, parents)
    rq.rvq_beam_reorder(dims, parents, rq.rvq_beam_states([(state, state), (state, held)], layered=True))
    assert torch.equal(held, want) and torch.equal(state, want)


def test_reorder_python_refuses_overlaps():
    search = rq.BeamSearch(3, 4, 10)
    parents = torch.zeros((3, 4), dtype=torch.int32, device=DEV)
    state = torch.zeros((3, 4, 16), device=DEV)
    with pytest.raises(rq.RVQError):
        search.reorder(parents, state, torch.zeros((3, 1, 16), device=DEV).expand(3, 4, 16))
    wide = torch.zeros(3 * 4 * 16 + 4, device=DEV)
    with pytest.raises(rq.RVQError):
        search.reorder(parents, wide[4:].view(3, 4, 16), wide[:-4].view(3, 4, 16))
    # a source may be expanded: it is only read
    assert search.reorder(parents, torch.ones((3, 1, 16), device=DEV).expand(3, 4, 16)).eq(1).all()


def test_norm_and_distill_side_by_side_in_one_buffer():
    """Outputs in the other half of their inputs' rows, and between the inputs' rows: nothing is shared."""
    g = gen(7)
    rows, width = 50, 96
    w = 1 + 0.2 * randn(g, width)
    buffer = randn(g, rows, 3 * width)
    x, dy, out = buffer.split(width, 1)
    val, tol = ref.norm(x, w, None, 1e-5, dy)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    rq.rvq_layer_norm(x, w, None, 1e-5, out, mean, rstd)
    ref.check(out, val["y"], tol["y"], "y")
    rq.rvq_layer_norm_backward(dy, x, w, mean, rstd, out, None, None, None)
    ref.check(out, val["dx"], tol["dx"], "dx")
    buffer = randn(g, 2 * rows, width)
    z, d = buffer[0::2], buffer[1::2]
    t, codes = torch.topk(randn(g, rows, width), 8, dim=1)
    loss = torch.empty(rows, device=DEV)
    val, tol, _ = ref.distill(z, t, codes.to(torch.int32), None, None, 1.0)
    rq.rvq_distill(z, t, codes.to(torch.int32), None, None, 1.0, loss, dlogits=d)
    ref.check(loss, val["loss"], tol["loss"], "loss")
    ref.check(d, val["dlogits"], tol["dlogits"], "dlogits")


# ---------------------------------------------------------------------------
# the beam step's order
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("vocab,select", [(40, 3), (1025, 5), (70000, 4), (70000, 40)])
def test_beam_ties_of_rounded_totals(vocab, select):
    """Scores so large that a total's rounding swallows what tells the values apart.  Raw values: their totals are
    equal, the lower code is first.  Log probabilities: within a beam the larger logit is first all the same."""
    rising = (torch.arange(vocab, device=DEV) % 97).float() / 1024                     # the larger ones are not the first ones
    scores = torch.tensor([[1048576.0, 1048576.0]], device=DEV)        # an ulp of 1/8
    logits = torch.stack([rising, rising.flip(0)])[None].contiguous()
    for raw in (True, False):
        search = rq.BeamSearch(1, 2, vocab, select, "raw" if raw else "logits")
        out, parents, codes, _ = search.select(logits, scores)
        total = scores.double()[:, :, None] + (logits.double() if raw else torch.log_softmax(logits.double(), 2))
        total = total.float()                             # few values, of many candidates each
        assert len(total.unique()) < len(rising.unique())
        values, z = total[0].tolist(), logits[0].tolist()
        best = sorted((-values[b][v], b, 0.0 if raw else -z[b][v], v) for b in range(2) for v in range(vocab))[:select]
        assert parents[0].tolist() == [c[1] for c in best]
        assert codes[0].tolist() == [c[3] for c in best], raw
        assert out[0].tolist() == [-c[0] for c in best]


def test_beam_of_one_from_the_last_position():
    g = gen(8)
    logits = (randn(g, 6, 3, 1030) * 48).round() / 16
    scores = -(randn(g, 6, 1) * 24).round().abs() / 8
    search = rq.BeamSearch(6, 1, 1025, 1)
    out, parents, codes, _ = search.select(logits[:, -1:, :1025], scores)
    assert torch.equal(codes, logits[:, -1, :1025].argmax(1, keepdim=True).int()) and not bool(parents.any())
    want = scores.double() + torch.log_softmax(logits[:, -1, :1025].double(), 1).amax(1, keepdim=True)
    # as for every step: 16 roundings of the largest term
    ref.check(out, want, 16 * ref.U * (want.abs().cpu() + logits.abs().max().item() + math.log(1025)), "scores")


# ---------------------------------------------------------------------------
# distillation
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("vocab", [100, 3000, 20000])
def test_distill_lowest_temperature(vocab, tail):
    """At the lowest temperature that is taken both sides are all on their largest logit: no loss, no gradient."""
    g = gen(vocab)
    z = randn(g, 5, vocab)
    t, codes = torch.topk(z, 4, dim=1)
    t, codes, lse = t - t[:, :1], codes.to(torch.int32), torch.zeros(5, device=DEV) if tail else None
    loss, d = torch.full((5,), math.nan, device=DEV), torch.full_like(z, math.nan)
    rq.rvq_distill(z, t, codes, lse, None, 4.3e-39, loss, dlogits=d)
    assert bool((loss == 0).all()) and bool((d == 0).all())


# ---------------------------------------------------------------------------
# kernels that a call reaches only by where its tensors lie, or by its counts
# ---------------------------------------------------------------------------

def places_of(width):
    """(stride, shift) of x, dy, y and dx."""
    return {"all": [(width + 1, 0), (width + 3, 1), (width + 2, 5), (width, 3)],
            "dense results": [(width + 3, 0), (width, 0), (width, 0), (width, 0)],
            "y": [(width + 8, 0), (width + 8, 0), (width + 8, 1), (width + 8, 0)],
            "dx": [(width + 8, 0), (width + 8, 0), (width + 8, 0), (width + 9, 0)],
            "dy": [(width + 8, 2), (width + 8, 1), (width + 8, 2), (width + 8, 2)]}


@pytest.mark.parametrize("dtype,pdtype", [(F32, F32), (BF16, F32), (BF16, BF16), (F16, F32), (F16, F16)])
@pytest.mark.parametrize("width", [1, 40, 256, 300, 700, 1000, 1024])
def test_norm_tensors_that_lie_differently(width, dtype, pdtype):
    """Up to 1024 columns element by element: a warp's rows, its sums added to the other warps' in shared memory.  Rows
    that leave warps, and blocks' last rounds, without work; several rounds."""
    g = gen(width)
    w, b = (1 + 0.2 * randn(g, width)).to(pdtype), (0.3 * randn(g, width)).to(pdtype)
    for rows in (1, 3, 37, 2600):
        x, dy = randn(g, rows, width).to(dtype), randn(g, rows, width).to(dtype)
        for places in places_of(width).values():
            check_norm(x, dy, w, b, places)


@pytest.mark.parametrize("dtype,pdtype", [(F32, F32), (BF16, F32), (F16, F16)])
@pytest.mark.parametrize("width", [1025, 1500, 4097, 8192, 9001, 12289, 16384])
def test_norm_wide_tensors_that_lie_differently(width, dtype, pdtype):
    g = gen(width)
    w, b = (1 + 0.2 * randn(g, width)).to(pdtype), (0.3 * randn(g, width)).to(pdtype)
    for rows, kinds in ((1, ("all",)), (161, ("all", "dense results", "dx"))):
        x, dy = randn(g, rows, width).to(dtype), randn(g, rows, width).to(dtype)
        for kind in kinds:
            check_norm(x, dy, w, b, places_of(width)[kind])


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("width,stride", [(768, 771), (1025, 1031), (96, 100)])
def test_layer_norm_of_a_slice(width, stride, dtype):
    """The differentiable function on part of wider rows: its results and gradients are dense."""
    g = gen(stride)
    x, dy = randn(g, 300, width).to(dtype), randn(g, 300, width).to(dtype)
    w, b = 1 + 0.2 * randn(g, width), 0.3 * randn(g, width)
    wide = rows_in(x, stride, 0)
    leaf = [t.detach().requires_grad_() for t in (wide, w, b)]
    y = rq.layer_norm(*leaf)
    y.backward(dy)
    val, tol = ref.norm(x, w, b, 1e-5, dy)
    for k, got in (("y", y.detach()), ("dx", leaf[0].grad), ("dweight", leaf[1].grad), ("dbias", leaf[2].grad)):
        ref.check(got, val[k], tol[k], k)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("groups,beams,vocab,select", [(1, 2, 70000, 64), (2, 3, 65536, 48), (1, 1, 140000, 33),
                                                       (1, 64, 40000, 64), (3, 5, 20000, 64)])
def test_beam_many_kept_of_long_rows(groups, beams, vocab, select, dtype):
    """A row over several blocks with more than 32 entries kept: the bar comes from the halves of the lanes."""
    g = gen(vocab + select)
    logits = ((randn(g, groups, beams, vocab) * 48).round() / 16).to(dtype)
    scores = -(randn(g, groups, beams) * 24).round().abs() / 8
    finished = torch.zeros((groups, beams), dtype=torch.bool, device=DEV)
    finished[0, -1] = beams > 1
    for raw in (True, False):
        for z in (logits, (logits * 0.25).round()):         # the second: many equal totals
            if not raw and beams > 1:
                # equal totals of different beams are told apart by rounding that the 64-bit statement does not have:
                # one beam a group alive
                scores = torch.where(torch.arange(beams, device=DEV) == beams // 2 - 1, scores, -INF)
            search = rq.BeamSearch(groups, beams, vocab, select, "raw" if raw else "logits", dtype, vocab - 1)
            out, parents, codes, done = search.select(z, scores, finished)
            want = ref_beam(z, scores, finished, vocab - 1, select, raw)
            assert torch.equal(parents.long(), want[1]) and torch.equal(codes.long(), want[2])
            size = z.float().abs().max().item() + math.log(vocab)
            there = torch.isfinite(want[0])
            ref.check(out, want[0], 0.0 if raw else 16 * ref.U * torch.where(there, want[0].abs() + size, 0.0), "scores")
            ended = (want[1] < 0) | (want[2] == vocab - 1)
            assert torch.equal(done, ended | finished.gather(1, want[1].clamp(min=0)))


def ref_beam(logits, scores, finished, end_code, select, raw):
    """predictor_ref.beam's rule by one stable sort a group (its lists take long for millions of candidates)."""
    groups, beams, vocab = logits.shape
    x = logits.float() if raw else logits.double()
    total = scores[:, :, None] + x if raw else scores.double()[:, :, None] + torch.log_softmax(x, 2)
    only = torch.arange(vocab, device=DEV) == end_code
    total = torch.where(finished[:, :, None], torch.where(only, scores[:, :, None].to(total.dtype), -INF), total)
    # equal totals of one beam: in log probabilities the larger logit, which in 64 bits has the larger total
    value, at = torch.sort(total.reshape(groups, -1), dim=1, descending=True, stable=True)
    value, at = value[:, :select], at[:, :select]
    there = value > -INF
    return torch.where(there, value.double(), -INF), torch.where(there, at // vocab, -1), torch.where(there, at % vocab, -1)


def test_quantiser_on_other_streams():
    """RVQ on torch's streams and on one that only has a handle, with frames that are converted on the way."""
    import rvq_inputs as ri
    load = ri.WORKLOAD_BY_NAME["tiny"]
    w = ri.weights_to_torch(ri.make_weights(load), DEV)
    rvq = rq.RVQ(w["w_in"], w["codebook"], w["w_out"], device=DEV)
    x = torch.randn(250, load.D, dtype=torch.float64, device=DEV)
    want = [t.clone() for t in rvq.reconstruct(x)]
    side = torch.cuda.Stream()

    class Handle:
        cuda_stream = side.cuda_stream

    for stream in (side, Handle()):
        torch.cuda.synchronize()
        busy()
        with torch.cuda.stream(side):
            busy(10)
        held = x.clone()
        side.wait_stream(torch.cuda.current_stream())
        codes = rvq.encode(held, stream=stream)
        y = rvq.decode(codes, stream=stream)
        both = rvq.reconstruct(held, stream=stream)
        del held
        junk = torch.full_like(x, 9.0)
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip((*want, *want), (codes, y, *both)):
            assert torch.equal(a, b)
        del junk
    torch.cuda.synchronize()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("vocab", [200, 3000, 20000])
def test_distill_infinite_teacher(vocab, tail):
    g = gen(vocab + 1)
    z = randn(g, 3, vocab)
    t, codes = torch.topk(z + randn(g, 3, vocab), 6, dim=1)
    lse = torch.logsumexp(t, 1) + 0.5 if tail else None
    t[1, 2] = INF
    codes = codes.to(torch.int32)
    loss, d = torch.empty(3, device=DEV), torch.empty_like(z)
    rq.rvq_distill(z, t, codes, lse, None, 1.0, loss, dlogits=d)
    assert bool(torch.isfinite(loss[::2]).all()) and bool(torch.isfinite(d[::2]).all())
    if tail:
        assert loss[1].item() == INF and d[1, codes[1, 2].item()].item() == -INF
        assert int(torch.isfinite(d[1]).sum()) == vocab - 1
    else:
        assert bool(torch.isnan(loss[1])) and bool(torch.isnan(d[1]).all())


@pytest.mark.parametrize("vocab", [200, 3000, 20000])
def test_distill_list_with_everything(vocab):
    """A teacher and a mask that leave nothing off the list: with the teacher's logits shifted by their largest, as the
    header says, the tail has no share and the loss is finite."""
    g = gen(vocab + 2)
    z = randn(g, 40, vocab)
    t, codes = torch.topk(z + 60 + 8 * randn(g, 40, vocab), 40, dim=1)
    keep = torch.zeros_like(z, dtype=torch.bool).scatter_(1, codes, True)
    z[~keep] = -INF
    t = t - t[:, :1]
    lse = torch.logsumexp(t.double(), 1).float()
    codes = codes.to(torch.int32)
    loss, d = torch.empty(40, device=DEV), torch.empty_like(z)
    rq.rvq_distill(z, t, codes, lse, None, 1.0, loss, dlogits=d)
    val, tol, _ = ref.distill(z, t, codes, lse, None, 1.0)
    assert bool(torch.isfinite(val["loss"]).all())
    ref.check(loss, val["loss"], tol["loss"], "loss")
    ref.check(d, val["dlogits"], tol["dlogits"], "dlogits")
