"""Cases of the code predictor's operators: layer norm, distillation from a teacher's top logits, and the beam step.

`run` computes a case in its plain form (elementary torch operations in 32
bits), or, where `own` is true, with the framework's kernels.  `exact` states
the same operators in 64 bits, apart from the plain form.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
DEVICE = "cuda"

# A tail mass below this is the rounding of the sum that it is the rest of.
TAIL_FLOOR = 2.0 ** -20


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def _norm(name, rows, width, dtype, train, params="f32", pad=0):
    return {"name": name, "op": "norm", "rows": rows, "width": width, "dtype": dtype, "train": train,
            "params": params, "pad": pad}


def _distill(name, rows, vocab, top, dtype, tail, temperature, masked=0.0, passes=1, ragged=False, mask_code=False):
    return {"name": name, "op": "distill", "rows": rows, "vocab": vocab, "top": top, "dtype": dtype, "tail": tail,
            "temperature": temperature, "masked": masked, "passes": passes, "ragged": ragged, "mask_code": mask_code}


def _beam(name, groups, beams, vocab, select, dtype, raw=False, first=False, finished=0.0, layers=1, length=1,
          width=1024, state="f32"):
    return {"name": name, "op": "beam", "groups": groups, "beams": beams, "vocab": vocab, "select": select,
            "dtype": dtype, "raw": raw, "first": first, "finished": finished, "layers": layers, "length": length,
            "width": width, "state": state}


def listed():
    return [
        # one new frame of a predictor that answers as it goes: nothing but latency
        _norm("norm_one_frame", 1, 1024, "bf16", False),
        # a training batch of 16 utterances of 750 frames at the 32-stage codec's width, in full precision
        _norm("norm_train_768", 12000, 768, "f32", True),
        # rows of an odd width inside wider ones: features with the mask code's column beside them
        _norm("norm_train_odd", 20011, 1025, "f16", True, params="same", pad=6),
        # the benchmark's batch of 256 utterances, as a bf16 training step normalises it
        _norm("norm_train_192k", 192000, 1024, "bf16", True),
        # one utterance's last second: 25 frames of 8 heads, 1024 codes and the mask code
        _distill("distill_25_frames", 200, 1025, 16, "f32", False, 1.0, ragged=True),
        # a training batch of 8 heads with the mask code (never allowed) as the last column, padding frames without weight
        _distill("distill_8_heads", 96000, 1025, 32, "bf16", True, 2.0, masked=0.1, mask_code=True),
        # 32 heads of 1024 codes in full precision: the deep codec's predictor, loss and gradient as separate steps of a graph
        _distill("distill_32_heads", 384000, 1024, 16, "f32", True, 1.5, passes=2),
        # the longest codebook that the quantiser takes, flattened into one vocabulary
        _distill("distill_65536", 4096, 65536, 64, "bf16", True, 1.0, masked=0.05),
        # one utterance, four beams, one stage's codes and the mask code
        _beam("beam_one_utterance", 1, 4, 1025, 4, "bf16"),
        # the quantiser's own search: 12000 frames keep 4 candidates a stage, residuals follow
        _beam("beam_encode_frames", 12000, 4, 1024, 4, "f32", raw=True),
        # a serving batch over 4096 codes, some beams done, with the keys and values of 750 frames
        _beam("beam_4096_with_cache", 16, 8, 4096, 8, "f16", finished=0.125, layers=4, length=750, width=512,
              state="bf16"),
        # the widest selection: twice the beams wanted from 8 x 65536 candidates
        _beam("beam_65536", 32, 8, 65536, 16, "bf16"),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "distill", "beam"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "norm":
        width = _log_int(rng, 40, 16384)
        if rng.random() < 0.6:
            width = max(16, width // 16 * 16)
        rows = _log_int(rng, 1, max(2, 98_000_000 // width))
        case = _norm("", rows, width, dtype, rng.random() < 0.7, rng.choice(["f32", "same"]),
                     rng.choice([0, 0, 8, 3]))
    elif op == "distill":
        vocab = _log_int(rng, 100, 131072)
        if rng.random() < 0.5:
            vocab = max(64, vocab // 64 * 64)
        rows = _log_int(rng, 1, max(2, 130_000_000 // vocab))
        case = _distill("", rows, vocab, _log_int(rng, 4, min(128, vocab // 4)), dtype, rng.random() < 0.6,
                        rng.choice([0.7, 1.0, 2.0, 4.0]), rng.choice([0.0, 0.2]), rng.choice([1, 1, 2]),
                        rng.random() < 0.3, rng.random() < 0.3)
    else:
        vocab = _log_int(rng, 64, 131072)
        beams = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        groups = _log_int(rng, 1, min(4096, max(2, 12_000_000 // (vocab * beams))))
        raw = rng.random() < 0.3
        case = _beam("", groups, beams, vocab, rng.choice([1, beams, beams, 2 * beams]), "f32" if raw else dtype, raw,
                     rng.random() < 0.15, 0.0 if raw else rng.choice([0.0, 0.25]), rng.choice([1, 2, 4]),
                     rng.choice([1, 1, 25, 100]), rng.choice([64, 256, 1000, 1024]), rng.choice(["f32", "bf16"]))
        rows = groups * max(beams, case["select"]) * case["layers"] * case["length"] * case["width"]
        if rows > 90_000_000:
            case["length"] = 1
    del case["name"]
    return case


def work(case):
    if case["op"] == "norm":
        n, e = case["rows"] * case["width"], SIZES[case["dtype"]]
        p = case["width"] * (4 if case["params"] == "f32" else e)
        if not case["train"]:
            return {"bytes": 2 * n * e + 2 * p, "flops": 8 * n}
        # forward: x in, y out; backward: x and dy in, dx out; the parameters and their gradients
        return {"bytes": 5 * n * e + 5 * p + 16 * case["rows"], "flops": 22 * n}
    if case["op"] == "distill":
        rows = case["rows"] - round(case["masked"] * case["rows"])
        e = SIZES[case["dtype"]]
        per = 8 * case["top"] + (4 if case["tail"] else 0) + 8
        reads = (2 if case["passes"] == 2 else 1) * rows * case["vocab"] * e
        return {"bytes": reads + case["rows"] * case["vocab"] * e + rows * per, "flops": 8 * rows * case["vocab"]}
    g, b, n = case["groups"], case["beams"], case["select"]
    live = 1 if case["first"] else b - round(case["finished"] * b)
    row = case["layers"] * case["length"] * case["width"] * SIZES[case["state"]]
    parents = b * (1 - (1 - 1 / b) ** n) if not case["first"] else 1  # distinct ones, where all are as likely
    logits = g * live * case["vocab"]
    return {"bytes": logits * SIZES[case["dtype"]] + g * (n * 13 + b * 5) + g * row * (n + parents), "flops": 4 * logits}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed * 7919 + 17)
    return {"norm": _prepare_norm, "distill": _prepare_distill, "beam": _prepare_beam}[case["op"]](case, gen)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEVICE)


def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device=DEVICE)


def _padded(rows, width, pad, dtype):
    return torch.empty((rows, width + pad), dtype=dtype, device=DEVICE)[:, :width]


def _prepare_norm(case, gen):
    rows, width, dtype = case["rows"], case["width"], DTYPES[case["dtype"]]
    pdtype = torch.float32 if case["params"] == "f32" else dtype
    s = {"case": case, "eps": 1e-5}
    s["x"] = _padded(rows, width, case["pad"], dtype)
    # features with an offset and a scale of their own in every row
    s["x"].copy_(_randn(gen, rows, width) * (0.5 + _rand(gen, rows, 1)) + 0.3 * _randn(gen, rows, 1))
    s["weight"] = (1 + 0.2 * _randn(gen, width)).to(pdtype)
    s["bias"] = (0.1 * _randn(gen, width)).to(pdtype)
    s["y"] = _padded(rows, width, case["pad"], dtype)
    if case["train"]:
        s["mean"], s["rstd"] = torch.empty((2, rows), device=DEVICE).unbind(0)
        s["dy"] = _padded(rows, width, case["pad"], dtype)
        s["dy"].copy_(_randn(gen, rows, width) * 0.1)
        s["dx"] = _padded(rows, width, case["pad"], dtype)
        s["dweight"], s["dbias"] = torch.empty_like(s["weight"]), torch.empty_like(s["bias"])
    return s


def _prepare_distill(case, gen):
    rows, vocab, top, dtype = case["rows"], case["vocab"], case["top"], DTYPES[case["dtype"]]
    s = {"case": case, "temperature": case["temperature"]}
    logits = torch.empty((rows, vocab), dtype=dtype, device=DEVICE)
    top_logits = torch.empty((rows, top), dtype=dtype, device=DEVICE)
    top_codes = torch.empty((rows, top), dtype=torch.int32, device=DEVICE)
    teacher_lse = torch.empty(rows, device=DEVICE)
    step = max(1, (1 << 26) // vocab)
    for a in range(0, rows, step):
        b = min(rows, a + step)
        z = _randn(gen, b - a, vocab) * 2.5
        teacher = 0.7 * z + 2.0 * _randn(gen, b - a, vocab)
        if case["mask_code"]:  # a code that is never allowed, as a mask of the type's lowest value leaves it
            z[:, -1] = torch.finfo(dtype).min
            teacher[:, -1] = -math.inf
        logits[a:b] = z.to(dtype)
        v, i = torch.topk(teacher, top, dim=1)
        top_logits[a:b] = v.to(dtype)
        top_codes[a:b] = i.to(torch.int32)
        teacher_lse[a:b] = torch.logsumexp(teacher / case["temperature"], 1)
    weights = 0.8 ** torch.randint(0, 8, (rows,), generator=gen, device=DEVICE).float()
    padding = torch.randperm(rows, generator=gen, device=DEVICE)[: round(case["masked"] * rows)]
    weights[padding] = 0.0
    if case["ragged"]:  # lists that were cut by probability: their ends are empty
        length = torch.randint(1, top + 1, (rows, 1), generator=gen, device=DEVICE)
        top_codes[torch.arange(top, device=DEVICE)[None] >= length] = -1
    s.update(logits=logits, top_logits=top_logits, top_codes=top_codes, weights=weights,
             teacher_lse=teacher_lse if case["tail"] else None)
    s["loss"], s["dlogits"] = torch.empty(rows, device=DEVICE), torch.empty_like(logits)
    s["lse"] = torch.empty((rows, 2), device=DEVICE)
    # 16-bit floats with few exponents get their gradients through a loss scale, as a training step gives it
    scale = 1024.0 if dtype == torch.float16 else 1.0
    s["grad_loss"] = torch.full((rows,), scale, device=DEVICE) if case["passes"] == 2 else None
    if case["passes"] == 1:
        weights.mul_(scale)
    return s


def _prepare_beam(case, gen):
    g, b, v, n = case["groups"], case["beams"], case["vocab"], case["select"]
    s = {"case": case}
    if case["raw"]:
        # what a search over quantiser stages adds to minus the residual's squared norm: 2 r.z - |z|^2
        s["logits"] = _randn(gen, g, b, v) * 8.0 - 40.0
    else:
        # logits as a 16-bit head leaves them
        s["logits"] = (_randn(gen, g, b, v) * 2.5).to(torch.bfloat16).to(DTYPES[case["dtype"]])
    finished = torch.zeros((g, b), dtype=torch.bool, device=DEVICE)
    done = round(case["finished"] * b)
    if done:
        finished.scatter_(1, torch.argsort(_rand(gen, g, b), 1)[:, :done], True)
    s["finished"], s["end_code"] = finished, v - 1
    s["scores"] = _beam_scores(case, gen, s["logits"], finished, s["end_code"])
    s["out_scores"] = torch.empty((g, n), device=DEVICE)
    s["parents"] = torch.empty((g, n), dtype=torch.int32, device=DEVICE)
    s["codes"] = torch.empty((g, n), dtype=torch.int32, device=DEVICE)
    s["out_finished"] = torch.empty((g, n), dtype=torch.bool, device=DEVICE)
    shape = (case["layers"], g, b, case["length"], case["width"])
    s["state"] = torch.empty(shape, dtype=DTYPES[case["state"]], device=DEVICE)
    s["state"].normal_(generator=gen)
    s["out_state"] = torch.empty((shape[0], g, n) + shape[3:], dtype=s["state"].dtype, device=DEVICE)
    return s


def _beam_scores(case, gen, logits, finished, end_code):
    """Scores of the beams so far.  Drawn again for a group in which two of the
    best candidates lie nearer to one another than 32 bits tell apart."""
    g, b, n = case["groups"], case["beams"], case["select"]

    def fresh():
        scores = -8.0 - 12.0 * _rand(gen, g, b).sort(1).values
        if case["first"]:
            scores[:, 1:] = -math.inf
        return scores

    scores = fresh()
    if case["raw"]:
        return scores
    k = min(n + 1, case["vocab"])
    best = torch.empty((g, b, k), dtype=torch.float64, device=DEVICE)
    step = max(1, (1 << 24) // (b * case["vocab"]))
    for a in range(0, g, step):
        z = logits[a:a + step].double()
        best[a:a + step] = torch.topk(z, k, dim=2).values - torch.logsumexp(z, 2, keepdim=True)
    beam = torch.arange(b, device=DEVICE).repeat_interleave(k)
    for _ in range(60):
        total = scores.double()[:, :, None] + best
        total = torch.where(finished[:, :, None], -math.inf, total)
        total[:, :, 0] = torch.where(finished, scores.double(), total[:, :, 0])
        value, at = total.reshape(g, -1).sort(1, descending=True)
        value, at = value[:, :n + 1], beam[at[:, :n + 1]]
        gap = value[:, :-1] - value[:, 1:]
        gap = torch.where(torch.isnan(gap), math.inf, gap)
        near = (gap < 2e-4) & ~((at[:, :-1] == at[:, 1:]) & (gap == 0))
        bad = near.any(1)
        if not bool(bad.any()):
            break
        scores = torch.where(bad[:, None], fresh(), scores)
    return scores


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "distill": _own_distill, "beam": _own_beam}[op](state)
    return {"norm": _plain_norm, "distill": _plain_distill, "beam": _plain_beam}[op](state)


def _own_norm(s):
    import residual_vector_quantisation_gb300 as rq
    if not s["case"]["train"]:
        rq.rvq_layer_norm(s["x"], s["weight"], s["bias"], s["eps"], s["y"])
        return {"y": s["y"]}
    if "workspace" not in s:
        nbytes = rq.rvq_layer_norm_workspace_bytes(s["case"]["rows"], s["case"]["width"])
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device=DEVICE)
    rq.rvq_layer_norm(s["x"], s["weight"], s["bias"], s["eps"], s["y"], s["mean"], s["rstd"])
    rq.rvq_layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"],
                               s["workspace"])
    return {k: s[k] for k in ("y", "dx", "dweight", "dbias")}


def _own_distill(s):
    import residual_vector_quantisation_gb300 as rq
    teacher = (s["top_logits"], s["top_codes"], s["teacher_lse"])
    if s["grad_loss"] is None:
        rq.rvq_distill(s["logits"], *teacher, s["weights"], s["temperature"], s["loss"], dlogits=s["dlogits"])
    else:
        rq.rvq_distill(s["logits"], *teacher, s["weights"], s["temperature"], s["loss"], lse=s["lse"])
        rq.rvq_distill_backward(s["grad_loss"], s["logits"], *teacher, s["weights"], s["temperature"], s["lse"],
                                s["dlogits"])
    return {"loss": s["loss"], "dlogits": s["dlogits"]}


def _own_beam(s):
    import residual_vector_quantisation_gb300 as rq
    if "plan" not in s:
        c = s["case"]
        dims = rq.rvq_beam_dims(c["groups"], c["beams"], c["vocab"], c["select"],
                                rq.RVQ_BEAM_RAW if c["raw"] else rq.RVQ_BEAM_LOGITS, rq.DTYPES[s["logits"].dtype])
        workspace = torch.empty(rq.rvq_beam_workspace_bytes(dims), dtype=torch.uint8, device=DEVICE)
        s["plan"] = dims, workspace, rq.rvq_beam_states([(s["state"], s["out_state"])], layered=True)
    dims, workspace, states = s["plan"]
    rq.rvq_beam_select(dims, s["logits"], s["scores"], s["finished"], s["end_code"], s["out_scores"], s["parents"],
                       s["codes"], s["out_finished"], workspace)
    rq.rvq_beam_reorder(dims, s["parents"], states)
    return {"scores": s["out_scores"], "parents": s["parents"], "codes": s["codes"], "finished": s["out_finished"],
            "state": s["out_state"]}


def _plain_norm(s):
    x, weight, bias = s["x"].float(), s["weight"].float(), s["bias"].float()
    centred = x - x.mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt((centred * centred).mean(1, keepdim=True) + s["eps"])
    hat = centred * rstd
    y = (hat * weight + bias).to(s["x"].dtype)
    if not s["case"]["train"]:
        return {"y": y}
    dy = s["dy"].float()
    g = dy * weight
    dx = rstd * (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True))
    return {"y": y, "dx": dx.to(s["x"].dtype),
            "dweight": (dy * hat).sum(0).to(s["weight"].dtype), "dbias": dy.sum(0).to(s["bias"].dtype)}


def _plain_distill(s):
    scale = 1.0 / s["temperature"]
    z, t = s["logits"].float() * scale, s["top_logits"].float() * scale
    entry = s["top_codes"] >= 0
    codes = torch.where(entry, s["top_codes"], s["top_codes"][:, :1]).long()  # every list has a first entry
    most = z.amax(1, keepdim=True)
    e = torch.exp(z - most)
    total = e.sum(1, keepdim=True)
    lse = most + torch.log(total)
    t = torch.where(entry, t, -math.inf)
    if s["teacher_lse"] is None:
        high = t.amax(1, keepdim=True)
        teacher_lse = high + torch.log(torch.exp(t - high).sum(1, keepdim=True))
    else:
        teacher_lse = s["teacher_lse"][:, None]
    log_q = t - teacher_lse
    q = torch.exp(log_q)
    log_p = z.gather(1, codes) - lse
    loss = torch.where(entry & (q > 0), q * (log_q - log_p), 0.0).sum(1)
    if s["teacher_lse"] is None:
        grad = e / total
    else:
        rest = e.scatter(1, codes, 0.0)
        rest_sum = rest.sum(1, keepdim=True)
        q_rest = 1.0 - q.sum(1, keepdim=True)
        q_rest = torch.where(q_rest > TAIL_FLOOR, q_rest, 0.0)
        p_rest = rest_sum / total
        loss = loss + torch.where(q_rest > 0, q_rest * (torch.log(q_rest) - torch.log(p_rest)), 0.0)[:, 0]
        grad = rest * torch.where(rest_sum > 0, (p_rest - q_rest) / rest_sum, 0.0)
    at = torch.exp(log_p) - q
    grad.scatter_(1, codes, torch.where(entry, at, at[:, :1]))
    weight = s["weights"]
    scale = weight * scale if s["grad_loss"] is None else weight * s["grad_loss"] * scale
    live = weight != 0
    dlogits = torch.where(live[:, None], grad * scale[:, None], 0.0).to(s["logits"].dtype)
    return {"loss": torch.where(live, loss * weight, 0.0), "dlogits": dlogits}


def _plain_beam(s):
    c = s["case"]
    g, b, v, n = c["groups"], c["beams"], c["vocab"], c["select"]
    x, scores = s["logits"].float(), s["scores"][:, :, None]
    if not c["raw"]:
        most = x.amax(2, keepdim=True)
        x = x - (most + torch.log(torch.exp(x - most).sum(2, keepdim=True)))
    total = scores + x
    code = torch.arange(v, device=x.device)
    only = torch.where(code == s["end_code"], scores, -math.inf)
    total = torch.where(s["finished"][:, :, None], only, total).reshape(g, b * v) + 0.0
    # one whole number a candidate: its score's order, then the lowest index
    bits = total.view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    lowest = -(1 << 62)
    order = torch.where(torch.isnan(total) | (total == -math.inf), lowest, order * (1 << 27) - torch.arange(b * v, device=x.device))
    if b * v < n:
        order = torch.cat([order, order.new_full((g, n - b * v), lowest)], 1)
        total = torch.cat([total, total.new_full((g, n - b * v), -math.inf)], 1)
    value, at = torch.topk(order, n, dim=1)
    there = value != lowest
    parents = torch.where(there, at // v, -1)
    codes = torch.where(there, at % v, -1)
    chosen = torch.where(there, total.gather(1, at), -math.inf)
    held = parents.clamp(min=0)
    finished = torch.where(there, s["finished"].gather(1, held) | (codes == s["end_code"]), True)
    state = s["state"][:, torch.arange(g, device=x.device)[:, None], held]
    state = torch.where(there[None, :, :, None, None], state, 0)
    return {"scores": chosen, "parents": parents.to(torch.int32), "codes": codes.to(torch.int32), "finished": finished,
            "state": state}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "distill": _exact_distill, "beam": _exact_beam}[case["op"]](s)


def _exact_norm(s):
    x, w = s["x"].double(), s["weight"].double()
    var, mu = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
    sd = (var + s["eps"]).sqrt()
    y = (x - mu) / sd * w + s["bias"].double()
    if not s["case"]["train"]:
        return {"y": y}
    dy = s["dy"].double()
    u = (x - mu) / sd
    dweight, dbias = torch.einsum("rd,rd->d", dy, u), dy.sum(0)
    d = x.shape[1]
    a = dy @ w / d
    c = torch.einsum("rd,rd,d->r", dy, u, w) / d
    dx = (dy * w - a[:, None] - u * c[:, None]) / sd
    return {"y": y, "dx": dx, "dweight": dweight, "dbias": dbias}


def _exact_distill(s):
    rows, vocab = s["logits"].shape
    temperature = s["temperature"]
    loss = torch.zeros(rows, dtype=torch.float64, device=DEVICE)
    dlogits = torch.zeros((rows, vocab), dtype=torch.float64, device=DEVICE)
    step = max(1, (1 << 25) // vocab)
    for a in range(0, rows, step):
        b = min(rows, a + step)
        n = b - a
        weight = s["weights"][a:b].double()
        log_p = torch.log_softmax(s["logits"][a:b].double() / temperature, 1)
        codes = s["top_codes"][a:b].long()
        row, col = (codes >= 0).nonzero(as_tuple=True)
        code = codes[row, col]
        t = torch.full((n, codes.shape[1]), -math.inf, dtype=torch.float64, device=DEVICE)
        t[row, col] = s["top_logits"][a:b].double()[row, col] / temperature
        given = s["teacher_lse"]
        log_q = t - (torch.logsumexp(t, 1) if given is None else given[a:b].double())[:, None]
        lq, lp = log_q[row, col], log_p[row, code]
        q = lq.exp()
        some = q > 0
        row_loss = torch.zeros(n, dtype=torch.float64, device=DEVICE)
        row_loss.index_add_(0, row[some], q[some] * (lq[some] - lp[some]))
        grad = log_p.exp()
        if given is not None:
            others = log_p.clone()
            others[row, code] = -math.inf
            log_rest = torch.logsumexp(others, 1)
            q_rest = 1.0 - log_q.exp().sum(1)
            q_rest = torch.where(q_rest > TAIL_FLOOR, q_rest, 0.0)
            row_loss += torch.where(q_rest > 0, q_rest * (q_rest.log() - log_rest), 0.0)
            grad -= q_rest[:, None] * (others - log_rest[:, None]).exp()
        grad.index_put_((row, code), lp.exp() - q)
        up = weight / temperature
        if s["grad_loss"] is not None:
            up = up * s["grad_loss"][a:b].double()
        loss[a:b] = torch.where(weight == 0, 0.0, weight * row_loss)
        dlogits[a:b] = torch.where(weight[:, None] == 0, 0.0, up[:, None] * grad)
    return {"loss": loss, "dlogits": dlogits}


def _exact_beam(s):
    c = s["case"]
    g, b, v, n = c["groups"], c["beams"], c["vocab"], c["select"]
    scores = torch.full((g, n), -math.inf, dtype=torch.float64, device=DEVICE)
    step = max(1, (1 << 24) // (b * v))
    for a in range(0, g, step):
        x = s["logits"][a:a + step].double()
        if not c["raw"]:
            x = torch.log_softmax(x, 2)
        held = s["scores"][a:a + step].double()
        x = x + held[:, :, None]
        done = s["finished"][a:a + step]
        x[done] = -math.inf
        x[..., s["end_code"]] = torch.where(done, held, x[..., s["end_code"]])
        best = torch.sort(x.reshape(len(x), -1), 1, descending=True).values[:, :n]
        scores[a:a + step, :best.shape[1]] = best
    return {"scores": scores, "parents": None, "codes": None, "finished": None, "state": None}
