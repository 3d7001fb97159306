"""Cases of more of the code predictor's operators: log probabilities of given codes (with entropy and the top
alternatives), root-mean-square norm (with the residual's addition, dropout and an output in 8 bits), and dropout.

`run` computes a case in its plain form (elementary torch operations in 32
bits), or, where `own` is true, with the framework's kernels.  `exact` states
the same operators in 64 bits, apart from the plain form.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
DEVICE = "cuda"
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
E4M3_MOST = 448.0
LEAST_SCALE = 2.0 ** -126


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def _log_probs(name, rows, vocab, dtype, top=0, train=False, entropy=True, temperature=1.0, padding=0.0,
               mask_code=False, pad=0):
    return {"name": name, "op": "log_probs", "rows": rows, "vocab": vocab, "dtype": dtype, "top": top, "train": train,
            "entropy": entropy, "temperature": temperature, "padding": padding, "mask_code": mask_code, "pad": pad}


def _rms(name, rows, width, dtype, train=False, residual=True, dropout=0.0, params="f32", pad=0, block=-1, power=False):
    # block: -1: no output in 8 bits, 0: a scale a row, else a scale for as many columns
    return {"name": name, "op": "rms", "rows": rows, "width": width, "dtype": dtype, "train": train,
            "residual": residual, "dropout": dropout, "params": params, "pad": pad, "block": block, "power": power}


def _dropout(name, rows, width, dtype, p, train=False, residual=False, pad=0):
    return {"name": name, "op": "dropout", "rows": rows, "width": width, "dtype": dtype, "p": p, "train": train,
            "residual": residual, "pad": pad}


def listed():
    return [
        # one frame of 8 heads as it is decoded: how sure each head is, and its runners-up; nothing but latency
        _log_probs("log_probs_one_frame", 8, 1025, "bf16", top=4, mask_code=True),
        # a training batch of 8 heads with the mask code (never allowed) last: log probability and entropy, and the
        # gradient of both; padding frames have no code
        _log_probs("log_probs_8_heads", 96000, 1025, "bf16", train=True, padding=0.1, mask_code=True),
        # a teacher's lists for distillation: 32 heads of 1024 codes in full precision, the 16 best of each
        _log_probs("log_probs_teacher", 384000, 1024, "f32", top=16, temperature=1.5),
        # the longest codebook that the quantiser takes, flattened into one vocabulary, in training
        _log_probs("log_probs_65536", 4096, 65536, "bf16", train=True, entropy=False),
        # a few positions of that vocabulary as they are answered: few rows, long ones
        _log_probs("log_probs_few_long", 6, 65536, "f16", top=32, temperature=0.8),
        # one new frame before a projection in 8 bits
        _rms("rms_one_frame", 1, 1024, "bf16", block=32, power=True),
        # a training batch of 16 utterances of 750 frames at the 32-stage codec's width, in full precision
        _rms("rms_train_768", 12000, 768, "f32", train=True),
        # the benchmark's batch of 256 utterances: the sublayer's output dropped and added, normalised; and back
        _rms("rms_train_192k", 192000, 1024, "bf16", train=True, dropout=0.1),
        # rows of an odd width inside wider ones, a scale a row
        _rms("rms_8bit_odd", 20011, 1025, "f16", pad=6, block=0),
        # a serving batch before a projection in 8 bits, a scale for 128 columns
        _rms("rms_8bit_4096", 32768, 4096, "bf16", block=128),
        # one utterance's frames
        _dropout("dropout_one_utterance", 750, 1024, "bf16", 0.1),
        # the benchmark's batch: a sublayer's output dropped and added, and the gradient
        _dropout("dropout_train_192k", 192000, 1024, "bf16", 0.1, train=True, residual=True),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["log_probs", "rms", "dropout"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "log_probs":
        vocab = _log_int(rng, 100, 131072)
        if rng.random() < 0.5:
            vocab = max(64, vocab // 64 * 64)
        rows = _log_int(rng, 1, max(2, 130_000_000 // vocab))
        train = rng.random() < 0.5
        case = _log_probs("", rows, vocab, dtype, 0 if train else rng.choice([0, 1, 3, 8, 20, 64]), train,
                          rng.random() < 0.7, rng.choice([0.7, 1.0, 2.0]), rng.choice([0.0, 0.2]), rng.random() < 0.3,
                          rng.choice([0, 0, 8, 3]))
    elif op == "rms":
        width = _log_int(rng, 40, 16384)
        if rng.random() < 0.6:
            width = max(16, width // 16 * 16)
        rows = _log_int(rng, 1, max(2, 90_000_000 // width))
        train = rng.random() < 0.6
        case = _rms("", rows, width, dtype, train, rng.random() < 0.8, rng.choice([0.0, 0.1, 0.5]) if train else 0.0,
                    rng.choice(["f32", "same"]), rng.choice([0, 0, 8, 3]),
                    -1 if train else rng.choice([-1, 0, 0, 32, 64, 128]), rng.random() < 0.5)
    else:
        width = _log_int(rng, 40, 16384)
        if rng.random() < 0.6:
            width = max(16, width // 16 * 16)
        rows = _log_int(rng, 1, max(2, 90_000_000 // width))
        case = _dropout("", rows, width, dtype, rng.choice([0.05, 0.1, 0.3, 0.5]), rng.random() < 0.5,
                        rng.random() < 0.5, rng.choice([0, 0, 8, 3]))
    del case["name"]
    return case


def _blocks(case):
    return 1 if case["block"] == 0 else -(-case["width"] // case["block"])


def work(case):
    e = SIZES[case["dtype"]]
    if case["op"] == "log_probs":
        n, rows = case["rows"] * case["vocab"], case["rows"]
        per = 4 + 4 + (4 if case["entropy"] else 0) + 8 * case["top"]
        if not case["train"]:
            return {"bytes": n * e + rows * per, "flops": 6 * n}
        # forward: logits in; backward, after the caller's loss: logits in again, their gradient out
        return {"bytes": 3 * n * e + rows * (per + 16), "flops": 14 * n}
    n = case["rows"] * case["width"]
    if case["op"] == "rms":
        p = case["width"] * (4 if case["params"] == "f32" else e)
        most = case["residual"] or case["dropout"] > 0   # the sum is an output of its own
        read, wrote = n * e * (2 if case["residual"] else 1) + p, n * e if most else 0
        if case["block"] < 0:
            wrote += n * e
        else:
            wrote += n + case["rows"] * _blocks(case) * (1 if case["power"] else 4)
        if not case["train"]:
            return {"bytes": read + wrote, "flops": 6 * n}
        # backward: dy, the sum and the gradient that reaches the sum in; one or two gradients out
        back = n * e * ((3 if most else 2) + (1 if case["dropout"] == 0 or not case["residual"] else 2))
        return {"bytes": read + wrote + back + 2 * p + 8 * case["rows"], "flops": 20 * n}
    passes = (3 if case["residual"] else 2) + (2 if case["train"] else 0)
    return {"bytes": passes * n * e, "flops": 4 * n * (2 if case["train"] else 1)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed * 7919 + 29)
    return {"log_probs": _prepare_log_probs, "rms": _prepare_rms, "dropout": _prepare_dropout}[case["op"]](case, gen, seed)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEVICE)


def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device=DEVICE)


def _padded(rows, width, pad, dtype):
    return torch.empty((rows, width + pad), dtype=dtype, device=DEVICE)[:, :width]


def _prepare_log_probs(case, gen, seed):
    rows, vocab, dtype = case["rows"], case["vocab"], DTYPES[case["dtype"]]
    s = {"case": case, "temperature": case["temperature"]}
    logits = _padded(rows, vocab, case["pad"], dtype)
    codes = torch.empty(rows, dtype=torch.int32, device=DEVICE)
    step = max(1, (1 << 26) // vocab)
    for a in range(0, rows, step):
        b = min(rows, a + step)
        z = _randn(gen, b - a, vocab) * 2.5
        if case["mask_code"]:  # a code that is never allowed, as a mask of the type's lowest value leaves it
            z[:, -1] = torch.finfo(dtype).min
        logits[a:b] = z.to(dtype)
        # codes as a model draws them: good ones, if rarely the best
        codes[a:b] = (z + 2.0 * _randn(gen, 1, vocab)).argmax(1).to(torch.int32)
    padding = torch.randperm(rows, generator=gen, device=DEVICE)[: round(case["padding"] * rows)]
    codes[padding] = -1
    s.update(logits=logits, codes=codes)
    s["log_probs"], s["lse"] = torch.empty(rows, device=DEVICE), torch.empty(rows, device=DEVICE)
    s["entropy"] = torch.empty(rows, device=DEVICE) if case["entropy"] else None
    s["top_log_probs"] = s["top_codes"] = s["stats"] = None
    if case["top"]:
        s["top_log_probs"] = torch.empty((rows, case["top"]), device=DEVICE)
        s["top_codes"] = torch.empty((rows, case["top"]), dtype=torch.int32, device=DEVICE)
    if case["train"]:
        s["stats"] = torch.empty((rows, 2), device=DEVICE)
        # advantages of a policy step, a weight of the entropy, and of the log sum's square; 16-bit floats with few
        # exponents get them through a loss scale
        scale = 1024.0 if dtype == torch.float16 else 1.0
        s["grad_log_probs"] = _randn(gen, rows) * scale
        s["grad_log_probs"][padding] = 0.0
        s["grad_entropy"] = torch.full((rows,), -0.05 * scale, device=DEVICE) if case["entropy"] else None
        s["grad_lse"] = 0.01 * _randn(gen, rows) * scale
        if case["entropy"]:
            s["grad_entropy"][padding] = 0.0
        s["grad_lse"][padding] = 0.0
        s["dlogits"] = _padded(rows, vocab, case["pad"], dtype)
    return s


def _random_stream(gen, seed):
    """What a training program has for its dropout: a seed, the number of the call's place in the model, and a step
    counter on the GPU (a captured step reads it anew)."""
    return {"seed": (seed * 0x9E3779B97F4A7C15 + 0x1234567) % (1 << 64), "offset": 7 + seed % 1000,
            "step": torch.randint(0, 1 << 20, (1,), generator=gen, device=DEVICE)}


def _prepare_rms(case, gen, seed):
    rows, width, dtype, pad = case["rows"], case["width"], DTYPES[case["dtype"]], case["pad"]
    pdtype = torch.float32 if case["params"] == "f32" else dtype
    s = {"case": case, "eps": 1e-6}
    s["x"] = _padded(rows, width, pad, dtype)
    s["x"].copy_(_randn(gen, rows, width) * (0.5 + _rand(gen, rows, 1)))
    s["residual"] = s["total"] = None
    if case["residual"]:
        s["residual"] = _padded(rows, width, pad, dtype)
        s["residual"].copy_(_randn(gen, rows, width) * 2.0 + 0.3 * _randn(gen, rows, 1))
    if case["residual"] or case["dropout"] > 0:
        s["total"] = _padded(rows, width, pad, dtype)
    s["weight"] = (1 + 0.2 * _randn(gen, width)).to(pdtype)
    s["random"] = _random_stream(gen, seed) if case["dropout"] > 0 else None
    s["y"] = s["q"] = s["scales"] = None
    if case["block"] >= 0:
        s["q"] = torch.empty((rows, width), dtype=E4M3, device=DEVICE)
        s["scales"] = torch.empty((rows, _blocks(case)), dtype=E8M0 if case["power"] else torch.float32, device=DEVICE)
    else:
        s["y"] = _padded(rows, width, pad, dtype)
    if case["train"]:
        s["rstd"] = torch.empty(rows, device=DEVICE)
        s["dy"] = _padded(rows, width, pad, dtype)
        s["dy"].copy_(_randn(gen, rows, width) * 0.1)
        s["dtotal"] = None
        if s["total"] is not None:
            s["dtotal"] = _padded(rows, width, pad, dtype)
            s["dtotal"].copy_(_randn(gen, rows, width) * 0.1)
        s["dresidual"] = _padded(rows, width, pad, dtype) if case["residual"] or case["dropout"] == 0 else None
        s["dx"] = _padded(rows, width, pad, dtype) if case["dropout"] > 0 else None
        s["dweight"] = torch.empty_like(s["weight"])
    return s


def _prepare_dropout(case, gen, seed):
    rows, width, dtype, pad = case["rows"], case["width"], DTYPES[case["dtype"]], case["pad"]
    s = {"case": case, "random": _random_stream(gen, seed)}
    s["x"], s["y"] = _padded(rows, width, pad, dtype), _padded(rows, width, pad, dtype)
    s["x"].copy_(_randn(gen, rows, width))
    s["residual"] = None
    if case["residual"]:
        s["residual"] = _padded(rows, width, pad, dtype)
        s["residual"].copy_(_randn(gen, rows, width) * 2.0)
    if case["train"]:
        s["dy"], s["dx"] = _padded(rows, width, pad, dtype), _padded(rows, width, pad, dtype)
        s["dy"].copy_(_randn(gen, rows, width) * 0.1)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"log_probs": _own_log_probs, "rms": _own_rms, "dropout": _own_dropout}[op](state)
    return {"log_probs": _plain_log_probs, "rms": _plain_rms, "dropout": _plain_dropout}[op](state)


def _given(**outputs):
    return {k: v for k, v in outputs.items() if v is not None}


def _own_log_probs(s):
    import residual_vector_quantisation_gb300 as rq
    rq.rvq_log_probs(s["logits"], s["codes"], s["temperature"], s["log_probs"], s["entropy"], s["lse"], s["stats"],
                     s["top_log_probs"], s["top_codes"])
    if s["case"]["train"]:
        rq.rvq_log_probs_backward(s["grad_log_probs"], s["grad_entropy"], s["grad_lse"], s["logits"], s["codes"],
                                  s["temperature"], s["stats"], s["entropy"], s["dlogits"])
    return _given(log_probs=s["log_probs"], entropy=s["entropy"], lse=s["lse"], top_log_probs=s["top_log_probs"],
                  top_codes=s["top_codes"], dlogits=s.get("dlogits"))


def _own_random(s, p):
    import residual_vector_quantisation_gb300 as rq
    r = s["random"]
    return rq.rvq_dropout_mask(p, r["seed"], r["offset"], r["step"])


def _own_rms(s):
    import residual_vector_quantisation_gb300 as rq
    c = s["case"]
    if "mask" not in s:
        s["mask"] = _own_random(s, c["dropout"]) if c["dropout"] > 0 else None
        if c["train"]:
            nbytes = rq.rvq_rms_norm_workspace_bytes(c["rows"], c["width"])
            s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device=DEVICE)
    rq.rvq_rms_norm(s["x"], s["weight"], s["eps"], s["y"], s.get("rstd"), residual=s["residual"], mask=s["mask"],
                    total=s["total"], q=s["q"], scales=s["scales"], block=max(0, c["block"]))
    if c["train"]:
        total = s["x"] if s["total"] is None else s["total"]
        rq.rvq_rms_norm_backward(s["dy"], total, s["weight"], s["rstd"], s["dresidual"], s["dweight"], s["workspace"],
                                 dtotal=s["dtotal"], mask=s["mask"], dx=s["dx"])
    return _given(y=s["y"], total=s["total"], q=s["q"], scales=s["scales"], dresidual=s.get("dresidual"),
                  dx=s.get("dx"), dweight=s.get("dweight"))


def _own_dropout(s):
    import residual_vector_quantisation_gb300 as rq
    if "mask" not in s:
        s["mask"] = _own_random(s, s["case"]["p"])
    rq.rvq_dropout(s["x"], s["mask"], s["y"], s["residual"])
    if not s["case"]["train"]:
        return {"y": s["y"]}
    rq.rvq_dropout(s["dy"], s["mask"], s["dx"])
    return {"y": s["y"], "dx": s["dx"]}


def _plain_log_probs(s):
    c = s["case"]
    inv = 1.0 / s["temperature"]
    x = s["logits"].float()
    most = x.amax(1, keepdim=True)
    d = (x - most) * inv
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    there = s["codes"] >= 0
    at = torch.where(there, s["codes"], 0).long()[:, None]
    log_probs = torch.where(there, (d.gather(1, at) - log_total)[:, 0], 0.0)
    out = {"log_probs": log_probs, "lse": (most * inv + log_total)[:, 0]}
    if c["entropy"]:
        out["entropy"] = (log_total - (torch.where(e > 0, e * d, 0.0)).sum(1, keepdim=True) / total)[:, 0]
    if c["top"]:
        # one whole number a code: its logit's order, then the lowest code
        bits = (x + 0.0).view(torch.int32)
        order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
        order = order * (1 << 24) - torch.arange(c["vocab"], device=x.device)
        out["top_codes"] = torch.topk(order, c["top"], dim=1).indices.to(torch.int32)
        out["top_log_probs"] = d.gather(1, out["top_codes"].long()) - log_total
    if c["train"]:
        g = torch.where(there, s["grad_log_probs"], 0.0)[:, None]
        p = e / total
        factor = s["grad_lse"][:, None] - g
        if c["entropy"]:
            factor = factor - s["grad_entropy"][:, None] * torch.where(e > 0, d - log_total + out["entropy"][:, None], 0.0)
        grad = p * factor
        grad.scatter_add_(1, at, g)
        out["dlogits"] = (grad * inv).to(s["logits"].dtype)
    return out


def _philox_bits(seed, offset, step, first, groups, device):
    """16 bits for each of 8 * groups elements (from element 8 * first on): Philox4x32-10 (Salmon et al., 2011) of the
    counters (group, offset + step * 2^32) under the key `seed`; products of 32-bit words in 64."""
    low = 0xFFFFFFFF
    g = torch.arange(first, first + groups, device=device)
    upper = step * (1 << 32) + (offset - (1 << 64) if offset >= 1 << 63 else offset)
    a, b = g & low, g >> 32
    c, d = (upper & low).expand_as(a), ((upper >> 32) & low).expand_as(a)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        p, q = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = ((q >> 32) & low) ^ b ^ k0, q & low, ((p >> 32) & low) ^ d ^ k1, p & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([a, b, c, d], 1)
    return torch.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)


def _plain_keep(s, p):
    """What stays of the elements, and the factor of what does."""
    c, r = s["case"], s["random"]
    n = c["rows"] * c["width"]
    drop = math.floor(p * 65536 + 0.5)
    bits = _philox_bits(r["seed"], r["offset"], r["step"], 0, -(-n // 8), s["x"].device)[:n]
    return (bits >= drop).view(c["rows"], c["width"]), 65536.0 / (65536 - drop)


def _plain_rms(s):
    c = s["case"]
    dtype = s["x"].dtype
    h = s["x"].float()
    if c["dropout"] > 0:
        keep, factor = _plain_keep(s, c["dropout"])
        h = torch.where(keep, h * factor, 0.0)
    if s["residual"] is not None:
        h = h + s["residual"].float()
    out = {}
    if s["total"] is not None:  # the sum goes on in the inputs' type, and that is what is normalised
        out["total"] = h.to(dtype)
        h = out["total"].float()
    weight = s["weight"].float()
    rstd = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + s["eps"])
    hat = h * rstd
    y = hat * weight
    if c["block"] >= 0:
        rows, width = y.shape
        blocks = _blocks(c)
        size = c["block"] or width
        wide = torch.nn.functional.pad(y, (0, blocks * size - width)).view(rows, blocks, size)
        scale = torch.clamp(wide.abs().amax(2) / E4M3_MOST, min=LEAST_SCALE)
        if c["power"]:
            fraction, exponent = torch.frexp(scale)  # fraction in [0.5, 1)
            scale = torch.ldexp(torch.ones_like(scale), exponent - (fraction == 0.5).int())
        q = torch.clamp(wide / scale[:, :, None], -E4M3_MOST, E4M3_MOST)
        out["q"] = q.view(rows, -1)[:, :width].to(E4M3)
        out["scales"] = scale.to(E8M0) if c["power"] else scale
    else:
        out["y"] = y.to(dtype)
    if c["train"]:
        dy = s["dy"].float()
        g = dy * weight
        dh = rstd * (g - hat * (g * hat).mean(1, keepdim=True))
        if s["dtotal"] is not None:
            dh = dh + s["dtotal"].float()
        if s["dresidual"] is not None:
            out["dresidual"] = dh.to(dtype)
        if c["dropout"] > 0:
            out["dx"] = torch.where(keep, dh * factor, 0.0).to(dtype)
        out["dweight"] = (dy * hat).sum(0).to(s["weight"].dtype)
    return out


def _plain_dropout(s):
    keep, factor = _plain_keep(s, s["case"]["p"])
    y = torch.where(keep, s["x"].float() * factor, 0.0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y.to(s["x"].dtype)}
    if s["case"]["train"]:
        out["dx"] = torch.where(keep, s["dy"].float() * factor, 0.0).to(s["x"].dtype)
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"log_probs": _exact_log_probs, "rms": _exact_rms, "dropout": _exact_dropout}[case["op"]](s)


def _exact_log_probs(s):
    c = s["case"]
    rows, vocab, temperature = c["rows"], c["vocab"], s["temperature"]
    out = {"log_probs": torch.zeros(rows, dtype=torch.float64, device=DEVICE),
           "lse": torch.zeros(rows, dtype=torch.float64, device=DEVICE)}
    if c["entropy"]:
        out["entropy"] = torch.zeros_like(out["lse"])
    if c["top"]:
        out["top_codes"] = None
        out["top_log_probs"] = torch.zeros((rows, c["top"]), dtype=torch.float64, device=DEVICE)
    if c["train"]:
        out["dlogits"] = torch.zeros((rows, vocab), dtype=torch.float64, device=DEVICE)
    step = max(1, (1 << 25) // vocab)
    for a in range(0, rows, step):
        b = min(rows, a + step)
        z = s["logits"][a:b].double() / temperature
        out["lse"][a:b] = torch.logsumexp(z, 1)
        log_p = torch.log_softmax(z, 1)
        p = log_p.exp()
        row = torch.arange(b - a, device=DEVICE)
        codes = s["codes"][a:b].long()
        has = codes >= 0
        out["log_probs"][a:b][has] = log_p[row[has], codes[has]]
        entropy = torch.special.entr(p).sum(1)
        if c["entropy"]:
            out["entropy"][a:b] = entropy
        if c["top"]:
            out["top_log_probs"][a:b] = torch.sort(log_p, 1, descending=True).values[:, :c["top"]]
        if c["train"]:
            given = torch.zeros(b - a, dtype=torch.float64, device=DEVICE)
            given[has] = s["grad_log_probs"][a:b].double()[has]
            grad = p * (s["grad_lse"][a:b].double() - given)[:, None]
            grad[row[has], codes[has]] += given[has]
            if c["entropy"]:  # d H / d z_j = -p_j log p_j - p_j H
                grad += s["grad_entropy"][a:b].double()[:, None] * (torch.special.entr(p) - p * entropy[:, None])
            out["dlogits"][a:b] = grad / temperature
    return out


def _exact_keep(s, p):
    """The mask with numpy's unsigned words."""
    c, r = s["case"], s["random"]
    n = c["rows"] * c["width"]
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    upper = (r["offset"] + (int(r["step"].item()) << 32)) % (1 << 64)
    g = np.arange(-(-n // 8), dtype=np.uint64)
    x = [g & low, g >> half, np.full_like(g, upper & 0xFFFFFFFF), np.full_like(g, upper >> 32)]
    for i in range(10):
        k0 = np.uint64((r["seed"] + i * 0x9E3779B9) & 0xFFFFFFFF)
        k1 = np.uint64(((r["seed"] >> 32) + i * 0xBB67AE85) & 0xFFFFFFFF)
        m0, m1 = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(m1 >> half) ^ x[1] ^ k0, m1 & low, (m0 >> half) ^ x[3] ^ k1, m0 & low]
    bits = np.stack([w.astype("<u4") for w in x], 1).view("<u2").reshape(-1)[:n]
    drop = int(p * 65536 + 0.5)
    keep = torch.from_numpy(bits.astype(np.int32) >= drop).to(DEVICE).view(c["rows"], c["width"])
    return keep, 65536 / (65536 - drop)


def _exact_rms(s):
    c = s["case"]
    dtype = s["x"].dtype
    x = s["x"].double()
    if c["dropout"] > 0:
        keep, factor = _exact_keep(s, c["dropout"])
        x = torch.where(keep, x * factor, torch.zeros_like(x))
    if s["residual"] is not None:
        x = x + s["residual"].double()
    out = {}
    if s["total"] is not None:
        out["total"] = x
        # the sum as the next layer reads it (32-bit sums: those, rounded to the type, are what it holds)
        held = s["x"].float()
        if c["dropout"] > 0:
            held = torch.where(keep, held * factor, torch.zeros_like(held))
        if s["residual"] is not None:
            held = held + s["residual"].float()
        x = held.to(dtype).double()
    w = s["weight"].double()
    width = x.shape[1]
    rms = (torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / width + s["eps"]).sqrt()
    y = x / rms * w
    if c["block"] >= 0:
        size = c["block"] or width
        q, scales = torch.empty_like(y), []
        for a in range(0, width, size):
            part = y[:, a:a + size]
            scale = (part.abs().amax(1) / 448).clamp(min=2.0 ** -126)
            if c["power"]:
                scale = torch.exp2(torch.ceil(torch.log2(scale)))
            q[:, a:a + size] = part / scale[:, None]
            scales.append(scale)
        out.update(q=q, scales=torch.stack(scales, 1))
    else:
        out["y"] = y
    if c["train"]:
        dy = s["dy"].double()
        u = x / rms
        back = torch.einsum("rd,rd,d->r", dy, u, w)[:, None] / width
        dh = (dy * w - u * back) / rms
        if s["dtotal"] is not None:
            dh = dh + s["dtotal"].double()
        if s["dresidual"] is not None:
            out["dresidual"] = dh
        if c["dropout"] > 0:
            out["dx"] = torch.where(keep, dh * factor, torch.zeros_like(dh))
        out["dweight"] = torch.einsum("rd,rd->d", dy, u)
    return out


def _exact_dropout(s):
    keep, factor = _exact_keep(s, s["case"]["p"])
    x = s["x"].double()
    y = torch.where(keep, x * factor, torch.zeros_like(x))
    out = {"y": y if s["residual"] is None else y + s["residual"].double()}
    if s["case"]["train"]:
        dy = s["dy"].double()
        out["dx"] = torch.where(keep, dy * factor, torch.zeros_like(dy))
    return out
