"""The code predictor's operators where calls can go wrong, as far as that shows
without a GPU."""

import contextlib
import ctypes
import itertools
import os
import random
import re
import subprocess

import pytest
import torch

import residual_vector_quantisation_gb300 as rq
from residual_vector_quantisation_gb300 import build as rqb, predictor

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "residual_vector_quantisation_gb300",
                    "csrc")


@pytest.fixture(scope="module", autouse=True)
def lib():
    rqb.build_library()
    return rq.load_library()


def kernels(name):
    """(name, parameters, body) of every __global__ function of a source file."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\(([^{]*)\)\s*{", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield m.group(1), m.group(2), text[m.end():at]


@pytest.mark.parametrize("name", ["rvq_norm.cu", "rvq_distill.cu", "rvq_beam.cu"])
def test_overlapping_kernels_take_no_read_only_pointers(name):
    """A kernel that starts while the one before it runs must not promise that what it reads is read-only for its
    whole life: `const ... __restrict__` on a pointer allows loads that are not coherent, and their reordering."""
    found = list(kernels(name))
    assert found
    for kernel, parameters, body in found:
        if "griddep_wait" in body:
            assert "__restrict__" not in parameters and "__ldg(" not in body, kernel


# ---------------------------------------------------------------------------
# the device of a call
# ---------------------------------------------------------------------------

class OnGpu:
    """A tensor that says it is on GPU `index`; its data are never looked at."""

    def __init__(self, index, *shape, dtype=torch.float32):
        self.t, self.index = torch.zeros(shape, dtype=dtype), index

    is_cuda = True
    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


class Stream:
    def __init__(self, index, handle):
        self.device_index, self.cuda_stream = index, handle


@pytest.fixture
def gpus(monkeypatch):
    """A library that records (entry point, current device, stream) of each call, and two GPUs that torch makes
    current; device 0 is."""
    calls, current = [], [0]

    class Library:
        def __getattr__(self, name):
            def call(*args):
                calls.append((name, current[0], args[-1]))
                return 0
            return call

    class Device:
        def __init__(self, index):
            self.index = index if isinstance(index, int) else index.index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    monkeypatch.setattr(rq, "load_library", lambda: Library())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda d=None: Stream(current[0] if d is None else torch.device(d).index,
                                              100 + (current[0] if d is None else torch.device(d).index)))
    return calls


F32, I32, U8 = torch.float32, torch.int32, torch.uint8
BEAM = rq.rvq_beam_dims(2, 3, 10, 3, 0, 0)


def operators(t):
    """Each entry point with tensors from t(*shape, dtype): {name: (call, the tensors it takes)}."""
    def with_tensors(call, *tensors):
        return call, list(tensors)

    rows, stats, w, ws = (lambda: t(4, 8)), (lambda: t(4)), (lambda: t(8)), (lambda: t(64, dtype=U8))
    top, codes = (lambda: t(4, 2)), (lambda: t(4, 2, dtype=I32))
    kept = lambda: t(2, 3, dtype=I32)  # noqa: E731
    return {
        "rvq_layer_norm": with_tensors(lambda x, w, b, y, m, r, **kw: rq.rvq_layer_norm(x, w, b, 1e-5, y, m, r, **kw),
                                       rows(), w(), w(), rows(), stats(), stats()),
        "rvq_layer_norm_backward": with_tensors(rq.rvq_layer_norm_backward, rows(), rows(), w(), stats(), stats(), rows(),
                                                w(), w(), ws()),
        "rvq_distill": with_tensors(lambda z, t, c, e, w, o, s, d, b, **kw: rq.rvq_distill(z, t, c, e, w, 1.0, o, s, d, b,
                                                                                          **kw),
                                    rows(), top(), codes(), stats(), stats(), stats(), t(4, 2), rows(),
                                    t(1, dtype=torch.int64)),
        "rvq_distill_backward": with_tensors(
            lambda g, z, t, c, e, w, s, d, **kw: rq.rvq_distill_backward(g, z, t, c, e, w, 1.0, s, d, **kw),
            stats(), rows(), top(), codes(), stats(), stats(), t(4, 2), rows()),
        "rvq_beam_select": with_tensors(
            lambda z, s, f, o, p, c, of, ws, **kw: rq.rvq_beam_select(BEAM, z, s, f, 1, o, p, c, of, ws, **kw),
            t(2, 3, 10), t(2, 3), t(2, 3, dtype=U8), t(2, 3), kept(), kept(), t(2, 3, dtype=U8), ws()),
        "rvq_beam_reorder": with_tensors(
            lambda p, a, b, **kw: rq.rvq_beam_reorder(BEAM, p, rq.rvq_beam_states([(a, b)]), **kw),
            kept(), t(2, 3, 4), t(2, 3, 4)),
    }


QUANTISER = rq.rvq_dims(8, 4, 16, 2, 0, 0, 0)


def quantiser(t):
    """The quantiser's own entry points, stated in the same way."""
    tables, scratch = (lambda: t(64, dtype=U8)), (lambda: t(64, dtype=U8))
    x, codes = (lambda: t(5, 8)), (lambda: t(5, 2, dtype=I32))
    return {
        "rvq_prepare": (lambda tab, a, b, c, d, e, **kw: rq.rvq_prepare(QUANTISER, a, b, c, d, e, tab, **kw),
                        [tables(), t(2, 4, 8), t(2, 16, 4), t(2, 8, 4), t(2, 4), t(2, 8)]),
        "rvq_encode": (lambda tab, a, c, s, **kw: rq.rvq_encode(QUANTISER, tab, a, 2, c, s, **kw),
                       [tables(), x(), codes(), scratch()]),
        "rvq_decode": (lambda tab, c, y, b, **kw: rq.rvq_decode(QUANTISER, tab, c, 2, y, b, **kw),
                       [tables(), codes(), x(), t(1, dtype=torch.int64)]),
        "rvq_reconstruct": (lambda tab, a, c, y, s, **kw: rq.rvq_reconstruct(QUANTISER, tab, a, 2, c, y, s, **kw),
                            [tables(), x(), codes(), x(), scratch()]),
        "rvq_encode_static": (lambda tab, a, c, **kw: rq.rvq_encode_static(QUANTISER, tab, a, 2, c, **kw),
                              [tables(), x(), codes()]),
        "rvq_read_status": (rq.rvq_read_status, [scratch()]),
        "rvq_read_error_count": (rq.rvq_read_error_count, [t(1, dtype=torch.int64)]),
    }


def every_call(t):
    return {**operators(t), **quantiser(t)}


NAMES = sorted(every_call(lambda *shape, dtype=F32: None))


@pytest.mark.parametrize("name", NAMES)
def test_calls_run_on_their_tensors_device(name, gpus):
    for index in (0, 1):
        call, tensors = every_call(lambda *shape, dtype=F32: OnGpu(index, *shape, dtype=dtype))[name]
        call(*tensors)
        assert gpus.pop() == (name, index, 100 + index)
        call(*tensors, stream=Stream(index, 7))
        assert gpus.pop() == (name, index, 7)
        with pytest.raises(ValueError):
            call(*tensors, stream=Stream(1 - index, 7))
    assert not gpus and torch._C._cuda_getDevice() == 0


@pytest.mark.parametrize("name", NAMES)
def test_calls_refuse_tensors_of_two_devices(name, gpus):
    call, tensors = every_call(lambda *shape, dtype=F32: OnGpu(0, *shape, dtype=dtype))[name]
    for i, t in enumerate(tensors if len(tensors) > 1 else []):
        for other in (OnGpu(1, *t.shape, dtype=t.dtype), t.t):
            with pytest.raises(ValueError):
                call(*tensors[:i], other, *tensors[i + 1:])
    assert not gpus


# ---------------------------------------------------------------------------
# a stream of the caller's
# ---------------------------------------------------------------------------

@pytest.fixture
def streams(monkeypatch):
    """The stream that torch would allocate on, and who told the allocator of which stream."""
    class Log:
        now, used, allocated = "current", [], {}

        def of(self, stream):
            return {p for p, s in self.used if s == stream}

    log = Log()
    log.used, log.allocated = [], {}

    class Scope:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            self.before, log.now = log.now, self.stream

        def __exit__(self, *_):
            log.now = self.before

    empty = torch.empty

    def allocate(*args, **kw):
        t = empty(*args, **kw)
        log.allocated[t.untyped_storage().data_ptr()] = log.now
        return t

    monkeypatch.setattr(torch, "empty", allocate)
    monkeypatch.setattr(torch.cuda, "stream", Scope)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: log.now)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True, raising=False)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: log.used.append((t.untyped_storage().data_ptr(), s)))
    return log


def storage(t):
    return t.untyped_storage().data_ptr()


def test_beam_search_on_a_stream(monkeypatch, streams):
    """What a step on a stream of the caller's writes is allocated there (a block freed by the current stream may still
    be in use by it), and nothing that it touches is given away before it has run."""
    ran = []
    monkeypatch.setattr(rq, "rvq_beam_select", lambda *a: ran.append((a[-1], streams.now)))
    monkeypatch.setattr(rq, "rvq_beam_reorder", lambda *a: ran.append((a[-1], streams.now)))
    monkeypatch.setattr(rq, "rvq_beam_states", lambda pairs, layered: pairs)
    search = rq.BeamSearch(2, 3, 10, end_code=1, device="cpu")
    logits, scores, finished = torch.zeros(2, 3, 10), torch.zeros(2, 3), torch.zeros((2, 3), dtype=torch.bool)
    out = search.select(logits, scores, finished, stream="side")
    assert ran.pop() == ("side", "side")
    assert {streams.allocated[storage(t)] for t in out} == {"side"}
    assert streams.of("side") == {storage(t) for t in (logits, scores, finished, search.workspace)}
    assert streams.of("current") == {storage(t) for t in out}

    streams.used.clear()
    state = torch.zeros(2, 3, 4)
    moved = search.reorder(out[1], state, stream="side")
    assert ran.pop() == ("side", "side") and streams.allocated[storage(moved)] == "side"
    assert streams.of("side") == {storage(out[1]), storage(state)} and streams.of("current") == {storage(moved)}

    streams.used.clear()
    place = torch.zeros(2, 3, 4)
    assert search.reorder(out[1], state, place, stream="side") is place
    assert streams.of("side") == {storage(out[1]), storage(state), storage(place)}

    assert ran.pop() == ("side", "side") and not ran
    streams.used.clear()
    search.reorder(search.select(logits, scores)[1], state)
    assert not streams.used and {s for s, _ in ran} == {None}


def test_quantiser_on_a_stream(monkeypatch, streams):
    """The quantiser's own calls in the same way, conversions of what they are given among them."""
    ran = []
    for name, value in (("rvq_dims_supported", 0), ("rvq_tables_bytes", 64), ("rvq_encode_scratch_bytes", 64)):
        monkeypatch.setattr(rq, name, lambda *a, value=value: value)
    monkeypatch.setattr(rq, "rvq_prepare", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    for name in ("rvq_encode", "rvq_decode", "rvq_reconstruct"):
        monkeypatch.setattr(rq, name, lambda *a: ran.append((a[-1], streams.now)))
    rvq = rq.RVQ(torch.zeros(2, 4, 8), torch.zeros(2, 16, 4), torch.zeros(2, 8, 4), device="cpu")
    converted = []
    frames = rvq._frames
    monkeypatch.setattr(rvq, "_frames", lambda x: (converted.append(streams.now), frames(x))[1])
    x, codes = torch.zeros(5, 8, dtype=torch.float64), torch.zeros(5, 2, dtype=torch.int64)
    for call, given in ((rvq.encode, x), (rvq.decode, codes), (rvq.reconstruct, x)):
        streams.used.clear()
        out = call(given, stream="side")
        out = out if isinstance(out, tuple) else (out,)
        assert ran.pop() == ("side", "side") and set(converted) == {"side"}
        assert {streams.allocated[storage(t)] for t in out} == {"side"}
        kept = {storage(given), storage(rvq.tables)} | ({storage(rvq._scratch)} if given is x else set())
        assert kept <= streams.of("side") and {storage(t) for t in out} <= streams.of("current")
        streams.used.clear()
        call(given)
        assert ran.pop() == (None, "current") and not streams.used
        converted[:] = ["side"]


# ---------------------------------------------------------------------------
# overlapping memory
# ---------------------------------------------------------------------------

WRAPPER = """
#include "rvq_overlap.h"
static rvq::RowSet set(const int64_t *v) {
  return {reinterpret_cast<const void *>(v[0]), v[1], {{v[2], v[3]}, {v[4], v[5]}, {v[6], v[7]}}};
}
extern "C" int itself(const int64_t *a) { return (int)rvq::overlaps_itself(set(a)); }
extern "C" int both(const int64_t *a, const int64_t *b) { return (int)rvq::overlap(set(a), set(b)); }
"""


@pytest.fixture(scope="module")
def regions(tmp_path_factory):
    where = tmp_path_factory.mktemp("overlap")
    source, library = where / "overlap.cpp", where / "overlap.so"
    source.write_text(WRAPPER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(source), "-o", str(library)], check=True)
    lib = ctypes.CDLL(str(library))
    return lambda *sets: (lib.itself if len(sets) == 1 else lib.both)(*((ctypes.c_int64 * 8)(*s) for s in sets))


def every_byte(base, row, *axes):
    counts, strides = axes[0::2], axes[1::2]
    return [base + sum(i * s for i, s in zip(index, strides)) + b
            for index in itertools.product(*(range(n) for n in counts)) for b in range(row)]


def test_overlaps_byte_by_byte(regions):
    """Random sets of rows, nested, interleaved and crossing, with negative strides and strides of 0."""
    r = random.Random(1)
    seen = set()
    for _ in range(6000):
        sets = []
        for _ in range(2):
            s = [1000 + r.randint(0, 60), r.randint(1, 6)]
            for _ in range(3):
                s += [r.choice([1, 1, 2, 3, 5]), r.choice([0, 1, 2, 3, 4, 6, 8, 12, 16, 24, 25, 48, -4, -12])]
            sets.append(s)
        if r.random() < 0.4:
            sets[1][3::2] = sets[0][3::2]
        bytes_of = [every_byte(*s) for s in sets]
        alone = int(len(set(bytes_of[0])) < len(bytes_of[0]))
        common = int(bool(set(bytes_of[0]) & set(bytes_of[1])))
        assert regions(sets[0]) == alone, sets[0]
        assert regions(*sets) == common and regions(*sets[::-1]) == common, sets
        seen.add((alone, common))
    assert len(seen) == 4


def test_overlaps_of_large_layouts(regions):
    g, t, w = 1 << 20, 4096, 1024
    keys = [1 << 40, w, 48, 2 * g * 8 * w, g, 2 * 8 * w, 8, 2 * w]       # [layer][group][beam][key, value][w]
    values = [(1 << 40) + w] + keys[1:]
    assert regions(keys) == 0 and regions(keys, values) == 0
    assert regions(keys, [(1 << 40) + w - 1] + keys[1:]) == 1
    assert regions([1 << 40, w, 48, 0, g, 8 * w, 8, w]) == 1
    # a part of one buffer to another part of it, with another number of slots and other strides
    assert regions([0, w, 48, g * 16 * t, g, 16 * t, 4, t], [w, w, 48, g * 16 * t, g, 16 * t, 16, t]) == 0
    assert regions([0, w, 48, g * 16 * t, g, 16 * t, 4, t], [w, t, 48, g * 16 * t, g, 16 * t, 16, t]) == 1
    # strides that do not nest are given up after a bounded number of steps, or told apart
    assert regions([0, 2, g, 3 << 30, g, 5 << 20, g, 7 << 10]) in (1, 2)
    assert regions([0, 1, 1 << 40, 2, 1, 0, 1, 0], [1, 1, 1 << 40, 4, 1, 0, 1, 0]) in (0, 2)


INVALID = -1


def test_reorder_refuses_overlaps(lib):
    """All of these are refused on the host: none reaches a launch."""
    dims = rq.rvq_beam_dims(3, 4, 100, 4, 0, 1)
    a, b, parents = 1 << 20, 2 << 20, ctypes.c_void_p(3 << 20)

    def state(src=a, dst=b, layers=2, row=16, ls=192, gs=64, bs=16, dls=192, dgs=64, dbs=16):
        return rq.rvq_beam_state(src, dst, layers, row, ls, gs, bs, dls, dgs, dbs)

    def run(*states, where=parents):
        return lib.rvq_beam_reorder(dims, where, (rq.rvq_beam_state * len(states))(*states), len(states), None)

    for bad in (state(dbs=0), state(dgs=0), state(dls=0), state(dbs=15), state(dgs=48), state(dls=176),     # in itself
                state(dst=a + 16), state(dst=a - 16), state(dst=a + 383), state(src=a, dst=a, bs=0, dbs=0),
                state(dst=a, gs=128, dgs=64)):
        assert run(bad) == INVALID
    assert run(state(), state(dst=b + 64)) == INVALID                          # two destinations
    assert run(state(), state(src=b, dst=4 << 20)) == INVALID                  # a chain
    assert run(state(src=a, dst=a), state(src=b, dst=a + 16)) == INVALID       # into what is reordered in place
    assert run(state(src=a, dst=a), state(src=a, dst=a)) == INVALID            # in place twice
    assert run(state(), where=ctypes.c_void_p(b + 380)) == INVALID             # over the parents


@pytest.mark.parametrize("vocab", [100, 70000])
def test_select_refuses_overlaps(lib, vocab):
    """Refused on the host; 3 groups, 4 beams in, 5 out."""
    a = 1 << 24
    place = {"z": a, "s": 2 * a, "f": 3 * a, "o": 4 * a, "p": 5 * a, "c": 6 * a, "of": 7 * a, "ws": 8 * a}

    def run(select, **kw):
        dims = rq.rvq_beam_dims(3, 4, vocab, select, 0, 1)
        at = {k: ctypes.c_void_p(v) for k, v in {**place, **kw}.items()}
        nbytes = lib.rvq_beam_workspace_bytes(dims)
        return lib.rvq_beam_select(dims, at["z"], vocab, at["s"], at["f"], 7, at["o"], at["p"], at["c"], at["of"],
                                   at["ws"], nbytes, None)

    assert run(5, o=place["s"]) == INVALID and run(5, of=place["f"]) == INVALID      # not the same number of slots
    for select, kept in ((4, 12), (5, 15)):
        assert run(select, o=place["s"] + 4) == INVALID and run(select, of=place["f"] + 11) == INVALID
        for out, size in (("o", 4), ("p", 4), ("c", 4), ("of", 1)):
            for other, bytes_of in (("s", 48), ("f", 12), ("z", 12 * vocab * 2), ("o", 4 * kept), ("p", 4 * kept),
                                    ("c", 4 * kept), ("of", kept)):
                if other in (out, {"o": "s", "of": "f"}.get(out)):
                    continue
                assert run(select, **{out: place[other] + (bytes_of - 1) // size * size}) == INVALID, (out, other)
                assert run(select, **{out: place[other] - (kept - 1) * size}) == INVALID, (out, other)
    if vocab > 1000:                                                                  # a workspace that is used
        for name in ("z", "s", "f", "o", "p", "c", "of"):
            assert run(4, ws=place[name]) == INVALID


def test_norm_and_distill_refuse_overlaps(lib):
    """Outputs that meet their inputs anywhere but row by row; refused on the host."""
    at = 1 << 24
    norm = rq.rvq_norm_dims(4, 64, 1, 0, 1e-5)                       # rows of 128 bytes
    distill = rq.rvq_distill_dims(4, 64, 8, 1, 0, 1.0)
    far = ctypes.c_void_p(1 << 26)
    for stride, to, to_stride in ((64, at, 65), (64, at + 2, 64), (64, at - 128, 64), (64, at + 3 * 128 + 126, 64),
                                  (96, at + 64 * 2 - 2, 96), (200, at + 128 + 2, 130)):
        x, y = ctypes.c_void_p(at), ctypes.c_void_p(to)
        assert lib.rvq_layer_norm(norm, x, stride, None, None, y, to_stride, None, None, None) == INVALID
        for dy, other in ((x, far), (far, x)):
            strides = (stride, 64) if dy is x else (64, stride)
            assert lib.rvq_layer_norm_backward(norm, dy, strides[0], other, strides[1], None, far, far, y, to_stride, None,
                                               None, None, 0, None) == INVALID
        assert lib.rvq_distill(distill, x, stride, far, far, None, None, far, None, y, to_stride, None, None) == INVALID
        assert lib.rvq_distill_backward(distill, None, x, stride, far, far, None, None, far, y, to_stride, None) == INVALID


def test_select_takes_one_beam_of_longer_rows(monkeypatch, gpus):
    """The last position's logits of [groups][length][vocab]: rows evenly spaced, the beams' axis of size one having a
    stride of its own."""
    strides = []
    monkeypatch.setattr(rq, "_enqueue", lambda name, on, stream, dims, p, stride, *rest: strides.append(stride))
    dims = rq.rvq_beam_dims(2, 1, 10, 1, 0, 0)
    kept = OnGpu(0, 2, 1, dtype=I32)

    def run(view):
        logits = OnGpu(0)
        logits.t = view
        rq.rvq_beam_select(dims, logits, OnGpu(0, 2, 1), None, -1, OnGpu(0, 2, 1), kept, kept, None,
                           OnGpu(0, 64, dtype=U8))
        return strides.pop()

    wide = torch.zeros(2, 5, 12)
    assert run(wide[:, -1:, :10]) == 60 and run(wide[:, -1, :10][:, None]) == 60 and run(wide[:, 0, :10]) == 60
    assert run(torch.zeros(2, 1, 10)) == 10
    dims = rq.rvq_beam_dims(2, 5, 10, 1, 0, 0)
    rows = OnGpu(0)
    rows.t = wide[..., :10]
    held, one = OnGpu(0, 2, 5), OnGpu(0, 2, 1)
    rq.rvq_beam_select(dims, rows, held, None, -1, one, kept, kept, None, OnGpu(0, 64, dtype=U8))
    assert strides.pop() == 12
    rows.t = torch.zeros(2, 6, 12)[:, :5, :10]
    with pytest.raises(ValueError):
        rq.rvq_beam_select(dims, rows, held, None, -1, one, kept, kept, None, OnGpu(0, 64, dtype=U8))


def test_distill_refuses_temperatures_without_an_inverse(lib):
    """1 / T, or log2(e) / T, past float32 (the temperature itself a positive number)."""
    far = ctypes.c_void_p(1 << 26)

    def run(rows, temperature):
        dims = rq.rvq_distill_dims(rows, 64, 8, 1, 0, temperature)
        return lib.rvq_distill(dims, ctypes.c_void_p(1 << 24), 64, far, far, None, None, far, None, None, 0, None, None)

    for temperature in (1.5e-45, 1e-39, 2.9e-39, 4.2e-39):
        assert run(4, temperature) == INVALID and run(0, temperature) == INVALID
    for temperature in (4.3e-39, 1.2e-38, 1.0, 3.4e38):      # no rows: nothing is launched
        assert run(0, temperature) == 0


def test_autograd_notices_what_is_written_in_place(monkeypatch):
    """The gradient over the logits, and states reordered in place: a backward pass that saved them must not use what
    was written over them."""
    monkeypatch.setattr(rq, "rvq_distill", lambda *a, **kw: None)
    monkeypatch.setattr(rq, "rvq_beam_reorder", lambda *a: None)
    monkeypatch.setattr(rq, "rvq_beam_states", lambda pairs, layered: pairs)
    leaf = torch.ones(2, 3, 8, requires_grad=True)
    logits = leaf * 2
    squared = logits * logits
    entries = torch.zeros(2, 3, 4)
    _, out = rq.distill_loss_and_grad(logits.detach(), entries, entries.int(), out=logits.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        squared.sum().backward()
    state = leaf * 3
    squared = state * state
    rq.BeamSearch(2, 3, 10, device="cpu").reorder(None, state.detach(), state.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        squared.sum().backward()


@pytest.mark.parametrize("dtype", [torch.int8, torch.uint8, torch.int16, torch.int32, torch.int64])
def test_teacher_codes_of_any_integer_type(dtype):
    """Narrow types (codes of 256 entries as bytes) hold no bound of 32 bits; a code past 32 bits stays out of range."""
    codes = [[5, 0, 100], [127, 7, 3]] + ([[-1, -7, 2]] if dtype != torch.uint8 else [])
    if dtype == torch.int64:
        codes.append([(1 << 32) + 5, -(1 << 40), 2 ** 31 - 1])
    given = torch.tensor(codes, dtype=dtype)
    entries = torch.zeros(len(codes), 3)
    _, (_, got, _, _) = predictor._teacher(torch.zeros(len(codes), 200), entries, given, None, None)
    want = codes if dtype == torch.int32 else [[min(max(c, -2), 2 ** 31 - 1) for c in row] for row in codes]
    assert got.dtype == torch.int32 and got.tolist() == want


def test_states_without_elements():
    """A cache before its first entry, wherever its axis of length zero is: nothing to move, nothing to refuse."""
    for row in ((0, 64), (4, 0, 64), (4, 2, 0), (0,)):
        states = rq.rvq_beam_states([(OnGpu(0, 2, 3, *row), OnGpu(0, 2, 5, *row))])
        assert states[0].row_bytes == 0
    states = rq.rvq_beam_states([(OnGpu(0, 2, 3, 4, 2), OnGpu(0, 2, 5, 4, 2))])
    assert states[0].row_bytes == 32
    with pytest.raises(ValueError):
        rq.rvq_beam_states([(OnGpu(0, 2, 3, 0, 64), OnGpu(0, 2, 5, 0, 65))])


def test_streams_of_other_libraries(gpus, streams, monkeypatch):
    """An object with nothing but the handle is a stream of the tensors' device."""
    class Handle:
        cuda_stream = 77

    call, tensors = quantiser(lambda *shape, dtype=F32: OnGpu(1, *shape, dtype=dtype))["rvq_encode"]
    call(*tensors, stream=Handle())
    assert gpus.pop() == ("rvq_encode", 1, 77)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: f"external {handle} {device}")
    rq._run_on(Handle(), "cuda:1", lambda: torch.empty(2), lambda: ())
    assert list(streams.allocated.values()) == ["external 77 cuda:1"]
