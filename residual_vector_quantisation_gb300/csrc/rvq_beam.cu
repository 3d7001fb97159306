// The beam step: selection of the best candidates over beams and codes, and
// the reordering of the states that follow them (rvq_beam_select,
// rvq_beam_reorder).
//
// Selection is one read of the logits.  k_beam_rows: blocks over pieces of the
// beams' rows, each leaving its piece's best `select` entries in order and its
// part of the row's log sum exp.  k_beam_groups: a warp per group walks those
// lists from their heads.
#include "rvq_internal.cuh"
#include "rvq_rows.cuh"

namespace rvq {
namespace {

constexpr int kBeamMax = 64;           // beams, and candidates kept
constexpr int kBeamMaxVocab = 1 << 24;
constexpr int kRowThreads = 256;
constexpr int kRowPiece = 16;          // elements of a thread per step
constexpr int kRowStep = kRowThreads * kRowPiece;
constexpr int kBeamMaxSplits = 16;

// An entry's place in the order: the larger value first, then the lower code.
// 0 is no entry (NaN and -inf have none).
__device__ __forceinline__ uint32_t order_of(float v) {
  if (!(v > -CUDART_INF_F)) return 0;
  const uint32_t b = __float_as_uint(v + 0.f);  // -0 becomes 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float v, int code) {
  const uint32_t o = order_of(v);
  return o ? (uint64_t)o << 32 | (uint32_t)~code : 0;
}

// A sum of e^x as s * e^m, m the largest x: joins (m2, s2) to (m, s).
__device__ __forceinline__ void join_sum(float &m, float &s, float m2, float s2) {
  const float mm = fmaxf(m, m2), z = mm == -CUDART_INF_F ? 0.f : mm;
  s = s * exp2_fast((m - z) * kLog2e) + s2 * exp2_fast((m2 - z) * kLog2e);
  m = mm;
}

// A piece's results in the workspace: its part of the row's sum of e^x and its
// best entries in order.
struct BeamParts {
  float2 *sum;     // [rows][splits]: m, s of s * e^m
  uint64_t *list;  // [rows][splits][select]
};

struct BeamArgs {
  rvq_beam_dims dm;
  const void *logits;
  int64_t stride;
  const float *scores;
  const uint8_t *finished;
  int32_t end_code;
  float *out_scores;
  int32_t *parents, *codes;
  uint8_t *out_finished;
  int splits;
  BeamParts parts;
};

// Whether a beam's row is read.
__device__ __forceinline__ bool beam_live(const BeamArgs &a, int64_t row) {
  return a.scores[row] > -CUDART_INF_F && !(a.finished && a.finished[row]);
}

template <class T>
__global__ void __launch_bounds__(kRowThreads) k_beam_rows(const BeamArgs a) {
  constexpr int N = 16 / (int)sizeof(T), NV = kRowPiece / N;
  constexpr int kRoom = kBeamMax * kRowPiece + kBeamMax;
  __shared__ uint64_t best[kBeamMax], most[kRowThreads], room[kRoom];
  __shared__ uint64_t bar;
  __shared__ int found;
  __shared__ float2 box[kRowThreads / 32];
  const int n = a.dm.select, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool raw = a.dm.mode == RVQ_BEAM_RAW;
  const int64_t row = blockIdx.x / a.splits;
  const int split = (int)(blockIdx.x % a.splits);
  if (!beam_live(a, row)) return;
  const RowVectors<T> in(static_cast<const T *>(a.logits) + row * a.stride, a.dm.vocab);
  // pieces of whole steps, as even as they come
  const int nv = in.count(), steps = (nv + kRowThreads * NV - 1) / (kRowThreads * NV);
  const int s0 = (int)((int64_t)steps * split / a.splits), s1 = (int)((int64_t)steps * (split + 1) / a.splits);
  const float add = raw ? a.scores[row] : 0.f;
  float m = -CUDART_INF_F, s = 0.f;
  if (tid < kBeamMax) best[tid] = 0;
  if (tid == 0) found = 0, bar = 0;
  for (int st = s0; st < s1; ++st) {
    float f[NV][N];
    uint64_t top = 0;
    float high = -CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = (st * NV + j) * kRowThreads + tid;
      uint4 u = v < nv ? in.load(v, from_float<T>(-CUDART_INF_F)) : make_uint4(0, 0, 0, 0);
      unpack16<T>(u, f[j]);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (v >= nv) f[j][i] = -CUDART_INF_F;
        if (raw) f[j][i] += add;
        high = fmaxf(high, f[j][i]);
        const uint64_t k = key_of(f[j][i], v * N + i - in.phase);
        top = k > top ? k : top;
      }
    }
    if (!raw) {
      const float at = high == -CUDART_INF_F ? 0.f : high;
      float t = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) t += exp2_fast((f[j][i] - at) * kLog2e);
      join_sum(m, s, high, t);
    }
    // The n-th best of the threads' best entries is a bar that n entries reach
    // and that those of n threads at most can reach.
    most[tid] = top;
    __syncthreads();
    int rank = 0;
    for (int i = 0; i < kRowThreads; ++i) rank += most[i] > top;
    const uint64_t held = best[n - 1];
    if (rank == n - 1 && top > held) bar = top;  // one thread at most: keys differ, and 0 is not > held
    __syncthreads();
    const uint64_t line = bar > held ? bar : held + 1;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int v = (st * NV + j) * kRowThreads + tid;
        const uint64_t k = key_of(f[j][i], v * N + i - in.phase);
        if (k >= line) room[atomicAdd(&found, 1)] = k;
      }
    __syncthreads();
    const int fresh = found, all = fresh + n;
    if (tid < n) room[fresh + tid] = best[tid];
    __syncthreads();
    // each entry's place among them (empty ones, 0, have none)
    for (int i = tid; i < all; i += kRowThreads) {
      const uint64_t k = room[i];
      if (!k) continue;
      int place = 0;
      for (int j = 0; j < all; ++j) place += room[j] > k;
      if (place < n) best[place] = k;
    }
    __syncthreads();
    if (tid == 0) found = 0, bar = 0;
  }
  __syncthreads();
  const int64_t at = row * a.splits + split;
  if (tid < n) a.parts.list[at * n + tid] = best[tid];
  if (raw) return;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    join_sum(m, s, m2, s2);
  }
  if (lane == 0) box[warp] = make_float2(m, s);
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kRowThreads / 32; ++w) join_sum(m, s, box[w].x, box[w].y);
    a.parts.sum[at] = make_float2(m, s);
  }
}

// One warp per group.  A lane keeps the heads of the lists lane, lane + 32,
// ...; the best head over the warp is chosen `select` times.
constexpr int kGroupWarps = 4;

struct Head {
  uint32_t total;  // order_of the candidate's total; 0: none left
  int32_t beam;
  uint64_t key;    // its entry: value, then code
};
__device__ __forceinline__ bool better(const Head &x, const Head &y) {
  if (x.total != y.total) return x.total > y.total;
  if (x.beam != y.beam) return x.beam < y.beam;
  return x.key > y.key;
}

__global__ void __launch_bounds__(32 * kGroupWarps) k_beam_groups(const BeamArgs a) {
  __shared__ float2 lse[kGroupWarps][kBeamMax];  // of a row: m, log s
  __shared__ uint8_t next[kGroupWarps][kBeamMax * kBeamMaxSplits];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t g = (int64_t)blockIdx.x * kGroupWarps + warp;
  if (g >= a.dm.groups) return;
  const int B = a.dm.beams, n = a.dm.select, S = a.splits, lists = B * S;
  const bool raw = a.dm.mode == RVQ_BEAM_RAW;
  for (int b = lane; b < B; b += 32) {
    const int64_t row = g * B + b;
    float m = 0.f, s = 1.f;
    if (!raw && beam_live(a, row)) {
      m = -CUDART_INF_F, s = 0.f;
      for (int i = 0; i < S; ++i) join_sum(m, s, a.parts.sum[row * S + i].x, a.parts.sum[row * S + i].y);
    }
    lse[warp][b] = make_float2(m, logf(s));
  }
  for (int i = lane; i < lists; i += 32) next[warp][i] = 0;
  __syncwarp();
  auto head = [&](int list) {
    const int b = list / S, at = next[warp][list];
    const int64_t row = g * B + b;
    Head h{0, b, 0};
    const float score = a.scores[row];
    if (!(score > -CUDART_INF_F) || at >= n) return h;
    if (a.finished && a.finished[row]) {
      if (list % S == 0 && at == 0) h.key = key_of(0.f, a.end_code), h.total = order_of(score);
      return h;
    }
    h.key = a.parts.list[(row * S + list % S) * n + at];
    if (h.key) {
      const float v = value_of((uint32_t)(h.key >> 32));
      h.total = order_of(raw ? v : score + ((v - lse[warp][b].x) - lse[warp][b].y));
    }
    return h;
  };
  Head mine{0, 0, 0};
  int from = -1;
  auto look = [&]() {
    mine.total = 0;
    from = -1;
    for (int i = lane; i < lists; i += 32) {
      const Head h = head(i);
      if (h.total && (from < 0 || better(h, mine))) mine = h, from = i;
    }
  };
  look();
  for (int j = 0; j < n; ++j) {
    const uint32_t total = __reduce_max_sync(0xffffffffu, mine.total);
    bool in = mine.total == total && total;
    const uint32_t beam = __reduce_min_sync(0xffffffffu, in ? (uint32_t)mine.beam : ~0u);
    in = in && (uint32_t)mine.beam == beam;
    const uint32_t hi = __reduce_max_sync(0xffffffffu, in ? (uint32_t)(mine.key >> 32) : 0u);
    in = in && (uint32_t)(mine.key >> 32) == hi;
    const uint32_t lo = __reduce_max_sync(0xffffffffu, in ? (uint32_t)mine.key : 0u);
    in = in && (uint32_t)mine.key == lo;
    const int64_t o = g * n + j;
    if (total == 0) {
      if (lane == 0) {
        a.out_scores[o] = -CUDART_INF_F;
        a.parents[o] = a.codes[o] = -1;
        if (a.out_finished) a.out_finished[o] = 1;
      }
    } else if (in) {
      const int code = (int)~(uint32_t)mine.key;
      a.out_scores[o] = value_of(mine.total);
      a.parents[o] = mine.beam;
      a.codes[o] = code;
      if (a.out_finished)
        a.out_finished[o] = (a.finished && a.finished[g * B + mine.beam]) || code == a.end_code;
      ++next[warp][from];
      look();
    }
  }
}

// ---------------------------------------------------------------------------
// reordering
// ---------------------------------------------------------------------------

struct StateList {
  rvq_beam_state s[RVQ_BEAM_MAX_STATES];
};

// One block per (layer, group, slot) and piece of the row, states on grid.z.
constexpr int kMoveThreads = 256;
__global__ void __launch_bounds__(kMoveThreads)
    k_beam_reorder(const __grid_constant__ StateList list, const int32_t *__restrict__ parents, int64_t groups,
                   int beams, int select) {
  const rvq_beam_state s = list.s[blockIdx.z];
  const int64_t slots = s.layers * groups * select;
  for (int64_t i = blockIdx.x; i < slots; i += gridDim.x) {
    const int64_t layer = i / (groups * select), gs = i % (groups * select), g = gs / select;
    const int j = (int)(gs % select), p = parents[gs];
    const char *src = static_cast<const char *>(s.src) + layer * s.src_layer_stride + g * s.src_group_stride +
                      (p >= 0 && p < beams ? p : 0) * s.src_beam_stride;
    char *dst = static_cast<char *>(s.dst) + layer * s.dst_layer_stride + g * s.dst_group_stride + j * s.dst_beam_stride;
    const bool none = p < 0 || p >= beams;
    const uintptr_t both = reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst) | (uintptr_t)s.row_bytes;
    const int64_t t = (int64_t)blockIdx.y * kMoveThreads + threadIdx.x, step = (int64_t)gridDim.y * kMoveThreads;
    if ((both & 15) == 0) {
      for (int64_t k = t; k < s.row_bytes / 16; k += step)
        reinterpret_cast<uint4 *>(dst)[k] = none ? make_uint4(0, 0, 0, 0) : reinterpret_cast<const uint4 *>(src)[k];
    } else if ((both & 3) == 0) {
      for (int64_t k = t; k < s.row_bytes / 4; k += step)
        reinterpret_cast<uint32_t *>(dst)[k] = none ? 0u : reinterpret_cast<const uint32_t *>(src)[k];
    } else {
      for (int64_t k = t; k < s.row_bytes; k += step) dst[k] = none ? 0 : src[k];
    }
  }
}

// In place: a block takes one piece of all beams' rows of a group through
// shared memory, W bytes a lane at a time.
template <class W>
__global__ void __launch_bounds__(kMoveThreads)
    k_beam_reorder_in_place(const __grid_constant__ StateList list, const int32_t *__restrict__ parents,
                            int64_t groups, int beams) {
  constexpr int kCols = 32;
  __shared__ W tile[kBeamMax][kCols];
  const rvq_beam_state s = list.s[blockIdx.z];
  if (s.src != s.dst) return;
  // widest words that the rows allow
  const uintptr_t all = reinterpret_cast<uintptr_t>(s.dst) | (uintptr_t)s.row_bytes | (uintptr_t)s.dst_layer_stride |
                        (uintptr_t)s.dst_group_stride | (uintptr_t)s.dst_beam_stride;
  const int wide = (all & 15) == 0 ? 16 : (all & 3) == 0 ? 4 : 1;
  if (wide != (int)sizeof(W)) return;
  const int64_t words = s.row_bytes / (int64_t)sizeof(W), pieces = (words + kCols - 1) / kCols;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kMoveThreads / 32;
  for (int64_t i = blockIdx.x; i < s.layers * groups * pieces; i += gridDim.x) {
    const int64_t piece = i % pieces, lg = i / pieces, g = lg % groups, layer = lg / groups;
    char *base = static_cast<char *>(s.dst) + layer * s.dst_layer_stride + g * s.dst_group_stride;
    const int64_t k = piece * kCols + lane;
    __syncthreads();
    for (int b = warp; b < beams; b += warps)
      if (k < words) tile[b][lane] = reinterpret_cast<const W *>(base + b * s.dst_beam_stride)[k];
    __syncthreads();
    for (int b = warp; b < beams; b += warps) {
      const int p = parents[g * beams + b];
      if (p == b || k >= words) continue;
      W v{};
      if (p >= 0 && p < beams) v = tile[p][lane];
      reinterpret_cast<W *>(base + b * s.dst_beam_stride)[k] = v;
    }
  }
}

rvq_status check_beam(const rvq_beam_dims &dm) {
  if (dm.groups < 0 || dm.beams <= 0 || dm.vocab <= 0 || dm.select <= 0 || !dtype_bytes(dm.dtype)) return RVQ_ERR_INVALID_ARG;
  if (dm.mode != RVQ_BEAM_LOGITS && dm.mode != RVQ_BEAM_RAW) return RVQ_ERR_INVALID_ARG;
  if (dm.beams > kBeamMax || dm.select > kBeamMax || dm.vocab > kBeamMaxVocab) return RVQ_ERR_UNSUPPORTED;
  if (dm.groups > (int64_t)(1 << 30) / (dm.beams * kBeamMaxSplits)) return RVQ_ERR_UNSUPPORTED;
  return RVQ_OK;
}

// Pieces of a row: enough blocks for the GPU, no piece below one step.
int beam_splits(const rvq_beam_dims &dm) {
  const int64_t rows = dm.groups * dm.beams, steps = (dm.vocab + kRowStep - 1) / kRowStep;
  int64_t s = rows > 0 ? (152 * 4 + rows - 1) / rows : 1;
  if (s > steps) s = steps;
  if (s > kBeamMaxSplits) s = kBeamMaxSplits;
  return (int)s;
}

size_t beam_list_at(const rvq_beam_dims &dm) {
  return align_up((size_t)(dm.groups * dm.beams) * beam_splits(dm) * sizeof(float2));
}

}  // namespace
}  // namespace rvq

extern "C" {

RVQ_API size_t rvq_beam_workspace_bytes(rvq_beam_dims dims) {
  using namespace rvq;
  if (check_beam(dims) != RVQ_OK) return 0;
  return beam_list_at(dims) +
         align_up(((size_t)(dims.groups * dims.beams) + (dims.groups == 0)) * beam_splits(dims) * dims.select * 8);
}

RVQ_API rvq_status rvq_beam_select(rvq_beam_dims dims, const void *logits, int64_t logits_stride, const float *scores,
                                   const uint8_t *finished, int32_t end_code, float *out_scores, int32_t *parents,
                                   int32_t *codes, uint8_t *out_finished, void *workspace, size_t workspace_bytes,
                                   rvq_stream_t stream) {
  using namespace rvq;
  const rvq_status c = check_beam(dims);
  if (c != RVQ_OK) return c;
  if (end_code >= dims.vocab || end_code < (finished ? 0 : -1)) return RVQ_ERR_INVALID_ARG;
  if (dims.groups == 0) return RVQ_OK;
  if (!logits || !scores || !out_scores || !parents || !codes || !workspace) return RVQ_ERR_INVALID_ARG;
  if (!aligned_to(logits, dtype_bytes(dims.dtype)) || !aligned_to(scores, 4) || !aligned_to(out_scores, 4) ||
      !aligned_to(parents, 4) || !aligned_to(codes, 4) || !aligned_to(workspace, 16))
    return RVQ_ERR_INVALID_ARG;
  if (logits_stride < dims.vocab && dims.groups * dims.beams > 1) return RVQ_ERR_INVALID_ARG;
  if (workspace_bytes < rvq_beam_workspace_bytes(dims)) return RVQ_ERR_INVALID_ARG;
  BeamArgs a{dims, logits, logits_stride, scores, finished, end_code, out_scores, parents, codes, out_finished,
             beam_splits(dims), {at<float2>(workspace, 0), at<uint64_t>(workspace, beam_list_at(dims))}};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const unsigned blocks = (unsigned)(dims.groups * dims.beams * a.splits);
  if (dims.dtype == RVQ_DTYPE_F32)
    k_beam_rows<float><<<blocks, kRowThreads, 0, st>>>(a);
  else if (dims.dtype == RVQ_DTYPE_BF16)
    k_beam_rows<__nv_bfloat16><<<blocks, kRowThreads, 0, st>>>(a);
  else
    k_beam_rows<__half><<<blocks, kRowThreads, 0, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return RVQ_ERR_CUDA;
  k_beam_groups<<<(unsigned)((dims.groups + kGroupWarps - 1) / kGroupWarps), 32 * kGroupWarps, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? RVQ_OK : RVQ_ERR_CUDA;
}

RVQ_API rvq_status rvq_beam_reorder(rvq_beam_dims dims, const int32_t *parents, const rvq_beam_state *states,
                                    int32_t n_states, rvq_stream_t stream) {
  using namespace rvq;
  const rvq_status c = check_beam(dims);
  if (c != RVQ_OK) return c;
  if (n_states < 0 || n_states > RVQ_BEAM_MAX_STATES || (n_states > 0 && !states)) return RVQ_ERR_INVALID_ARG;
  StateList move, swap;
  int moves = 0, swaps = 0;
  int64_t slots = 0, bytes = 0, pieces = 0;
  bool wide[3] = {false, false, false};
  for (int i = 0; i < n_states; ++i) {
    const rvq_beam_state &s = states[i];
    if (s.layers < 0 || s.row_bytes < 0) return RVQ_ERR_INVALID_ARG;
    if (s.layers == 0 || s.row_bytes == 0 || dims.groups == 0) continue;
    if (!s.src || !s.dst) return RVQ_ERR_INVALID_ARG;
    if (s.src == s.dst) {
      if (dims.select != dims.beams || s.src_layer_stride != s.dst_layer_stride ||
          s.src_group_stride != s.dst_group_stride || s.src_beam_stride != s.dst_beam_stride)
        return RVQ_ERR_INVALID_ARG;
      swap.s[swaps++] = s;
      const uintptr_t all = reinterpret_cast<uintptr_t>(s.dst) | (uintptr_t)s.row_bytes |
                            (uintptr_t)s.dst_layer_stride | (uintptr_t)s.dst_group_stride | (uintptr_t)s.dst_beam_stride;
      const int w = (all & 15) == 0 ? 16 : (all & 3) == 0 ? 4 : 1;
      wide[w == 16 ? 0 : w == 4 ? 1 : 2] = true;
      const int64_t p = s.layers * dims.groups * ((s.row_bytes / w + 31) / 32);
      pieces = p > pieces ? p : pieces;
    } else {
      move.s[moves++] = s;
      slots = s.layers * dims.groups * dims.select > slots ? s.layers * dims.groups * dims.select : slots;
      bytes = s.row_bytes > bytes ? s.row_bytes : bytes;
    }
  }
  if (moves + swaps == 0) return RVQ_OK;
  if (!parents || !aligned_to(parents, 4)) return RVQ_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (moves) {
    int64_t across = (bytes / 16 + kMoveThreads * 4 - 1) / (kMoveThreads * 4);
    across = across < 1 ? 1 : across > 64 ? 64 : across;
    const dim3 grid((unsigned)(slots < (1 << 20) ? slots : (1 << 20)), (unsigned)across, (unsigned)moves);
    k_beam_reorder<<<grid, kMoveThreads, 0, st>>>(move, parents, dims.groups, dims.beams, dims.select);
    if (cudaGetLastError() != cudaSuccess) return RVQ_ERR_CUDA;
  }
  if (swaps) {
    const dim3 grid((unsigned)(pieces < (1 << 16) ? pieces : (1 << 16)), 1, (unsigned)swaps);
    if (wide[0]) k_beam_reorder_in_place<uint4><<<grid, kMoveThreads, 0, st>>>(swap, parents, dims.groups, dims.beams);
    if (wide[1]) k_beam_reorder_in_place<uint32_t><<<grid, kMoveThreads, 0, st>>>(swap, parents, dims.groups, dims.beams);
    if (wide[2]) k_beam_reorder_in_place<uint8_t><<<grid, kMoveThreads, 0, st>>>(swap, parents, dims.groups, dims.beams);
    if (cudaGetLastError() != cudaSuccess) return RVQ_ERR_CUDA;
  }
  return RVQ_OK;
}

}  // extern "C"
