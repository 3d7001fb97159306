// The beam step: selection of the best candidates over beams and codes, and
// the reordering of the states that follow them (rvq_beam_select,
// rvq_beam_reorder).
//
// Selection is one read of the logits.  A warp takes pieces of a row (32
// elements a lane, in registers) and keeps the row's best `select` entries so
// far: the n-th best of the lanes' largest values is a bar that at least n
// entries reach and few others do, so that only those are put in order.  A
// group of few pieces runs in one block that also joins the beams
// (k_beam_group); larger ones spread a row over blocks (k_beam_rows), whose
// lists a second kernel joins (k_beam_join).
#include "rvq_internal.cuh"
#include "rvq_overlap.h"
#include "rvq_rows.cuh"
#include "rvq_top.cuh"
#include "sm103_ptx.cuh"

namespace rvq {
namespace {

constexpr int kBeamMax = kMostKept;    // beams, and candidates kept
constexpr int kBeamMaxVocab = 1 << 24;
constexpr int kRowWarps = 8;           // of a block that shares a row
constexpr int kGroupWarps = 16;        // most warps of a block that takes a group
constexpr int kGroupItems = 64;        // most pieces of such a group
constexpr int kMaxLists = 128;         // most lists that a group's join reads
constexpr int kLane = 32;              // elements of a lane in a piece of a group's block
constexpr int kRowVectors = 16;        // 16-byte vectors of a lane in a piece of a block that shares a row

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

// A row's pieces and, unless its values are taken raw, the sum of e^z as (m, s),
// s of this lane alone.
template <class T, int NV, int PARTS>
__device__ __forceinline__ void beam_pieces(const CutRow<T> &in, int first, int step, int n, bool raw, float add,
                                            WarpRoom &r, float &m, float &s) {
  constexpr int N = 16 / (int)sizeof(T);
  m = -CUDART_INF_F, s = 0.f;
  warp_pieces<T, NV, PARTS>(in, first, step, n, add, r, [&](const uint4 (&z)[NV], float edge, float high) {
    if (raw) return;
    const float top = fmaxf(m, warp_max_order(high)), at = top == -CUDART_INF_F ? 0.f : top;
    s *= exp2_fast((m - at) * kLog2e);
    m = top;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[N];
      unpack16<T>(z[j], f);
#pragma unroll
      for (int i = 0; i < N; ++i) s += exp2_fast((f[i] - at) * kLog2e);
    }
    s += exp2_fast((edge - at) * kLog2e);
  });
}

// The join of a group's lists in shared memory: `lists` of n entries each, list
// i of beam i / per, sum[i] its part of the beam's sum; by all threads.
struct Join {
  uint64_t room[2 * kRoom + kBeamMax], tie[2 * kRoom + kBeamMax];
  float2 lse[kBeamMax];   // of a beam: m, log s
  float score[kBeamMax];  // -inf: dead
  bool done[kBeamMax];    // finished
  uint32_t bar;
  int count;
};

__device__ __forceinline__ void put_candidate(const BeamArgs &a, int64_t g, int place, uint32_t total, int beam,
                                              int code, bool done) {
  const int64_t o = g * a.dm.select + place;
  a.out_scores[o] = total ? value_of(total) : -CUDART_INF_F;
  a.parents[o] = total ? beam : -1;
  a.codes[o] = total ? code : -1;
  if (a.out_finished)
    a.out_finished[o] = !total || done || code == a.end_code;
}

// At most 32 entries: a lane of the first warp has one each.
__device__ __forceinline__ void join_in_warp(const BeamArgs &a, int64_t g, const uint64_t *list, const float2 *sum,
                                             int per) {
  const int n = a.dm.select, lane = threadIdx.x & 31, entries = a.dm.beams * per * n;
  if (threadIdx.x >= 32) return;
  uint32_t total = 0;
  uint64_t key = 0;
  bool done = false;
  const int b = lane / n / per;
  if (lane < entries) {
    const int64_t row = g * a.dm.beams + b;
    const float score = a.scores[row];
    done = a.finished && a.finished[row];
    if (score > -CUDART_INF_F && !done) {
      key = list[lane];
      const float v = value_of((uint32_t)(key >> 32));
      if (a.dm.mode == RVQ_BEAM_RAW) {
        total = (uint32_t)(key >> 32);
      } else if (key) {
        float m = -CUDART_INF_F, s = 0.f;
        for (int i = 0; i < per; ++i) join_sum(m, s, sum[b * per + i].x, sum[b * per + i].y);
        total = order_of(score + ((v - m) - logf(s)));
      }
    } else if (lane % (per * n) == 0 && score > -CUDART_INF_F) {
      key = key_of(0.f, a.end_code), total = order_of(score);
    }
  }
  const uint64_t mine = (uint64_t)total << 32 | (uint32_t)~b;
  int place = 0;
  for (int i = 0; i < entries; ++i) {
    const uint64_t k = __shfl_sync(0xffffffffu, mine, i), t = __shfl_sync(0xffffffffu, key, i);
    place += k > mine || (k == mine && t > key);
  }
  const int found = __popc(__ballot_sync(0xffffffffu, total != 0));
  if (total && place < n) put_candidate(a, g, place, total, b, (int)~(uint32_t)key, done);
  if (lane >= found && lane < n) put_candidate(a, g, lane, 0, 0, 0, true);
  for (int i = lane + 32; i < n; i += 32) put_candidate(a, g, i, 0, 0, 0, true);
}

__device__ __forceinline__ void join_group(const BeamArgs &a, int64_t g, const uint64_t *list, const float2 *sum, int per, Join &w) {
  const int B = a.dm.beams, n = a.dm.select, lists = B * per, tid = threadIdx.x, lane = tid & 31;
  if (lists * n <= 32) return join_in_warp(a, g, list, sum, per);
  for (int b = tid; b < B; b += blockDim.x) {
    const int64_t row = g * B + b;
    const float score = a.scores[row];
    const bool done = a.finished && a.finished[row];
    float m = -CUDART_INF_F, s = 0.f;
    if (a.dm.mode != RVQ_BEAM_RAW && !done)
      for (int i = 0; i < per; ++i) join_sum(m, s, sum[b * per + i].x, sum[b * per + i].y);
    w.lse[b] = make_float2(m, logf(s));
    w.score[b] = score > -CUDART_INF_F ? score : -CUDART_INF_F;
    w.done[b] = done;
  }
  if (tid == 0) w.bar = 0, w.count = 0;
  __syncthreads();
  // Entry i's total and key.  A finished beam's one candidate is its first entry, a dead one has none; the
  // lists of both were never written.
  auto entry = [&](int i, uint64_t &key) -> uint32_t {
    const int b = i / n / per;
    const float score = w.score[b];
    key = 0;
    if (score == -CUDART_INF_F) return 0;
    if (w.done[b]) {
      if (i != b * per * n) return 0;
      key = key_of(0.f, a.end_code);
      return order_of(score);
    }
    key = list[i];
    if (!key || a.dm.mode == RVQ_BEAM_RAW) return (uint32_t)(key >> 32);
    return order_of(score + ((value_of((uint32_t)(key >> 32)) - w.lse[b].x) - w.lse[b].y));
  };
  // the best of the lists' last entries is a bar that n entries reach
  uint32_t bar = 0;
  uint64_t key;
  for (int i = tid; i < lists; i += blockDim.x) bar = max(bar, entry(i * n + n - 1, key));
  bar = __reduce_max_sync(0xffffffffu, bar);
  if (lane == 0 && bar) atomicMax(&w.bar, bar);
  __syncthreads();
  bar = max(w.bar, 1u);
  constexpr int kTop = 2 * kRoom;
  for (int i = tid; i < lists * n; i += blockDim.x) {
    const uint32_t t = entry(i, key);
    if (t >= bar) {
      const int at = atomicAdd(&w.count, 1);
      if (at < kTop) {
        w.room[at] = (uint64_t)t << 32 | (uint32_t)~(i / n / per);
        w.tie[at] = key;
      }
    }
  }
  __syncthreads();
  const int all = w.count;
  auto put = [&](int place, uint64_t k, uint64_t tie) {
    const int beam = (int)~(uint32_t)k;
    put_candidate(a, g, place, (uint32_t)(k >> 32), beam, (int)~(uint32_t)tie, w.done[beam]);
  };
  int found = min(all, n);
  if (all <= kTop) {
    for (int i = tid; i < all; i += blockDim.x) {
      const uint64_t k = w.room[i], t = w.tie[i];
      int place = 0;
      for (int j = 0; j < all; ++j) place += w.room[j] > k || (w.room[j] == k && w.tie[j] > t);
      if (place < n) put(place, k, t);
    }
  } else if (tid < 32) {
    // many equal totals: the best n one after the other
    uint64_t k0 = ~0ull, t0 = ~0ull;
    for (int c = 0; c < n; ++c) {
      uint64_t k = 0, t = 0;
      for (int i = lane; i < lists * n; i += 32) {
        const uint32_t total = entry(i, key);
        if (!total) continue;
        const uint64_t ki = (uint64_t)total << 32 | (uint32_t)~(i / n / per), ti = key;
        if ((ki < k0 || (ki == k0 && ti < t0)) && (ki > k || (ki == k && ti > t))) k = ki, t = ti;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const uint64_t k2 = __shfl_xor_sync(0xffffffffu, k, o), t2 = __shfl_xor_sync(0xffffffffu, t, o);
        if (k2 > k || (k2 == k && t2 > t)) k = k2, t = t2;
      }
      if (lane == 0) put(c, k, t);
      k0 = k, t0 = t;
    }
  }
  for (int j = found + tid; j < n; j += blockDim.x) put_candidate(a, g, j, 0, 0, 0, true);
}

// A block per group: `per` warps' shares of each beam's row, then the join.
// Bound by the chain of one group (score, row, bar, order, join: about 5 us)
// against the eight or so groups that an SM holds: 49 us a call in a graph for 12000
// groups of 4 rows of 1024 floats, whose bytes alone would take 30; with registers held
// down for more groups (3 and 4 blocks of 512 threads) it spills and loses.
template <class T, int PARTS>
__global__ void __launch_bounds__(32 * kGroupWarps, 2) k_beam_group(const BeamArgs a) {
  extern __shared__ uint64_t smem[];
  __shared__ Join join;
  const int n = a.dm.select, B = a.dm.beams, lane = threadIdx.x & 31, warps = blockDim.x >> 5, per = a.splits;
  uint64_t *list = smem;
  float2 *sum = reinterpret_cast<float2 *>(list + (size_t)B * per * n);
  WarpRoom &room = reinterpret_cast<WarpRoom *>(sum + B * per)[threadIdx.x >> 5];
  const int64_t g = blockIdx.x;
  const bool raw = a.dm.mode == RVQ_BEAM_RAW;
  ptx::griddep_launch_dependents();
  for (int i = threadIdx.x >> 5; i < B * per; i += warps) {
    const int64_t row = g * B + i / per;
    if (!beam_live(a, row)) continue;
    const CutRow<T> in(static_cast<const T *>(a.logits) + row * a.stride, a.dm.vocab);
    float m, s;
    beam_pieces<T, kLane * (int)sizeof(T) / 16, PARTS>(in, i % per, per, n, raw, raw ? a.scores[row] : 0.f, room, m, s);
    if (!raw) s = warp_sum(s);
    if (lane == 0) sum[i] = make_float2(m, s);
    for (int j = lane; j < n; j += 32) list[i * n + j] = room.best[j];
    __syncwarp();
  }
  __syncthreads();
  join_group(a, g, list, sum, per, join);
}

// `splits` blocks per row; each leaves its best entries and its part of the sum.
// 256 rows of 65536 bf16 (34 MB, 5 us of bandwidth) take 21 us here and 6 to 9
// in the join: a warp reads its 4096 elements at once and then works on them
// alone.  Half as many vectors a warp and twice the blocks took 25 us.
template <class T, int PARTS>
__global__ void __launch_bounds__(32 * kRowWarps) k_beam_rows(const BeamArgs a) {
  __shared__ WarpRoom room[kRowWarps];
  __shared__ uint64_t all[kRowWarps * kBeamMax];
  __shared__ float2 sums[kRowWarps];
  __shared__ uint64_t bar;
  __shared__ int count;
  const int n = a.dm.select, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool raw = a.dm.mode == RVQ_BEAM_RAW;
  const int64_t row = blockIdx.x / a.splits;
  const int split = (int)(blockIdx.x % a.splits);
  ptx::griddep_launch_dependents();
  if (!beam_live(a, row)) return;
  const CutRow<T> in(static_cast<const T *>(a.logits) + row * a.stride, a.dm.vocab);
  float m, s;
  beam_pieces<T, kRowVectors, PARTS>(in, split * kRowWarps + warp, a.splits * kRowWarps, n, raw,
                                     raw ? a.scores[row] : 0.f, room[warp], m, s);
  if (!raw) s = warp_sum(s);
  if (lane == 0) sums[warp] = make_float2(m, s);
  if (threadIdx.x == 0) bar = 0, count = 0;
  __syncthreads();
  // the best of the warps' last entries is a bar that n entries reach
  if (threadIdx.x < kRowWarps && room[threadIdx.x].best[n - 1])
    atomicMax(reinterpret_cast<unsigned long long *>(&bar), (unsigned long long)room[threadIdx.x].best[n - 1]);
  __syncthreads();
  for (int i = lane; i < n; i += 32) {
    const uint64_t k = room[warp].best[i];
    if (k && k >= bar) all[atomicAdd(&count, 1)] = k;
  }
  __syncthreads();
  const int c = count;
  uint64_t *out = a.parts.list + blockIdx.x * (int64_t)n;
  for (int i = threadIdx.x; i < c; i += blockDim.x) {
    int place = 0;
    for (int j = 0; j < c; ++j) place += all[j] > all[i];
    if (place < n) out[place] = all[i];
  }
  for (int j = c + threadIdx.x; j < n; j += blockDim.x) out[j] = 0;
  if (threadIdx.x == 0 && !raw) {
    for (int w = 1; w < kRowWarps; ++w) join_sum(sums[0].x, sums[0].y, sums[w].x, sums[w].y);
    a.parts.sum[blockIdx.x] = sums[0];
  }
}

__global__ void __launch_bounds__(256) k_beam_join(const BeamArgs a) {
  extern __shared__ uint64_t smem[];
  __shared__ Join join;
  const int lists = a.dm.beams * a.splits, n = a.dm.select;
  const int64_t g = blockIdx.x;
  float2 *sum = reinterpret_cast<float2 *>(smem + (size_t)lists * n);
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const auto *from = reinterpret_cast<const unsigned long long *>(a.parts.list) + g * lists * n;
  for (int i = threadIdx.x; i < lists * n; i += blockDim.x) smem[i] = __ldcg(from + i);
  for (int i = threadIdx.x; i < lists; i += blockDim.x) sum[i] = __ldcg(a.parts.sum + g * lists + i);
  __syncthreads();
  join_group(a, g, smem, sum, a.splits, join);
}

// ---------------------------------------------------------------------------
// reordering
// ---------------------------------------------------------------------------

struct StateList {
  rvq_beam_state s[RVQ_BEAM_MAX_STATES];
};

// A block per (layer, group) and piece of the row, all slots of the group: a
// parent that several slots have is read from memory once.  W: the widest word
// that the state's addresses allow; `pieces` of `words` words a row.
constexpr int kMoveThreads = 256, kMoveDepth = 4;
template <class W>
__device__ __forceinline__ void move_rows(const rvq_beam_state &s, const int32_t *parents, int64_t layer, int64_t g,
                                          int beams, int select, int64_t piece, int piece_words) {
  const int64_t words = s.row_bytes / (int64_t)sizeof(W), w0 = piece * piece_words;
  if (w0 >= words) return;
  const uint32_t here = (uint32_t)min((int64_t)piece_words, words - w0), all = here * (uint32_t)select;
  const char *src = static_cast<const char *>(s.src) + layer * s.src_layer_stride + g * s.src_group_stride + w0 * sizeof(W);
  char *dst = static_cast<char *>(s.dst) + layer * s.dst_layer_stride + g * s.dst_group_stride + w0 * sizeof(W);
  for (uint32_t i0 = threadIdx.x; i0 < all; i0 += kMoveThreads * kMoveDepth) {
    W v[kMoveDepth];
#pragma unroll
    for (int k = 0; k < kMoveDepth; ++k) {
      const uint32_t i = i0 + k * kMoveThreads;
      v[k] = W{};
      if (i < all) {
        const uint32_t j = i / here;
        const int p = parents[g * select + j];
        if (p >= 0 && p < beams) v[k] = reinterpret_cast<const W *>(src + p * s.src_beam_stride)[i - j * here];
      }
    }
#pragma unroll
    for (int k = 0; k < kMoveDepth; ++k) {
      const uint32_t i = i0 + k * kMoveThreads;
      if (i < all) {
        const uint32_t j = i / here;
        reinterpret_cast<W *>(dst + j * s.dst_beam_stride)[i - j * here] = v[k];
      }
    }
  }
}

__host__ __device__ inline int state_word(const rvq_beam_state &s) {
  const uintptr_t all = reinterpret_cast<uintptr_t>(s.src) | reinterpret_cast<uintptr_t>(s.dst) | (uintptr_t)s.row_bytes |
                        (uintptr_t)s.src_layer_stride | (uintptr_t)s.src_group_stride | (uintptr_t)s.src_beam_stride |
                        (uintptr_t)s.dst_layer_stride | (uintptr_t)s.dst_group_stride | (uintptr_t)s.dst_beam_stride;
  return (all & 15) == 0 ? 16 : (all & 3) == 0 ? 4 : 1;
}
// Words of a row that a block moves for each slot: 256 (4 KB; 2 KB measured 110
// against 90 us at 4 x 16 x 8 rows of 768 KB), more where there are few slots,
// fewer while the blocks do not fill the GPU.
inline int move_words(int select, int64_t rows, int64_t words) {
  int w = select < kMoveDepth ? kMoveThreads * kMoveDepth / select : kMoveThreads;
  while (w > 32 && rows * ((words + w - 1) / w) < 2 * 152) w /= 2;
  return w;
}

__global__ void __launch_bounds__(kMoveThreads)
    k_beam_reorder(const __grid_constant__ StateList list, const int32_t *parents, int64_t groups, int beams,
                   int select, int piece_words) {
  const rvq_beam_state &s = list.s[blockIdx.z];
  const int word = state_word(s);
  const int64_t pieces = (s.row_bytes / word + piece_words - 1) / piece_words;
  ptx::griddep_wait();
  for (int64_t lg = blockIdx.y; lg < s.layers * groups; lg += gridDim.y) {
    int64_t layer = 0, g = lg;
    if (s.layers > 1) layer = lg / groups, g = lg - layer * groups;
    for (int64_t piece = blockIdx.x; piece < pieces; piece += gridDim.x) {
      if (word == 16)
        move_rows<uint4>(s, parents, layer, g, beams, select, piece, piece_words);
      else if (word == 4)
        move_rows<uint32_t>(s, parents, layer, g, beams, select, piece, piece_words);
      else
        move_rows<uint8_t>(s, parents, layer, g, beams, select, piece, piece_words);
    }
  }
}

// In place: a block takes one piece of all beams' rows of a group through
// shared memory, W bytes a lane at a time.
template <class W>
__global__ void __launch_bounds__(kMoveThreads)
    k_beam_reorder_in_place(const __grid_constant__ StateList list, const int32_t *parents, int64_t groups,
                            int beams) {
  constexpr int kCols = 32;
  __shared__ W tile[kBeamMax][kCols];
  const rvq_beam_state s = list.s[blockIdx.z];
  ptx::griddep_wait();  // by every block: a grid that ended without it would let the next one start too early
  if (state_word(s) != (int)sizeof(W)) return;
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

// A kernel that may be brought up while the one before it on the stream ends:
// it waits (griddep_wait) before it reads or writes anything.  What the kernel
// before it writes (the parents, the lists) is no read-only data of this one: its
// pointers are neither __restrict__ nor read by the non-coherent path.
template <class... P, class... A>
cudaError_t launch_next(void (*kernel)(P...), dim3 grid, int block, size_t smem, cudaStream_t st, const A &...args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

rvq_status check_beam(const rvq_beam_dims &dm) {
  if (dm.groups < 0 || dm.beams <= 0 || dm.vocab <= 0 || dm.select <= 0 || !dtype_bytes(dm.dtype)) return RVQ_ERR_INVALID_ARG;
  if (dm.mode != RVQ_BEAM_LOGITS && dm.mode != RVQ_BEAM_RAW) return RVQ_ERR_INVALID_ARG;
  if (dm.beams > kBeamMax || dm.select > kBeamMax || dm.vocab > kBeamMaxVocab) return RVQ_ERR_UNSUPPORTED;
  if (dm.groups > (int64_t)(1 << 30) / kMaxLists) return RVQ_ERR_UNSUPPORTED;
  return RVQ_OK;
}

// How a call runs.  A group of at most kGroupItems pieces: one block, `splits`
// warps a row.  Else `splits` blocks a row: as many as fill the GPU, none
// without a piece for each of its warps.
struct BeamPlan {
  bool group;
  int splits, warps;
  size_t smem;
};
BeamPlan beam_plan(const rvq_beam_dims &dm) {
  // whole vectors alone make pieces: the elements beside them go with the first
  const int vec = 16 / dtype_bytes(dm.dtype), each = 32 * kLane / vec, full = dm.vocab / vec;
  const int pieces = full > each ? (full + each - 1) / each : 1;
  BeamPlan p{};
  p.group = (int64_t)dm.beams * pieces <= kGroupItems;
  if (p.group) {
    const int per = kGroupWarps / dm.beams;
    p.splits = per < 1 ? 1 : per > pieces ? pieces : per;
    p.warps = dm.beams * p.splits < kGroupWarps ? dm.beams * p.splits : kGroupWarps;
    p.smem = (size_t)dm.beams * p.splits * (dm.select * 8 + sizeof(float2)) + p.warps * sizeof(WarpRoom);
    return p;
  }
  const int64_t rows = dm.groups * dm.beams;
  int64_t s = rows > 0 ? (2 * 152 + rows - 1) / rows : 1;
  const int block = 32 * kRowVectors * kRowWarps, most = full > block ? (full + block - 1) / block : 1;
  s = s > most ? most : s;
  s = s > kMaxLists / dm.beams ? kMaxLists / dm.beams : s;
  p.splits = (int)s;
  p.warps = kRowWarps;
  p.smem = (size_t)dm.beams * p.splits * (dm.select * 8 + sizeof(float2));
  return p;
}

RowSet source_rows(const rvq_beam_dims &dm, const rvq_beam_state &s) {
  return {s.src, s.row_bytes, {{s.layers, s.src_layer_stride}, {dm.groups, s.src_group_stride}, {dm.beams, s.src_beam_stride}}};
}
RowSet target_rows(const rvq_beam_dims &dm, const rvq_beam_state &s) {
  return {s.dst, s.row_bytes, {{s.layers, s.dst_layer_stride}, {dm.groups, s.dst_group_stride}, {dm.select, s.dst_beam_stride}}};
}

// Blocks take rows in any order, and the states of a call at the same time: what
// one writes must meet nothing else that is written, and nothing that is read
// but the source of a move by the state that a later kernel reorders in place.
rvq_status check_states(const rvq_beam_dims &dm, const int32_t *parents, const StateList &move, int moves,
                        const StateList &swap, int swaps) {
  bool some = false, unknown = false;
  auto apart = [&](Overlap o) { some |= o == Overlap::kSome, unknown |= o == Overlap::kUnknown; };
  const int n = moves + swaps;
  auto state = [&](int i) -> const rvq_beam_state & { return i < moves ? move.s[i] : swap.s[i - moves]; };
  const RowSet from = row_set(parents, dm.groups * dm.select * (int64_t)sizeof(int32_t), 1, 0);
  for (int i = 0; i < n && !some; ++i) {
    const RowSet to = target_rows(dm, state(i));
    apart(overlaps_itself(to));
    apart(overlap(to, from));
    for (int j = 0; j < moves; ++j)
      if (i < moves) apart(overlap(to, source_rows(dm, state(j))));
    for (int j = i + 1; j < n; ++j) apart(overlap(to, target_rows(dm, state(j))));
  }
  return some ? RVQ_ERR_INVALID_ARG : unknown ? RVQ_ERR_UNSUPPORTED : RVQ_OK;
}

size_t beam_list_at(const rvq_beam_dims &dm, int splits) {
  return align_up((size_t)(dm.groups * dm.beams) * splits * sizeof(float2));
}

// Groups are chosen in any order: what one writes must meet nothing that another
// still reads.  Over the scores and flags that they come from, the outputs must
// be a group's own.
rvq_status check_outputs(const BeamArgs &a, bool group, const void *workspace, size_t workspace_bytes) {
  const rvq_beam_dims &dm = a.dm;
  const int64_t held = dm.groups * dm.beams, kept = dm.groups * dm.select;
  auto flat = [](const void *p, int64_t bytes) { return row_set(p, bytes, 1, 0); };
  const RowSet out[5] = {flat(a.out_scores, kept * 4), flat(a.parents, kept * 4), flat(a.codes, kept * 4),
                         flat(a.out_finished, a.out_finished ? kept : 0),
                         flat(workspace, group ? 0 : (int64_t)workspace_bytes)};
  const RowSet in[3] = {flat(a.scores, held * 4), flat(a.finished, a.finished ? held : 0),
                        row_set(a.logits, (int64_t)dm.vocab * dtype_bytes(dm.dtype), held, a.stride * dtype_bytes(dm.dtype))};
  const bool own = dm.select == dm.beams;
  for (int i = 0; i < 5; ++i) {
    if (out[i].row == 0) continue;
    for (int j = i + 1; j < 5; ++j)
      if (out[j].row && overlap(out[i], out[j]) != Overlap::kNone) return RVQ_ERR_INVALID_ARG;
    for (int j = 0; j < 3; ++j) {
      if (own && ((i == 0 && j == 0) || (i == 3 && j == 1)) && out[i].base == in[j].base) continue;
      if (in[j].row && overlap(out[i], in[j]) != Overlap::kNone) return RVQ_ERR_INVALID_ARG;
    }
  }
  return RVQ_OK;
}

std::atomic<bool> g_join_allowed[64];
template <class T, int PARTS>
cudaError_t launch_beam(const BeamArgs &a, const BeamPlan &p, cudaStream_t st) {
  if (p.group) {
    static std::atomic<bool> allowed[64];
    const auto kernel = k_beam_group<T, PARTS>;
    const cudaError_t e = p.smem > 24 * 1024 ? allow_smem(kernel, allowed) : cudaSuccess;
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)a.dm.groups, 32 * p.warps, p.smem, st>>>(a);
    return cudaGetLastError();
  }
  k_beam_rows<T, PARTS><<<(unsigned)(a.dm.groups * a.dm.beams * p.splits), 32 * kRowWarps, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && p.smem > 24 * 1024) e = allow_smem(k_beam_join, g_join_allowed);
  if (e != cudaSuccess) return e;
  return launch_next(k_beam_join, dim3((unsigned)a.dm.groups), 256, p.smem, st, a);
}
template <class T>
cudaError_t launch_beam(const BeamArgs &a, const BeamPlan &p, cudaStream_t st) {
  return a.dm.select <= 32 ? launch_beam<T, 2>(a, p, st) : launch_beam<T, 4>(a, p, st);
}

}  // namespace
}  // namespace rvq

extern "C" {

RVQ_API size_t rvq_beam_workspace_bytes(rvq_beam_dims dims) {
  using namespace rvq;
  if (check_beam(dims) != RVQ_OK) return 0;
  const BeamPlan p = beam_plan(dims);
  if (p.group || dims.groups == 0) return kAlign;  // nothing but the size's own sign that the dims are supported
  return beam_list_at(dims, p.splits) + align_up((size_t)(dims.groups * dims.beams) * p.splits * dims.select * 8);
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
  const BeamPlan p = beam_plan(dims);
  const BeamArgs a{dims, logits, logits_stride, scores, finished, end_code, out_scores, parents, codes, out_finished,
                   p.splits, {at<float2>(workspace, 0), at<uint64_t>(workspace, beam_list_at(dims, p.splits))}};
  const rvq_status apart = check_outputs(a, p.group, workspace, rvq_beam_workspace_bytes(dims));
  if (apart != RVQ_OK) return apart;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dims.dtype == RVQ_DTYPE_F32    ? launch_beam<float>(a, p, st)
                        : dims.dtype == RVQ_DTYPE_BF16 ? launch_beam<__nv_bfloat16>(a, p, st)
                                                       : launch_beam<__half>(a, p, st);
  return e == cudaSuccess ? RVQ_OK : RVQ_ERR_CUDA;
}

RVQ_API rvq_status rvq_beam_reorder(rvq_beam_dims dims, const int32_t *parents, const rvq_beam_state *states,
                                    int32_t n_states, rvq_stream_t stream) {
  using namespace rvq;
  const rvq_status c = check_beam(dims);
  if (c != RVQ_OK) return c;
  if (n_states < 0 || n_states > RVQ_BEAM_MAX_STATES || (n_states > 0 && !states)) return RVQ_ERR_INVALID_ARG;
  StateList move, swap;
  int moves = 0, swaps = 0;
  int64_t rows = 0, longest = 0, pieces = 0;
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
      const int w = state_word(s);
      wide[w == 16 ? 0 : w == 4 ? 1 : 2] = true;
      const int64_t p = s.layers * dims.groups * ((s.row_bytes / w + 31) / 32);
      pieces = p > pieces ? p : pieces;
    } else {
      move.s[moves++] = s;
      const int64_t across = s.row_bytes / state_word(s);
      rows = s.layers * dims.groups > rows ? s.layers * dims.groups : rows;
      longest = across > longest ? across : longest;
    }
  }
  if (moves + swaps == 0) return RVQ_OK;
  if (!parents || !aligned_to(parents, 4)) return RVQ_ERR_INVALID_ARG;
  const rvq_status apart = check_states(dims, parents, move, moves, swap, swaps);
  if (apart != RVQ_OK) return apart;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (moves) {
    // neighbouring blocks take neighbouring pieces
    const int words = move_words(dims.select, rows, longest);
    const int64_t most = (longest + words - 1) / words;
    const dim3 grid((unsigned)(most < (1 << 24) ? most : (1 << 24)), (unsigned)(rows < 65535 ? rows : 65535),
                    (unsigned)moves);
    if (launch_next(k_beam_reorder, grid, kMoveThreads, 0, st, move, parents, dims.groups, dims.beams, dims.select,
                    words) != cudaSuccess)
      return RVQ_ERR_CUDA;
  }
  if (swaps) {
    const dim3 grid((unsigned)(pieces < (1 << 16) ? pieces : (1 << 16)), 1, (unsigned)swaps);
    cudaError_t e = cudaSuccess;
    if (wide[0])
      e = launch_next(k_beam_reorder_in_place<uint4>, grid, kMoveThreads, 0, st, swap, parents, dims.groups, dims.beams);
    if (e == cudaSuccess && wide[1])
      e = launch_next(k_beam_reorder_in_place<uint32_t>, grid, kMoveThreads, 0, st, swap, parents, dims.groups,
                      dims.beams);
    if (e == cudaSuccess && wide[2])
      e = launch_next(k_beam_reorder_in_place<uint8_t>, grid, kMoveThreads, 0, st, swap, parents, dims.groups,
                      dims.beams);
    if (e != cudaSuccess) return RVQ_ERR_CUDA;
  }
  return RVQ_OK;
}

}  // extern "C"
