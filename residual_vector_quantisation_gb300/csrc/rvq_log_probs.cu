// Log probabilities of given codes, with the entropy of their distributions and
// the best alternatives (rvq_log_probs), and their gradient
// (rvq_log_probs_backward).
//
// With y = (z - m) log2(e) / T, m the row's largest logit, one read of the row
// gives s = sum 2^y and a = sum 2^y y (the running largest value as m: a larger
// one scales both), and from them
//   log p[c] = (z_c - m) / T - ln s,   H = ln s - ln 2 * a / s,   lse = m / T + ln s.
// Both terms of H are positive: they do not cancel.  (s holds the largest code's
// own 1: what the others have together below 2^-24 is rounded away in it and in
// ln s, so that of rows that are nearly certain H keeps its second term alone and
// is right to 2^-24 absolutely.)  The gradient needs no sum:
//   dz_j = (2^y_j (k0 + k1 y_j) + [j = c] g) / T.
#include "rvq_internal.cuh"
#include "rvq_overlap.h"
#include "rvq_top.cuh"
#include "sm103_ptx.cuh"

namespace rvq {
namespace {

constexpr int kMaxVocab = 1 << 20;
constexpr float kLn2 = 0.693147180559945309f;
// Below this y counts as this: 2^y is 0 there, and 2^y y has to be 0 for a mask's -inf too.
constexpr float kLowest = -200.f;

struct LogProbsArgs {
  rvq_log_probs_dims dm;
  const void *logits;
  int64_t stride;
  const int32_t *codes;
  float *log_probs, *entropy, *lse, *stats, *top_log_probs;
  int32_t *top_codes;
  int64_t *bad_codes;
  // backward
  const float *stats_in, *entropy_in, *grad_log_probs, *grad_entropy, *grad_lse;
  void *dlogits;
  int64_t dlogits_stride;
  float inv_t, c;  // 1 / T and log2(e) / T
};

// The larger one, NaN where one is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The sums of part of a row.
struct Tally {
  float m, s, a;
};
__device__ __forceinline__ Tally no_tally() { return {-CUDART_INF_F, 0.f, 0.f}; }
// The same sums relative to a larger value.
__device__ __forceinline__ Tally raise(Tally t, float m, float c) {
  const float at = m == -CUDART_INF_F ? 0.f : m;
  const float d = max_nan((t.m - at) * c, kLowest), f = exp2_fast(d);
  return {m, t.s * f, (t.a + t.s * d) * f};
}
__device__ __forceinline__ Tally warp_join(Tally v, float c) {
  const float m = warp_max_order(v.m);
  v = raise(v, m, c);
  return {m, warp_sum(v.s), warp_sum(v.a)};
}

// Adds values to a tally, relative to its m.  (ENT false: a is not wanted.)
template <bool ENT>
struct Adder {
  F2 minus, c2, s, a;
  __device__ __forceinline__ Adder(float m, float c) {
    m = m == -CUDART_INF_F ? 0.f : m;
    minus = f2(-m, -m), c2 = f2(c, c), s = a = f2(0.f, 0.f);
  }
  __device__ __forceinline__ void pair(F2 z) {
    float2 y = floats((z + minus) * c2);
    if constexpr (ENT) {
      y.x = max_nan(y.x, kLowest), y.y = max_nan(y.y, kLowest);
      const F2 e = f2(exp2_fast(y.x), exp2_fast(y.y));
      s = s + e;
      a = fma2(e, f2(y.x, y.y), a);
    } else {
      s = s + f2(exp2_fast(y.x), exp2_fast(y.y));
    }
  }
  template <class T>
  __device__ __forceinline__ void vector(const uint4 &v) {
    F2 f[8 / sizeof(T)];
    unpack_pairs<T>(v, f);
#pragma unroll
    for (int i = 0; i < 8 / (int)sizeof(T); ++i) pair(f[i]);
  }
  __device__ __forceinline__ float sum(F2 v) const {
    const float2 p = floats(v);
    return p.x + p.y;
  }
};

// A row's results from its tally: one thread.
template <class T>
__device__ __forceinline__ void put_row(const LogProbsArgs &a, int64_t row, const T *z, Tally t) {
  const float log_s = logf(t.s);  // -inf: nothing has a probability
  if (a.lse) a.lse[row] = t.s == 0.f ? -CUDART_INF_F : __fdiv_rn(t.m, a.dm.temperature) + log_s;
  if (a.entropy) a.entropy[row] = t.s == 0.f ? 0.f : log_s - kLn2 * __fdiv_rn(t.a, t.s);
  if (a.stats) a.stats[2 * row] = t.m, a.stats[2 * row + 1] = t.s;
  if (a.codes == nullptr) return;
  const int code = a.codes[row];
  const bool there = code >= 0 && code < a.dm.vocab;
  if (a.bad_codes && code != -1 && !there) atomicAdd(reinterpret_cast<unsigned long long *>(a.bad_codes), 1ull);
  a.log_probs[row] = !there ? 0.f : t.s == 0.f ? -CUDART_INF_F : (to_float(z[code]) - t.m) * a.inv_t - log_s;
}
// Place i of its alternatives.
__device__ __forceinline__ void put_top(const LogProbsArgs &a, int64_t row, int i, uint64_t key, Tally t, float log_s) {
  const int64_t at = row * a.dm.top + i;
  a.top_codes[at] = key ? (int)~(uint32_t)key : -1;
  a.top_log_probs[at] = key ? (value_of((uint32_t)(key >> 32)) - t.m) * a.inv_t - log_s : -CUDART_INF_F;
}

template <class T>
__device__ __forceinline__ CutRow<T> row_of(const LogProbsArgs &a, int64_t row) {
  return CutRow<T>(static_cast<const T *>(a.logits) + row * a.stride, a.dm.vocab);
}

// ---------------------------------------------------------------------------
// a row in a warp
// ---------------------------------------------------------------------------

constexpr int kRowWarps = 4;  // of a block

// Bound by instructions: 439 a row of 1025 codes, 180 of them for the elements (a
// power, its sum and its product with the exponent), the rest for two sums, the
// edges and the results.  60 000 x 1025 bf16: 31 us (bytes alone: 18).
template <class T, int NV, bool ENT>
__global__ void __launch_bounds__(32 * kRowWarps) k_log_probs(const LogProbsArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x * (int64_t)kRowWarps + (threadIdx.x >> 5);
  if (row >= a.dm.rows) return;
  const CutRow<T> r = row_of<T>(a, row);
  uint4 raw[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) raw[j] = lane + j * 32 < r.full ? r.vector(lane + j * 32) : all_low<T>();
  const int edge_at = r.edge(lane);
  const float edge = edge_at >= 0 ? to_float(r.z[edge_at]) : -CUDART_INF_F;
  float m = edge;
#pragma unroll
  for (int j = 0; j < NV; ++j) m = fmaxf(m, largest_of<T>(raw[j]));
  m = warp_max_order(m);
  Adder<ENT> sums(m, a.c);
#pragma unroll
  for (int j = 0; j < NV; ++j) sums.template vector<T>(raw[j]);
  sums.pair(f2(edge, -CUDART_INF_F));
  const Tally t = {m, warp_sum(sums.sum(sums.s)), ENT ? warp_sum(sums.sum(sums.a)) : 0.f};
  if (lane == 0) put_row(a, row, r.z, t);
}

// With the best alternatives: 1200 instructions a row of 1024 codes and 16 kept,
// two thirds of them for finding the bar, reading again what reaches it and
// ordering it.  384 000 x 1024 f32: 510 us (bytes alone: 239), with registers held
// down for 8 blocks an SM; 546 as the compiler would have it (72 registers).
template <class T>
__global__ void __launch_bounds__(32 * kRowWarps, 8) k_log_probs_top(const LogProbsArgs a) {
  constexpr int NV = 32 * (int)sizeof(T) / 16;
  __shared__ WarpRoom room[kRowWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = a.dm.top;
  const int64_t row = blockIdx.x * (int64_t)kRowWarps + warp;
  if (row >= a.dm.rows) return;
  const CutRow<T> r = row_of<T>(a, row);
  Tally t = no_tally();
  warp_pieces<T, NV, 4>(r, 0, 1, n, 0.f, room[warp], [&](const uint4 (&z)[NV], float edge, float high) {
    // (one piece: nothing to raise)
    t.m = warp_max_order(high);
    Adder<true> sums(t.m, a.c);
#pragma unroll
    for (int j = 0; j < NV; ++j) sums.template vector<T>(z[j]);
    sums.pair(f2(edge, -CUDART_INF_F));
    t.s = sums.sum(sums.s), t.a = sums.sum(sums.a);
  });
  t.s = warp_sum(t.s), t.a = warp_sum(t.a);
  if (lane == 0) put_row(a, row, r.z, t);
  const float log_s = logf(t.s);
  for (int i = lane; i < n; i += 32) put_top(a, row, i, room[warp].best[i], t, log_s);
}

// ---------------------------------------------------------------------------
// a row in a block, or in a cluster of them
// ---------------------------------------------------------------------------

constexpr int kMaxWarps = 16, kMaxCluster = 8;

// All blocks of the cluster have come here; what they wrote before is seen after.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The row's tally, in every thread of the cluster's first block (`box`: of a
// block's warps; `parts`: in the first block, the blocks' tallies).  An arrival of
// all blocks has to be under way: this waits for it (they have all started, and
// may be written to) and ends with the next barrier, so that what a block wrote
// into the first one's memory after that arrival is there too.
__device__ __forceinline__ Tally row_tally(Tally v, float c, Tally *box, Tally *parts, int rank, int cs) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  v = warp_join(v, c);
  if (lane == 0) box[threadIdx.x >> 5] = v;
  __syncthreads();
  v = warp_join(lane < warps ? box[lane] : no_tally(), c);
  if (cs == 1) return v;
  cluster_wait();
  if (threadIdx.x == 0) {
    const uint32_t to = ptx::cluster_map((uint32_t)__cvta_generic_to_shared(parts + rank), 0);
    ptx::st_cluster_f32(to, v.m), ptx::st_cluster_f32(to + 4, v.s), ptx::st_cluster_f32(to + 8, v.a);
  }
  cluster_arrive();
  cluster_wait();
  return rank == 0 ? warp_join(lane < cs ? parts[lane] : no_tally(), c) : v;
}

// Each thread raises its own largest value as it goes; U vectors of it are under
// way while U are added.  Bound by bandwidth: with the gradient's kernel 241 us for
// 4096 x 65536 bf16 (98 % of a copy's rate).
template <class T, bool ENT>
__global__ void __launch_bounds__(32 * kMaxWarps) k_log_probs_row(const LogProbsArgs a, const int cs) {
  constexpr int U = 4;
  __shared__ Tally box[kMaxWarps], parts[kMaxCluster];
  const int64_t row = blockIdx.x / (unsigned)cs;
  const int rank = cs == 1 ? 0 : (int)ptx::cluster_ctarank();
  if (cs > 1) cluster_arrive();
  const CutRow<T> r = row_of<T>(a, row);
  const int step = cs * blockDim.x, first = rank * blockDim.x + threadIdx.x;
  uint4 raw[U];
  auto load = [&](int v0) {
#pragma unroll
    for (int j = 0; j < U; ++j) raw[j] = v0 + j * step < r.full ? r.vector(v0 + j * step) : all_low<T>();
  };
  load(first);
  const int edge_at = rank == 0 ? r.edge(threadIdx.x) : -1;
  Tally t = no_tally();
  if (edge_at >= 0) {
    const float edge = to_float(r.z[edge_at]);
    t.m = fmaxf(edge, t.m);
    Adder<ENT> sums(t.m, a.c);
    sums.pair(f2(edge, -CUDART_INF_F));
    t.s = sums.sum(sums.s), t.a = sums.sum(sums.a);
  }
  for (int v0 = first; v0 < r.full; v0 += U * step) {
    float most = t.m;
#pragma unroll
    for (int j = 0; j < U; ++j) most = fmaxf(most, largest_of<T>(raw[j]));
    if (most > t.m) t = raise(t, most, a.c);
    Adder<ENT> sums(t.m, a.c);
#pragma unroll
    for (int j = 0; j < U; ++j) sums.template vector<T>(raw[j]);
    load(v0 + U * step);
    t.s += sums.sum(sums.s);
    if constexpr (ENT) t.a += sums.sum(sums.a);
  }
  t = row_tally(t, a.c, box, parts, rank, cs);
  if (rank == 0 && threadIdx.x == 0) put_row(a, row, r.z, t);
}

// The best n of `lists` ordered lists of n entries each, `stride` apart, by the
// block: put(place, entry) for each of them; returns their number.
struct ListRoom {
  uint64_t all[kMaxWarps * kMostKept];
  unsigned long long bar;
  int count;
};
template <class F>
__device__ __forceinline__ int join_lists(const uint64_t *list, int stride, int lists, int n, ListRoom &w, F put) {
  if (threadIdx.x == 0) w.bar = 0, w.count = 0;
  __syncthreads();
  // the best of the lists' last entries is a bar that n entries reach
  if ((int)threadIdx.x < lists) {
    const uint64_t last = list[(int)threadIdx.x * stride + n - 1];
    if (last) atomicMax(&w.bar, (unsigned long long)last);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < lists * n; i += blockDim.x) {
    const uint64_t k = list[i / n * stride + i % n];
    if (k && k >= w.bar) w.all[atomicAdd(&w.count, 1)] = k;
  }
  __syncthreads();
  const int c = w.count;
  for (int i = threadIdx.x; i < c; i += blockDim.x) {
    const uint64_t k = w.all[i];
    int place = 0;
    for (int j = 0; j < c; ++j) place += w.all[j] > k;
    if (place < n) put(place, k);
  }
  return min(c, n);
}

// With the best alternatives: each warp orders its pieces, the block the warps'
// lists, the cluster's first block the blocks'.  6 rows of 65536 f16 with 32 kept
// take 18 us over 8 blocks a row: latency of one piece's ordering and two joins.
// 4096 rows of 65536 bf16 with 16 kept take 387 us (bytes alone: 79), with 64 kept
// 11.3 ms: of 100 pieces 7 have more entries above the bar than there is room for.
template <class T, int NV>
__global__ void __launch_bounds__(32 * kMaxWarps) k_log_probs_row_top(const LogProbsArgs a, const int cs) {
  extern __shared__ uint64_t smem[];
  __shared__ Tally box[kMaxWarps], parts[kMaxCluster];
  __shared__ uint64_t gathered[kMaxCluster * kMostKept];
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, n = a.dm.top;
  ListRoom &lists = *reinterpret_cast<ListRoom *>(smem);
  WarpRoom *room = reinterpret_cast<WarpRoom *>(smem + sizeof(ListRoom) / 8);
  const int64_t row = blockIdx.x / (unsigned)cs;
  const int rank = cs == 1 ? 0 : (int)ptx::cluster_ctarank();
  if (cs > 1) cluster_arrive();
  const CutRow<T> r = row_of<T>(a, row);
  Tally t = no_tally();
  warp_pieces<T, NV, 4>(r, rank * warps + warp, cs * warps, n, 0.f, room[warp],
                     [&](const uint4 (&z)[NV], float edge, float high) {
                       const float m = fmaxf(t.m, warp_max_order(high));
                       t = raise(t, m, a.c);
                       Adder<true> sums(m, a.c);
#pragma unroll
                       for (int j = 0; j < NV; ++j) sums.template vector<T>(z[j]);
                       sums.pair(f2(edge, -CUDART_INF_F));
                       t.s += sums.sum(sums.s), t.a += sums.sum(sums.a);
                     });
  __syncthreads();
  if (cs > 1) {  // the first block has started: the lists go into its memory before row_tally's barrier
    cluster_wait();
    cluster_arrive();
  }
  const uint32_t to = cs > 1 ? ptx::cluster_map((uint32_t)__cvta_generic_to_shared(gathered + rank * n), 0) : 0;
  auto put = [&](int place, uint64_t k) {
    if (cs > 1)
      ptx::st_cluster_v2u32(to + 8 * place, (uint32_t)k, (uint32_t)(k >> 32));
    else
      gathered[place] = k;
  };
  const int found = join_lists(room[0].best, (int)(sizeof(WarpRoom) / 8), warps, n, lists, put);
  for (int i = found + threadIdx.x; i < n; i += blockDim.x) put(i, 0);
  t = row_tally(t, a.c, box, parts, rank, cs);
  if (rank != 0) return;
  if (threadIdx.x == 0) put_row(a, row, r.z, t);
  const float log_s = logf(t.s);
  if (cs == 1) {
    for (int i = threadIdx.x; i < n; i += blockDim.x) put_top(a, row, i, gathered[i], t, log_s);
    return;
  }
  const int all = join_lists(gathered, n, cs, n, lists, [&](int place, uint64_t k) { put_top(a, row, place, k, t, log_s); });
  for (int i = all + threadIdx.x; i < n; i += blockDim.x) put_top(a, row, i, 0, t, log_s);
}

// ---------------------------------------------------------------------------
// the gradient
// ---------------------------------------------------------------------------

constexpr int kBackWarps = 8;

// A warp per piece of a row (`pieces` of NV vectors a lane each).  60 000 x 1025
// bf16 with the entropy's gradient: 42 us (bytes alone: 36), 491 instructions a row.
template <class T, int NV, bool ENT>
__global__ void __launch_bounds__(32 * kBackWarps) k_log_probs_backward(const LogProbsArgs a, const int pieces) {
  constexpr int N = 16 / (int)sizeof(T);
  const int lane = threadIdx.x & 31;
  const int64_t item = blockIdx.x * (int64_t)kBackWarps + (threadIdx.x >> 5);
  const int64_t row = pieces == 1 ? item : item / pieces;
  const int piece = (int)(item - row * pieces);
  if (row >= a.dm.rows) return;
  const CutRow<T> r = row_of<T>(a, row);
  T *d = static_cast<T *>(a.dlogits) + row * a.dlogits_stride;
  const int v0 = piece * NV * 32 + lane;
  uint4 raw[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (v0 + j * 32 < r.full) raw[j] = r.vector(v0 + j * 32);
  const int edge_at = piece == 0 ? r.edge(lane) : -1;
  const float edge = edge_at >= 0 ? to_float(r.z[edge_at]) : 0.f;
  int code = a.codes ? a.codes[row] : -1;
  float g = a.grad_log_probs ? a.grad_log_probs[row] : 0.f;
  const float gh = ENT ? a.grad_entropy[row] : 0.f, gl = a.grad_lse ? a.grad_lse[row] : 0.f;
  const float m = a.stats_in[2 * row], s = a.stats_in[2 * row + 1], entropy = ENT ? a.entropy_in[row] : 0.f;
  if (code < 0 || code >= a.dm.vocab) code = -1, g = 0.f;
  // no gradient reaches the row, or nothing in it has a probability
  const bool zero = (g == 0.f && gh == 0.f && gl == 0.f) || s == 0.f;
  const float scale = __fdividef(1.f, s), at_code = zero ? 0.f : g * a.inv_t;
  const float k0 = (gl - g - (ENT ? gh * (entropy - logf(s)) : 0.f)) * scale, k1 = -gh * kLn2 * scale;
  const F2 minus = f2(-m, -m), c2 = f2(a.c, a.c), k0s = f2(k0, k0), k1s = f2(k1, k1), inv_t = f2(a.inv_t, a.inv_t);
  auto grad = [&](F2 z) {
    const F2 p = (z + minus) * c2;
    float2 y = floats(p);
    if constexpr (ENT) y.x = max_nan(y.x, kLowest), y.y = max_nan(y.y, kLowest);
    const F2 e = f2(exp2_fast(y.x), exp2_fast(y.y));
    return (ENT ? e * fma2(k1s, f2(y.x, y.y), k0s) : e * k0s) * inv_t;  // (1 / T last: a power of 0 stays 0)
  };
  const bool same = ((reinterpret_cast<uintptr_t>(r.z) ^ reinterpret_cast<uintptr_t>(d)) & 15) == 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = v0 + j * 32;
    if (v >= r.full) continue;
    float f[N] = {};
    if (!zero) {
      F2 z[N / 2];
      unpack_pairs<T>(raw[j], z);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const float2 g2 = floats(grad(z[i]));
        f[2 * i] = g2.x, f[2 * i + 1] = g2.y;
      }
    }
    const int first = r.head + v * N;
    if (code >= first && code < first + N)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (code == first + i) f[i] += at_code;
    if (same) {
      *reinterpret_cast<uint4 *>(d + first) = pack16<T>(f);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) d[first + i] = from_float<T>(f[i]);
    }
  }
  if (edge_at >= 0)
    d[edge_at] = from_float<T>((zero ? 0.f : floats(grad(f2(edge, edge))).x) + (edge_at == code ? at_code : 0.f));
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

template <class... P, class... A>
cudaError_t launch_cluster(void (*kernel)(P...), int64_t rows, int cs, int block, size_t smem, cudaStream_t st,
                           const A &...args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(rows * cs));
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cs, at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cs > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// How a row of `full` vectors lies: over a cluster of blocks where there are
// fewer rows than SMs, each with two warps of `each` vectors a lane at least; over
// at most 512 threads of a block.
struct RowPlan {
  int blocks, threads;
};
inline RowPlan row_plan(int64_t rows, int full, int each) {
  int cs = 1, threads = 64;
  while (cs < kMaxCluster && rows * cs * 2 <= 152 && full >= cs * 2 * 64 * each) cs *= 2;
  while (threads < 32 * kMaxWarps && cs * threads * each < full) threads *= 2;
  return {cs, threads};
}

template <class T, int NV>
cudaError_t launch_warp(const LogProbsArgs &a, cudaStream_t st) {
  const unsigned blocks = (unsigned)((a.dm.rows + kRowWarps - 1) / kRowWarps);
  if (a.entropy)
    k_log_probs<T, NV, true><<<blocks, 32 * kRowWarps, 0, st>>>(a);
  else
    k_log_probs<T, NV, false><<<blocks, 32 * kRowWarps, 0, st>>>(a);
  return cudaGetLastError();
}

template <class T>
cudaError_t launch_forward(const LogProbsArgs &a, cudaStream_t st) {
  constexpr int N = 16 / (int)sizeof(T), NV = 32 / N;  // vectors of 32 elements
  const int full = a.dm.vocab / N;
  if (full <= 32 * NV) {  // a warp's registers
    if (a.dm.top) {
      k_log_probs_top<T><<<(unsigned)((a.dm.rows + kRowWarps - 1) / kRowWarps), 32 * kRowWarps, 0, st>>>(a);
      return cudaGetLastError();
    }
    switch ((full + 32 * (NV / 4) - 1) / (32 * (NV / 4))) {
      case 0:
      case 1: return launch_warp<T, NV / 4>(a, st);
      case 2: return launch_warp<T, NV / 2>(a, st);
      case 3: return launch_warp<T, NV / 4 * 3>(a, st);
      default: return launch_warp<T, NV>(a, st);
    }
  }
  if (a.dm.top) {
    constexpr int kEach = 8;
    const RowPlan p = row_plan(a.dm.rows, full, kEach);
    const size_t smem = sizeof(ListRoom) + p.threads / 32 * sizeof(WarpRoom);
    const auto kernel = k_log_probs_row_top<T, kEach>;
    static std::atomic<bool> allowed[64];
    const cudaError_t e = allow_smem(kernel, allowed);
    if (e != cudaSuccess) return e;
    return launch_cluster(kernel, a.dm.rows, p.blocks, p.threads, smem, st, a, p.blocks);
  }
  const RowPlan p = row_plan(a.dm.rows, full, 4);
  return launch_cluster(a.entropy ? k_log_probs_row<T, true> : k_log_probs_row<T, false>, a.dm.rows, p.blocks, p.threads, 0,
                        st, a, p.blocks);
}

template <class T>
cudaError_t launch_backward(const LogProbsArgs &a, cudaStream_t st) {
  constexpr int N = 16 / (int)sizeof(T), NV = 4;
  const int full = a.dm.vocab / N, pieces = full > 0 ? (full + 32 * NV - 1) / (32 * NV) : 1;
  const unsigned blocks = (unsigned)((a.dm.rows * pieces + kBackWarps - 1) / kBackWarps);
  if (a.grad_entropy)
    k_log_probs_backward<T, NV, true><<<blocks, 32 * kBackWarps, 0, st>>>(a, pieces);
  else
    k_log_probs_backward<T, NV, false><<<blocks, 32 * kBackWarps, 0, st>>>(a, pieces);
  return cudaGetLastError();
}

// Rows go to the grid's first axis, at most 2^30 blocks of a launch.
cudaError_t launch_log_probs(LogProbsArgs a, bool backward, cudaStream_t st) {
  a.inv_t = 1.f / a.dm.temperature, a.c = kLog2e * a.inv_t;
  const int64_t rows = a.dm.rows;
  const int e = dtype_bytes(a.dm.dtype);
  const int64_t most = ((int64_t)1 << 30) / (backward ? (a.dm.vocab + 127) / 128 : kMaxCluster);
  for (int64_t r0 = 0; r0 < rows; r0 += most) {
    LogProbsArgs b = a;
    b.dm.rows = rows - r0 < most ? rows - r0 : most;
    auto skip = [&](auto &p, int64_t n) {
      if (p) p += n;
    };
    b.logits = static_cast<const char *>(a.logits) + r0 * a.stride * e;
    if (a.dlogits) b.dlogits = static_cast<char *>(a.dlogits) + r0 * a.dlogits_stride * e;
    skip(b.codes, r0), skip(b.log_probs, r0), skip(b.entropy, r0), skip(b.lse, r0), skip(b.stats, 2 * r0);
    skip(b.top_log_probs, r0 * a.dm.top), skip(b.top_codes, r0 * a.dm.top), skip(b.stats_in, 2 * r0);
    skip(b.entropy_in, r0), skip(b.grad_log_probs, r0), skip(b.grad_entropy, r0), skip(b.grad_lse, r0);
    cudaError_t err;
    switch (a.dm.dtype) {
      case RVQ_DTYPE_F32: err = backward ? launch_backward<float>(b, st) : launch_forward<float>(b, st); break;
      case RVQ_DTYPE_BF16: err = backward ? launch_backward<__nv_bfloat16>(b, st) : launch_forward<__nv_bfloat16>(b, st); break;
      default: err = backward ? launch_backward<__half>(b, st) : launch_forward<__half>(b, st);
    }
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

rvq_status check_log_probs(const LogProbsArgs &a) {
  const rvq_log_probs_dims &dm = a.dm;
  const int e = dtype_bytes(dm.dtype);
  if (dm.rows < 0 || dm.vocab <= 0 || dm.top < 0 || !e) return RVQ_ERR_INVALID_ARG;
  constexpr float kMost = 3.402823466e38f;  // of a temperature, and of what launch_log_probs makes of it
  if (!(dm.temperature > 0.f) || dm.temperature > kMost || !(kLog2e * (1.f / dm.temperature) <= kMost))
    return RVQ_ERR_INVALID_ARG;
  if (dm.vocab > kMaxVocab || dm.top > kMostKept) return RVQ_ERR_UNSUPPORTED;
  if (dm.rows == 0) return RVQ_OK;
  if (!a.logits || !aligned_to(a.logits, e) || (dm.rows > 1 && a.stride < dm.vocab)) return RVQ_ERR_INVALID_ARG;
  for (const void *p : {(const void *)a.codes, (const void *)a.log_probs, (const void *)a.entropy, (const void *)a.lse,
                        (const void *)a.stats, (const void *)a.top_log_probs, (const void *)a.top_codes,
                        (const void *)a.stats_in, (const void *)a.entropy_in, (const void *)a.grad_log_probs,
                        (const void *)a.grad_entropy, (const void *)a.grad_lse})
    if (!aligned_to(p, 4)) return RVQ_ERR_INVALID_ARG;
  return aligned_to(a.bad_codes, 8) ? RVQ_OK : RVQ_ERR_INVALID_ARG;
}

// Whether the outputs meet one another or an input (a set at null is none).
template <int W, int R>
bool all_apart(const RowSet (&written)[W], const RowSet (&read)[R]) {
  for (int i = 0; i < W; ++i) {
    if (!written[i].base) continue;
    for (int j = i + 1; j < W; ++j)
      if (written[j].base && overlap(written[i], written[j]) != Overlap::kNone) return false;
    for (const RowSet &r : read)
      if (r.base && overlap(written[i], r) != Overlap::kNone) return false;
  }
  return true;
}
inline RowSet bytes_at(const void *p, int64_t n) { return row_set(p, n, 1, 0); }

}  // namespace
}  // namespace rvq

extern "C" {

RVQ_API rvq_status rvq_log_probs(rvq_log_probs_dims dims, const void *logits, int64_t logits_stride,
                                 const int32_t *codes, float *log_probs, float *entropy, float *lse, float *stats,
                                 float *top_log_probs, int32_t *top_codes, int64_t *bad_codes, rvq_stream_t stream) {
  using namespace rvq;
  LogProbsArgs a{};
  a.dm = dims, a.logits = logits, a.stride = logits_stride, a.codes = codes, a.log_probs = log_probs;
  a.entropy = entropy, a.lse = lse, a.stats = stats, a.top_log_probs = top_log_probs, a.top_codes = top_codes;
  a.bad_codes = bad_codes;
  const rvq_status s = check_log_probs(a);
  if (s != RVQ_OK || dims.rows == 0) return s;
  if ((log_probs == nullptr) != (codes == nullptr) || (top_log_probs == nullptr) != (dims.top == 0) ||
      (top_codes == nullptr) != (dims.top == 0) || (!log_probs && !entropy && !lse && !stats && !dims.top))
    return RVQ_ERR_INVALID_ARG;
  const int64_t n = dims.rows * 4, e = dtype_bytes(dims.dtype);
  const RowSet written[] = {bytes_at(log_probs, n), bytes_at(entropy, n), bytes_at(lse, n), bytes_at(stats, 2 * n),
                            bytes_at(top_log_probs, dims.top * n), bytes_at(top_codes, dims.top * n),
                            bytes_at(bad_codes, 8)};
  const RowSet read[] = {row_set(logits, dims.vocab * e, dims.rows, logits_stride * e), bytes_at(codes, n)};
  if (!all_apart(written, read)) return RVQ_ERR_INVALID_ARG;
  return launch_log_probs(a, false, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? RVQ_OK : RVQ_ERR_CUDA;
}

RVQ_API rvq_status rvq_log_probs_backward(rvq_log_probs_dims dims, const float *grad_log_probs,
                                          const float *grad_entropy, const float *grad_lse, const void *logits,
                                          int64_t logits_stride, const int32_t *codes, const float *stats,
                                          const float *entropy, void *dlogits, int64_t dlogits_stride,
                                          rvq_stream_t stream) {
  using namespace rvq;
  LogProbsArgs a{};
  a.dm = dims, a.logits = logits, a.stride = logits_stride, a.codes = codes, a.stats_in = stats, a.entropy_in = entropy;
  a.grad_log_probs = grad_log_probs, a.grad_entropy = grad_entropy, a.grad_lse = grad_lse;
  a.dlogits = dlogits, a.dlogits_stride = dlogits_stride;
  const rvq_status s = check_log_probs(a);
  if (s != RVQ_OK || dims.rows == 0) return s;
  const int64_t n = dims.rows * 4, e = dtype_bytes(dims.dtype);
  if (!stats || !dlogits || !aligned_to(dlogits, (uintptr_t)e) || (dims.rows > 1 && dlogits_stride < dims.vocab) ||
      (grad_log_probs && !codes) || (grad_entropy && !entropy))
    return RVQ_ERR_INVALID_ARG;
  // blocks take rows in any order: the gradient may lie over the logits row by row
  if (!rows_apart(dlogits, dlogits_stride * e, logits, logits_stride * e, dims.rows, dims.vocab * e))
    return RVQ_ERR_INVALID_ARG;
  const RowSet written[] = {row_set(dlogits, dims.vocab * e, dims.rows, dlogits_stride * e)};
  const RowSet read[] = {bytes_at(grad_log_probs, n), bytes_at(grad_entropy, n), bytes_at(grad_lse, n),
                         bytes_at(codes, n), bytes_at(stats, 2 * n), bytes_at(entropy, n)};
  if (!all_apart(written, read)) return RVQ_ERR_INVALID_ARG;
  return launch_log_probs(a, true, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? RVQ_OK : RVQ_ERR_CUDA;
}

}  // extern "C"
