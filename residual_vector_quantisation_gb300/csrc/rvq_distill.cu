// Distillation from a teacher's top logits, forward and backward (rvq_distill,
// rvq_distill_backward).
//
// Per row: the sum of the student's exponentials, the teacher's few entries,
// the loss, and the gradient
//   on the list   w / T (p_j - q_j)
//   off the list  w / T p_v                        (q renormalised)
//                 w / T p_v (p_r - q_r) / p_r      (with the tail bucket).
// With the tail the row's sum is taken over the codes without an entry only (a
// bit per code marks the entries) and the entries are added to it: p_r is then
// a sum, not 1 minus a sum, and keeps its digits when the list holds nearly
// everything.
#include "rvq_internal.cuh"
#include "rvq_overlap.h"
#include "rvq_rows.cuh"

namespace rvq {
namespace {

constexpr int kDistillMaxVocab = 1 << 20;
constexpr int kDistillMaxTop = 256;  // a power of two
constexpr float kTailFloor = 9.5367431640625e-07f;  // 2^-20: a smaller 1 - sum q is that sum's rounding

struct DistillArgs {
  rvq_distill_dims dm;
  const void *logits;
  int64_t logits_stride;
  const void *top_logits;
  const int32_t *top_codes;
  const float *teacher_lse, *weights, *grad_loss;
  float *loss, *sums;       // of the forward pass
  const float *sums_in;     // of the backward pass alone
  void *dlogits;
  int64_t dlogits_stride;
  int64_t *bad_codes;
  float inv_t, c;  // 1 / T and log2(e) / T
};

__device__ __forceinline__ float load_any(const void *p, int32_t dtype, int64_t i) {
  if (dtype == RVQ_DTYPE_F32) return static_cast<const float *>(p)[i];
  if (dtype == RVQ_DTYPE_BF16) return to_float(static_cast<const __nv_bfloat16 *>(p)[i]);
  return to_float(static_cast<const __half *>(p)[i]);
}

// A sum of e^(z / T) as s * e^(m / T), m the largest z (a row of the type's
// lowest values has a sum like any other: z - m is taken before the scale).
// c = log2(e) / T throughout.
struct Sum {
  float m, s;
};
__device__ __forceinline__ Sum no_sum() { return {-CUDART_INF_F, 0.f}; }
__device__ __forceinline__ float share(float z, float m, float c) { return exp2_fast((z - m) * c); }
__device__ __forceinline__ Sum join(Sum a, Sum b, float c) {
  const float m = fmaxf(a.m, b.m), at = m == -CUDART_INF_F ? 0.f : m;
  return {m, a.s * share(a.m, at, c) + b.s * share(b.m, at, c)};
}
__device__ __forceinline__ Sum warp_join(Sum v, float c) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
    v = join(v, {__shfl_xor_sync(0xffffffffu, v.m, o), __shfl_xor_sync(0xffffffffu, v.s, o)}, c);
  return v;
}

// A row of logits and where its gradient goes.  Element e has place e - head +
// 8: a vector's places start at a multiple of N.
template <class T>
struct Row : CutRow<T> {
  using CutRow<T>::N, CutRow<T>::z, CutRow<T>::head;
  T *d;       // null: no gradient wanted
  bool same;  // z and d start equally far from a boundary
  __device__ __forceinline__ Row(const DistillArgs &a, int64_t row)
      : CutRow<T>(static_cast<const T *>(a.logits) + row * a.logits_stride, a.dm.vocab),
        d(a.dlogits ? static_cast<T *>(a.dlogits) + row * a.dlogits_stride : nullptr) {
    same = ((reinterpret_cast<uintptr_t>(z) ^ reinterpret_cast<uintptr_t>(d)) & 15) == 0;
  }
  __device__ __forceinline__ int place(int e) const { return e - head + 8; }
  __device__ __forceinline__ void put(int v, const float (&f)[N]) const {
    T *at = d + head + v * N;
    if (same) {
      *reinterpret_cast<uint4 *>(at) = pack16<T>(f);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) at[i] = from_float<T>(f[i]);
    }
  }
};

// The bits that mark the codes with an entry.  By owner (rows in registers): a
// word per thread, bit j * N + i for element i of its j-th vector, and a word
// for the elements beside the vectors, a bit per thread.  By place (long rows):
// a bit per element, place e - head + 8.
struct Spot {
  int word;
  uint32_t bit;
};
template <class T>
__device__ __forceinline__ Spot spot(const Row<T> &r, int e, int log_threads) {
  constexpr int N = Row<T>::N;
  if (log_threads < 0) return {r.place(e) >> 5, 1u << (r.place(e) & 31)};
  const int k = e - r.head, v = k / N;
  if (k >= 0 && v < r.full)
    return {v & ((1 << log_threads) - 1), 1u << ((v >> log_threads) * N + (k & (N - 1)))};
  return {1 << log_threads, 1u << (e < r.head ? e : N + k - r.full * N)};
}
inline int distill_words(int vocab, int threads) { return threads ? threads + 1 : (vocab + 8 + 31) / 32; }

// A row's entries: code (-1: empty), the teacher's logit t, the student's z;
// of one warp, in its registers (SMALL: at most 32) or in shared memory.
template <bool SMALL>
struct TopList {
  uint32_t *bits;
  int32_t *codes;
  float *ts, *zs;
  int code;
  float t, z;  // SMALL
  __device__ __forceinline__ TopList(uint32_t *at, int words, int top) : bits(at) {
    codes = reinterpret_cast<int32_t *>(at + words);
    ts = reinterpret_cast<float *>(codes + top), zs = ts + top;
    code = -1;
  }
  template <class F>
  __device__ __forceinline__ void each(int top, F f) const {
    if constexpr (SMALL) {
      f(code, t, z);
    } else {
#pragma unroll 1
      for (int j = threadIdx.x & 31; j < top; j += 32) f(codes[j], ts[j], zs[j]);
    }
  }
};
inline size_t distill_smem(int words, int top, bool small) { return (size_t)(words + (small ? 0 : 3 * top)) * 4; }

// The lane's first entry, asked for before anything else of the row is known.
struct FirstEntry {
  int code;
  float t;
  __device__ __forceinline__ FirstEntry(const DistillArgs &a, int64_t row) {
    const int lane = threadIdx.x & 31;
    const bool there = lane < a.dm.top;
    code = there ? a.top_codes[row * a.dm.top + lane] : -1;
    t = there ? load_any(a.top_logits, a.dm.top_dtype, row * a.dm.top + lane) : -CUDART_INF_F;
  }
};

// One warp reads a row's entries (bits cleared before).  An entry counts where
// its code is in range and stands for the first time, by the list's order.
template <class T, bool SMALL>
__device__ __forceinline__ void read_top(const DistillArgs &a, int64_t row, const Row<T> &r, int log_threads,
                                         const FirstEntry &first, TopList<SMALL> &l) {
  const int lane = threadIdx.x & 31, top = a.dm.top;
  int bad = 0;
#pragma unroll 1
  for (int j0 = 0; j0 < top; j0 += 32) {
    const int j = j0 + lane;
    int code = first.code;
    float t = first.t;
    if (!SMALL && j0) {
      code = j < top ? a.top_codes[row * top + j] : -1;
      t = j < top ? load_any(a.top_logits, a.dm.top_dtype, row * top + j) : -CUDART_INF_F;
    }
    bool ok = code >= 0 && code < a.dm.vocab, seen = false;
    const float z = ok ? to_float(r.z[code]) : -CUDART_INF_F;
    if (ok) {
      const Spot p = spot(r, code, log_threads);
      seen = atomicOr(&l.bits[p.word], p.bit) & p.bit;
    }
    const unsigned all_seen = __ballot_sync(0xffffffffu, seen);
    if (all_seen) {  // a code twice: the first of its lanes has it, unless an earlier 32 had
      const unsigned same = __match_any_sync(0xffffffffu, ok ? code : -1 - lane);
      ok = ok && __ffs(same) - 1 == lane && (same & ~all_seen);
    }
    bad += code != -1 && !ok;
    code = ok ? code : -1;
    t = ok ? t : -CUDART_INF_F;
    if constexpr (SMALL) {
      l.code = code, l.t = t, l.z = ok ? z : -CUDART_INF_F;
      break;
    } else {
      if (j < top) l.codes[j] = code, l.ts[j] = t, l.zs[j] = ok ? z : -CUDART_INF_F;
      __syncwarp();
    }
  }
  if (a.bad_codes && __any_sync(0xffffffffu, bad)) {
    bad = __reduce_add_sync(0xffffffffu, bad);
    if (lane == 0) atomicAdd(reinterpret_cast<unsigned long long *>(a.bad_codes), (unsigned long long)bad);
  }
}

// What the list alone gives, relative to the list's largest logits (t_m, z_m):
//   u_j = q_j (with the tail) or e^((t_j - t_m) / T) (renormalised: q_j = u_j / u),
//   u = sum u_j,  on = sum e^((z_j - z_m) / T),
//   ul = sum u_j ((t_j - t_m) / T - t_log - (z_j - z_m) / T) / kMaxTop (which
//   keeps the sum in range while any u_j of it is).
// Logarithms of single entries are natural ones: a logit of the type's lowest
// value, times log2(e), would be -inf.
struct TopSums {
  bool any;
  float t_m, t_log, z_m, on, u, ul;
};
__device__ __forceinline__ float entry_u(const TopSums &r, float t, float inv_t) {
  return exp2_fast(fmaf(t - r.t_m, inv_t, -r.t_log) * kLog2e);
}

template <bool SMALL>
__device__ __forceinline__ TopSums top_sums(const DistillArgs &a, float teacher_lse, const TopList<SMALL> &l) {
  const bool tail = a.teacher_lse != nullptr;
  const float inv_t = a.inv_t;
  TopSums r;
  bool any = false;
  float tm = -CUDART_INF_F, zm = -CUDART_INF_F;
  l.each(a.dm.top, [&](int code, float t, float z) {  // empty entries are -inf
    any |= code >= 0;
    tm = fmaxf(tm, t);
    zm = fmaxf(zm, z);
  });
  r.any = __any_sync(0xffffffffu, any);
  zm = warp_max_order(zm);
  r.z_m = zm == -CUDART_INF_F ? 0.f : zm;
  if (tail) {
    r.t_m = 0.f, r.t_log = teacher_lse;
  } else {
    tm = warp_max_order(tm);
    r.t_m = tm == -CUDART_INF_F ? 0.f : tm, r.t_log = 0.f;
  }
  r.on = r.u = r.ul = 0.f;
  l.each(a.dm.top, [&](int code, float t, float z) {
    if (code < 0) return;
    const float zr = (z - r.z_m) * inv_t, lt = fmaf(t - r.t_m, inv_t, -r.t_log);
    const float u = exp2_fast(lt * kLog2e);
    r.on += exp2_fast(zr * kLog2e);
    r.u += u;
    if (u != 0.f) r.ul = fmaf(u * (1.f / kDistillMaxTop), lt - zr, r.ul);  // a NaN goes on
  });
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    if (tail) r.on += __shfl_xor_sync(0xffffffffu, r.on, o);
    r.u += __shfl_xor_sync(0xffffffffu, r.u, o);
    r.ul += __shfl_xor_sync(0xffffffffu, r.ul, o);
  }
  return r;
}

// What the gradient needs of a row: off the list e^((z - m) / T) * rest_scale
// (`zero`: nothing), on it (e^((z - all_m) / T) * all_r - u_j * u_r) * scale.
struct RowPlan {
  float m, rest_scale, scale, loss, all_m, all_r, u_r;
  bool zero;
};

// The plan from `sum`, the sum over every code (renormalised) or over the
// codes without an entry (with the tail).
__device__ __forceinline__ RowPlan plan_row(bool tail, float w, Sum sum, const TopSums &t, float c, float inv_t) {
  const Sum all = tail && t.any ? join(sum, {t.z_m, t.on}, c) : sum;
  RowPlan r{sum.m, 0.f, w * inv_t, 0.f, all.m, 0.f, 1.f, false};
  if (!t.any || (!tail && t.u == 0.f)) {
    r.scale = 0.f;
    r.zero = true;
    return r;
  }
  const float log_all = logf(all.s);
  if (all.s != 0.f) r.all_r = __fdividef(1.f, all.s);
  // sum q_j (log q_j - log p_j), log p_j = log_p + (z_j - z_m) / T
  const float log_p = all.s == 0.f ? -CUDART_INF_F : (t.z_m - all.m) * inv_t - log_all;
  float loss;
  if (tail) {
    loss = t.u == 0.f ? 0.f : fmaf(-t.u, log_p, t.ul * kDistillMaxTop);
  } else {
    r.u_r = __fdividef(1.f, t.u);
    loss = t.ul * r.u_r * kDistillMaxTop - logf(t.u) - log_p;
  }
  if (t.u != t.u) loss = r.scale = t.u;
  r.rest_scale = __fdividef(r.scale, sum.s);
  if (tail) {
    float q_rest = 1.f - t.u;
    if (q_rest <= kTailFloor) q_rest = 0.f;
    // log q_r - log p_r, p_r = (sum.s / all.s) e^((sum.m - all.m) / T)
    const float ratio = sum.s == 0.f ? CUDART_INF_F
                                     : logf(__fdividef(q_rest * all.s, sum.s)) - (sum.m - all.m) * inv_t;
    if (q_rest != 0.f) loss = fmaf(q_rest, ratio, loss);
    r.rest_scale *= sum.s * share(sum.m, all.m, c) * r.all_r - q_rest;
  }
  if (sum.s == 0.f) r.m = 0.f, r.rest_scale = 0.f;  // no code off the list has a share
  r.loss = loss * w;
  return r;
}

// The entries' gradients, over what was written in their place.
template <class T, bool SMALL>
__device__ __forceinline__ void put_top(const DistillArgs &a, const Row<T> &r, const RowPlan &p, const TopSums &ts,
                                        const TopList<SMALL> &l) {
  l.each(a.dm.top, [&](int code, float t, float z) {
    if (code < 0) return;
    const float on = p.all_r == 0.f ? 0.f : share(z, p.all_m, a.c) * p.all_r;
    r.d[code] = from_float<T>(p.scale == 0.f ? 0.f : (on - entry_u(ts, t, a.inv_t) * p.u_r) * p.scale);
  });
}

// e^((z - m) / T).  m is subtracted first: as 2^(z c - m c), one operation less,
// the product m c would have to be exact (masks of -1e9 and of the type's
// lowest value are large ms).
struct Power {
  float m, c;
  F2 minus, c2;
  __device__ __forceinline__ Power(float m_, float c_) {
    m = m_ == -CUDART_INF_F ? 0.f : m_;
    c = c_;
    minus = f2(-m, -m), c2 = f2(c, c);
  }
  __device__ __forceinline__ float operator()(float z) const { return exp2_fast((z - m) * c); }
  template <class T>
  __device__ __forceinline__ void operator()(const uint4 &v, float (&e)[16 / sizeof(T)]) const {
    F2 f[8 / sizeof(T)];
    unpack_pairs<T>(v, f);
#pragma unroll
    for (int i = 0; i < 8 / (int)sizeof(T); ++i) {
      const float2 y = floats((f[i] + minus) * c2);
      e[2 * i] = exp2_fast(y.x), e[2 * i + 1] = exp2_fast(y.y);
    }
  }
};
// A vector of a gradient: the powers times `factor`.
template <class T>
__device__ __forceinline__ void put_scaled(const Row<T> &r, int v, float (&e)[16 / sizeof(T)], F2 factor) {
#pragma unroll
  for (int i = 0; i < 8 / (int)sizeof(T); ++i) {
    const float2 y = floats(f2(e[2 * i], e[2 * i + 1]) * factor);
    e[2 * i] = y.x, e[2 * i + 1] = y.y;
  }
  r.put(v, e);
}

// A thread's share of a row in registers: the vectors t, t + threads, ... and
// perhaps an edge element.
template <class T, int NV>
struct Share {
  static constexpr int N = 16 / (int)sizeof(T);
  float e[NV][N], edge;
  int edge_at;
  uint4 raw[NV];
  __device__ __forceinline__ void load(const Row<T> &r, int t, int threads) {
#pragma unroll
    for (int j = 0; j < NV; ++j) raw[j] = t + j * threads < r.full ? r.vector(t + j * threads) : all_low<T>();
    edge_at = r.edge(t);
    edge = edge_at >= 0 ? to_float(r.z[edge_at]) : -CUDART_INF_F;
  }
  __device__ __forceinline__ float most() const {
    float m = edge;
#pragma unroll
    for (int j = 0; j < NV; ++j) m = fmaxf(m, largest_of<T>(raw[j]));
    return m;
  }
  // The powers in place of the values; the sum of those without a bit (in `skip` and, for the edge, `skip_edge`).
  __device__ __forceinline__ float powers(const Power &pw, uint32_t skip, bool skip_edge) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      pw.template operator()<T>(raw[j], e[j]);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (!(skip >> (j * N + i) & 1)) s += e[j][i];
    }
    edge = pw(edge);
    return skip_edge ? s : s + edge;  // (without one it is 0)
  }
  __device__ __forceinline__ void put(const Row<T> &r, float factor, int t, int threads) {
    const F2 factors = f2(factor, factor);
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (t + j * threads < r.full) put_scaled(r, t + j * threads, e[j], factors);
    if (edge_at >= 0) r.d[edge_at] = from_float<T>(edge * factor);
  }
};

// The sum over a row's threads: a warp's, or a block's through `box` (after a
// barrier that every earlier use of it has passed).
template <bool WARP>
__device__ __forceinline__ Sum row_join(Sum v, float c, Sum *box) {
  v = warp_join(v, c);
  if constexpr (!WARP) {
    const int lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) box[threadIdx.x >> 5] = v;
    __syncthreads();
    v = warp_join(lane < (int)blockDim.x >> 5 ? box[lane] : no_sum(), c);
  }
  return v;
}

// The sum over the codes without an entry, from its own largest value: where
// the entries hold all but 1e-25 of the row.
template <class T, bool WARP>
__device__ __noinline__ Sum small_rest(const Row<T> &r, const uint32_t *bits, int log_threads, int t, int threads,
                                       float c, Sum *box) {
  Sum sum = no_sum();
  for (int e = t; e < r.width; e += threads) {
    const Spot p = spot(r, e, log_threads);
    const float z = to_float(r.z[e]);
    if (!(bits[p.word] & p.bit)) sum = join(sum, {z, z == -CUDART_INF_F ? 0.f : 1.f}, c);
  }
  return row_join<WARP>(sum, c, box);
}
constexpr float kSmallRest = 1e-25f;

// A gradient of zeros, and a row without weight: thread t of `threads`.
template <class T>
__device__ __forceinline__ void put_zeros(const Row<T> &r, int t, int threads) {
  const float zero[Row<T>::N] = {};
  for (int v = t; v < r.full; v += threads) r.put(v, zero);
  const int at = r.edge(t);
  if (at >= 0) r.d[at] = from_float<T>(0.f);
}
template <class T>
__device__ __forceinline__ void skip_row(const DistillArgs &a, int64_t row, const Row<T> &r, int t, int threads) {
  if (t == 0 && a.sums_in == nullptr) {
    a.loss[row] = 0.f;
    if (a.sums) a.sums[2 * row] = a.sums[2 * row + 1] = 0.f;
  }
  if (r.d) put_zeros(r, t, threads);
}

// A row in the registers of a warp (WARP: kRowWarps rows a block, no barrier)
// or of a block: one read of the logits, one write of the gradient.
//
// What bounds it: the latency of a row's chain (entries, their logits, two
// reductions) against the rows that an SM holds, so registers are held down to
// let more rows in: for 96 000 rows of 1025 bf16 with 32 entries 110 us as the
// compiler would have it (78 registers, 6 blocks an SM), 100 at 7 and 95 at 8
// blocks; for 384 000 rows of 1024 f32 (two passes) 892 us at 5, 819 at 6, 848
// at 7, 910 at 8 blocks (90 and 814 us since then, with one logarithm fewer a
// row).  The bytes alone would take 59 and 704 us.  Blocks of
// more than 512 threads, for rows above 16384, were slower than two reads (89
// against 73 us for 2000 rows of 30 000 bf16).
constexpr int kRowWarps = 4, kMaxWarps = 16;
template <class T, int NV, bool WARP, bool SMALL>
__global__ void __launch_bounds__(WARP ? 32 * kRowWarps : 32 * kMaxWarps, WARP ? (sizeof(T) == 4 ? 6 : 8) : 1)
    k_distill(const DistillArgs a) {
  extern __shared__ uint32_t smem[];
  __shared__ Sum box[32];
  __shared__ TopSums shared_top;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, top = a.dm.top;
  const int t = WARP ? lane : threadIdx.x, threads = WARP ? 32 : blockDim.x, log_threads = 31 - __clz(threads);
  const int64_t row = WARP ? (int64_t)blockIdx.x * kRowWarps + warp : blockIdx.x;
  if (row >= a.dm.rows) return;
  const bool tail = a.teacher_lse != nullptr, known = a.sums_in != nullptr, lister = WARP || warp == 0;
  const float c = a.c;
  // what does not depend on anything is asked for first
  float w = a.weights ? a.weights[row] : 1.f;
  const float teacher_lse = tail ? a.teacher_lse[row] : 0.f;
  Sum sum = no_sum();
  float up = 1.f;
  if (known) {
    sum = {a.sums_in[2 * row], a.sums_in[2 * row + 1]};
    if (a.grad_loss) up = a.grad_loss[row];
  }
  const FirstEntry first(a, row);
  const Row<T> r(a, row);
  if (w == 0.f) return skip_row(a, row, r, t, threads);
  w *= up;
  Share<T, NV> x;
  x.load(r, t, threads);
  TopList<SMALL> l(smem + (WARP ? (size_t)warp * (33 + (SMALL ? 0 : 3 * top)) : 0), threads + 1, top);
  l.bits[t] = 0;
  if (t == 0) l.bits[threads] = 0;
  TopSums ts;
  if constexpr (WARP) {
    __syncwarp();
    read_top(a, row, r, 5, first, l);
    __syncwarp();
    ts = top_sums(a, teacher_lse, l);
  } else {
    __syncthreads();
    if (lister) {
      read_top(a, row, r, log_threads, first, l);
      __syncwarp();
      ts = top_sums(a, teacher_lse, l);
      if (lane == 0) shared_top = ts;
    }
    __syncthreads();
    ts = shared_top;
  }
  float m = sum.m;
  uint32_t skip = 0;
  bool skip_edge = false;
  if (!known) {
    m = warp_max_order(x.most());
    if (tail) {
      skip = l.bits[t];
      skip_edge = t < 32 && (l.bits[threads] >> t & 1);
    }
  }
  const float s = x.powers(Power(m, c), skip, skip_edge);
  if (!known) {
    if constexpr (WARP) {
      sum = {m, warp_sum(s)};
    } else {
      const float all = warp_sum(s);
      if (lane == 0) box[warp] = {m, all};
      __syncthreads();
      sum = warp_join(lane < threads >> 5 ? box[lane] : no_sum(), c);
    }
    if (tail && sum.s < kSmallRest) {
      sum = small_rest<T, WARP>(r, l.bits, log_threads, t, threads, c, box);
      m = sum.m;
      x.load(r, t, threads);
      x.powers(Power(m, c), 0, false);
    }
  }
  const RowPlan p = plan_row(tail, w, sum, ts, c, a.inv_t);
  if (!known && t == 0) {
    a.loss[row] = p.loss;
    if (a.sums) a.sums[2 * row] = sum.m, a.sums[2 * row + 1] = sum.s;
  }
  if (!r.d) return;
  if (p.zero) return put_zeros(r, t, threads);
  float factor = p.rest_scale;
  if (!WARP && factor != 0.f) factor *= share(m, p.m, c);  // a warp's powers are from its own largest value
  x.put(r, factor, t, threads);
  if constexpr (WARP)
    __syncwarp();
  else
    __syncthreads();
  if (lister) put_top(a, r, p, ts, l);
}

// Longer rows: a row per block, read twice (the second time mostly from the
// L2), U vectors of a thread at a time.  4096 rows of 65536 bf16 take 246 us
// where the bytes alone would take 156: 304 rows are in flight, a third of the
// second reads misses the L2, and fewer rows in flight leave the SMs waiting at
// the rows' ends (one block of 1024 threads an SM: 347 us).
constexpr int kLongThreads = 512;
template <class T, int U, bool SMALL>
__global__ void __launch_bounds__(kLongThreads) k_distill_long(const DistillArgs a) {
  constexpr int N = 16 / (int)sizeof(T);
  extern __shared__ uint32_t smem[];
  __shared__ Sum box[32];
  __shared__ TopSums shared_top;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, threads = blockDim.x;
  const int top = a.dm.top, words = (a.dm.vocab + 8 + 31) / 32;
  const int64_t row = blockIdx.x;
  const Row<T> r(a, row);
  float w = a.weights ? a.weights[row] : 1.f;
  const FirstEntry first(a, row);
  if (w == 0.f) return skip_row(a, row, r, threadIdx.x, threads);
  const bool tail = a.teacher_lse != nullptr, known = a.sums_in != nullptr;
  const float c = a.c;
  uint4 raw[U];
  auto load = [&](int v0) {
#pragma unroll
    for (int j = 0; j < U; ++j) raw[j] = v0 + j * threads < r.full ? r.vector(v0 + j * threads) : all_low<T>();
  };
  load(threadIdx.x);  // on its way while the entries are read
  TopList<SMALL> l(smem, words, top);
  for (int i = threadIdx.x; i < words; i += threads) l.bits[i] = 0;
  __syncthreads();
  if (warp == 0) {
    read_top(a, row, r, -1, first, l);
    __syncwarp();
    const TopSums t = top_sums(a, tail ? a.teacher_lse[row] : 0.f, l);
    if (lane == 0) shared_top = t;
  }
  __syncthreads();
  const TopSums ts = shared_top;
  const int edge = r.edge(threadIdx.x);
  Sum sum;
  if (known) {
    sum = {a.sums_in[2 * row], a.sums_in[2 * row + 1]};
    if (a.grad_loss) w *= a.grad_loss[row];
  } else {
    float m = edge >= 0 ? to_float(r.z[edge]) : -CUDART_INF_F, s = 0.f;
    Power pw(m, c);
    if (edge >= 0) {
      const Spot p = spot(r, edge, -1);
      if (!(tail && (l.bits[p.word] & p.bit))) s = pw(to_float(r.z[edge]));
    }
    for (int v0 = threadIdx.x; v0 < r.full; v0 += U * threads) {
      float most = m;
#pragma unroll
      for (int j = 0; j < U; ++j) most = fmaxf(most, largest_of<T>(raw[j]));
      if (most > m) {
        s *= share(m, most, c);
        m = most;
        pw = Power(m, c);
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int v = v0 + j * threads, at = v * N + 8;
        const uint32_t skip = tail && v < r.full ? l.bits[at >> 5] >> (at & 31) & ((1u << N) - 1) : 0;
        float e[N];
        pw.template operator()<T>(raw[j], e);
        if (skip) {  // rare in a long row
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (skip >> i & 1) e[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) s += e[i];
      }
      load(v0 + U * threads);
    }
    sum = row_join<false>({m, s}, c, box);
    if (tail && sum.s < kSmallRest) sum = small_rest<T, false>(r, l.bits, -1, threadIdx.x, threads, c, box);
  }
  const RowPlan p = plan_row(tail, w, sum, ts, c, a.inv_t);
  if (!known && threadIdx.x == 0) {
    a.loss[row] = p.loss;
    if (a.sums) a.sums[2 * row] = sum.m, a.sums[2 * row + 1] = sum.s;
  }
  if (!r.d) return;
  if (p.zero) return put_zeros(r, threadIdx.x, threads);
  const Power pw(p.m, c);
  const F2 factor = f2(p.rest_scale, p.rest_scale);
  for (int v0 = threadIdx.x; v0 < r.full; v0 += U * threads) {
    load(v0);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (v0 + j * threads >= r.full) continue;
      float e[N];
      pw.template operator()<T>(raw[j], e);
      put_scaled(r, v0 + j * threads, e, factor);
    }
  }
  if (edge >= 0) r.d[edge] = from_float<T>(pw(to_float(r.z[edge])) * p.rest_scale);
  __syncthreads();
  if (warp == 0) put_top(a, r, p, ts, l);
}

// How a row is laid over threads: at most 32 elements of its vectors a thread,
// in a warp or a block of 64 .. 512; above that the two reads (threads 0).
struct DistillShape {
  int threads, vectors;  // of a row; of a thread
};
inline DistillShape distill_shape(int vocab, int n) {
  const int full = vocab / n;
  for (int threads = 32; threads <= 32 * kMaxWarps; threads *= 2) {
    const int each = (full + threads - 1) / threads;
    if (each * n <= 32) return {threads, each > 0 ? each : 1};
  }
  return {0, 1};
}

template <class T, int NV, bool SMALL>
cudaError_t launch_distill_list(const DistillArgs &a, int threads, cudaStream_t st) {
  const size_t smem = distill_smem(distill_words(a.dm.vocab, threads), a.dm.top, SMALL);
  if (threads == 32)
    k_distill<T, NV, true, SMALL>
        <<<(unsigned)((a.dm.rows + kRowWarps - 1) / kRowWarps), 32 * kRowWarps, smem * kRowWarps, st>>>(a);
  else
    k_distill<T, NV, false, SMALL><<<(unsigned)a.dm.rows, threads, smem, st>>>(a);
  return cudaGetLastError();
}
template <class T, int NV>
cudaError_t launch_distill_shape(const DistillArgs &a, int threads, cudaStream_t st) {
  return a.dm.top <= 32 ? launch_distill_list<T, NV, true>(a, threads, st) : launch_distill_list<T, NV, false>(a, threads, st);
}

template <class T>
cudaError_t launch_distill_typed(const DistillArgs &a, cudaStream_t st) {
  constexpr int N = 16 / (int)sizeof(T), U = 8 / N;  // vectors of 8 elements
  const DistillShape s = distill_shape(a.dm.vocab, N);
  if (s.threads) {
    switch ((s.vectors + U - 1) / U) {
      case 1: return launch_distill_shape<T, U>(a, s.threads, st);
      case 2: return launch_distill_shape<T, 2 * U>(a, s.threads, st);
      case 3: return launch_distill_shape<T, 3 * U>(a, s.threads, st);
      default: return launch_distill_shape<T, 4 * U>(a, s.threads, st);
    }
  }
  const auto kernel = a.dm.top <= 32 ? k_distill_long<T, 4, true> : k_distill_long<T, 4, false>;
  const size_t smem = distill_smem(distill_words(a.dm.vocab, 0), a.dm.top, a.dm.top <= 32);
  if (smem > 40 * 1024) {
    static std::atomic<bool> allowed[2][64];
    const cudaError_t e = allow_smem(kernel, allowed[a.dm.top <= 32]);
    if (e != cudaSuccess) return e;
  }
  kernel<<<(unsigned)a.dm.rows, kLongThreads, smem, st>>>(a);
  return cudaGetLastError();
}

// Rows go to the grid's first axis.
constexpr int64_t kDistillMaxRows = ((int64_t)1 << 31) - 8;
cudaError_t launch_distill_rows(const DistillArgs &a, cudaStream_t st) {
  switch (a.dm.dtype) {
    case RVQ_DTYPE_F32: return launch_distill_typed<float>(a, st);
    case RVQ_DTYPE_BF16: return launch_distill_typed<__nv_bfloat16>(a, st);
    default: return launch_distill_typed<__half>(a, st);
  }
}

cudaError_t launch_distill(DistillArgs a, cudaStream_t st) {
  a.inv_t = 1.f / a.dm.temperature, a.c = kLog2e * a.inv_t;
  const int64_t rows = a.dm.rows;
  const int e = dtype_bytes(a.dm.dtype), te = dtype_bytes(a.dm.top_dtype);
  for (int64_t r0 = 0; r0 < rows; r0 += kDistillMaxRows) {
    DistillArgs b = a;
    b.dm.rows = rows - r0 < kDistillMaxRows ? rows - r0 : kDistillMaxRows;
    auto skip = [&](auto &p, int64_t n) {
      if (p) p += n;
    };
    b.logits = static_cast<const char *>(a.logits) + r0 * a.logits_stride * e;
    b.top_logits = static_cast<const char *>(a.top_logits) + r0 * a.dm.top * te;
    b.top_codes += r0 * a.dm.top;
    if (a.dlogits) b.dlogits = static_cast<char *>(a.dlogits) + r0 * a.dlogits_stride * e;
    skip(b.teacher_lse, r0), skip(b.weights, r0), skip(b.grad_loss, r0), skip(b.loss, r0);
    skip(b.sums, 2 * r0), skip(b.sums_in, 2 * r0);
    const cudaError_t err = launch_distill_rows(b, st);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

rvq_status check_distill(const DistillArgs &a) {
  const rvq_distill_dims &dm = a.dm;
  const int e = dtype_bytes(dm.dtype), te = dtype_bytes(dm.top_dtype);
  if (dm.rows < 0 || dm.vocab <= 0 || dm.top <= 0 || !e || !te) return RVQ_ERR_INVALID_ARG;
  constexpr float kMost = 3.402823466e38f;  // of a temperature, and of what launch_distill makes of it
  if (!(dm.temperature > 0.f) || dm.temperature > kMost || !(kLog2e * (1.f / dm.temperature) <= kMost))
    return RVQ_ERR_INVALID_ARG;
  if (dm.vocab > kDistillMaxVocab || dm.top > kDistillMaxTop) return RVQ_ERR_UNSUPPORTED;
  if (dm.rows == 0) return RVQ_OK;
  if (!a.logits || !a.top_logits || !a.top_codes) return RVQ_ERR_INVALID_ARG;
  if (!aligned_to(a.logits, e) || !aligned_to(a.dlogits, e) || !aligned_to(a.top_logits, te)) return RVQ_ERR_INVALID_ARG;
  if (!aligned_to(a.top_codes, 4) || !aligned_to(a.teacher_lse, 4) || !aligned_to(a.weights, 4) ||
      !aligned_to(a.grad_loss, 4) || !aligned_to(a.loss, 4) || !aligned_to(a.sums, 4) || !aligned_to(a.sums_in, 4) ||
      !aligned_to(a.bad_codes, 8))
    return RVQ_ERR_INVALID_ARG;
  if (dm.rows > 1 && (a.logits_stride < dm.vocab || (a.dlogits && a.dlogits_stride < dm.vocab)))
    return RVQ_ERR_INVALID_ARG;
  // blocks take rows in any order
  if (a.dlogits && !rows_apart(a.dlogits, a.dlogits_stride * e, a.logits, a.logits_stride * e, dm.rows, (int64_t)dm.vocab * e))
    return RVQ_ERR_INVALID_ARG;
  return RVQ_OK;
}

}  // namespace
}  // namespace rvq

extern "C" {

RVQ_API rvq_status rvq_distill(rvq_distill_dims dims, const void *logits, int64_t logits_stride,
                               const void *top_logits, const int32_t *top_codes, const float *teacher_lse,
                               const float *weights, float *loss, float *lse, void *dlogits, int64_t dlogits_stride,
                               int64_t *bad_codes, rvq_stream_t stream) {
  const rvq::DistillArgs a{dims, logits, logits_stride, top_logits, top_codes, teacher_lse, weights, nullptr,
                           loss, lse, nullptr, dlogits, dlogits_stride, bad_codes};
  const rvq_status s = rvq::check_distill(a);
  if (s != RVQ_OK || dims.rows == 0) return s;
  if (!loss) return RVQ_ERR_INVALID_ARG;
  return rvq::launch_distill(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? RVQ_OK : RVQ_ERR_CUDA;
}

RVQ_API rvq_status rvq_distill_backward(rvq_distill_dims dims, const float *grad_loss, const void *logits,
                                        int64_t logits_stride, const void *top_logits, const int32_t *top_codes,
                                        const float *teacher_lse, const float *weights, const float *lse,
                                        void *dlogits, int64_t dlogits_stride, rvq_stream_t stream) {
  const rvq::DistillArgs a{dims, logits, logits_stride, top_logits, top_codes, teacher_lse, weights, grad_loss,
                           nullptr, nullptr, lse, dlogits, dlogits_stride, nullptr};
  const rvq_status s = rvq::check_distill(a);
  if (s != RVQ_OK || dims.rows == 0) return s;
  if (!lse || !dlogits) return RVQ_ERR_INVALID_ARG;
  return rvq::launch_distill(a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? RVQ_OK : RVQ_ERR_CUDA;
}

}  // extern "C"
