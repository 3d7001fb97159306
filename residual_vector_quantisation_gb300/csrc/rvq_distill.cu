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
#include "rvq_rows.cuh"

namespace rvq {
namespace {

constexpr int kDistillMaxVocab = 1 << 20;
constexpr int kDistillMaxTop = 256;
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

// What a row's shared memory holds: the bits of the codes with an entry, by
// place (RowVectors), and the entries: code (-1: empty), the teacher's logit t
// and the student's z.
struct TopList {
  uint32_t *bits;
  int32_t *code;
  float *t, *z;
};
__host__ __device__ inline int distill_bit_words(int vocab) { return (vocab + 8 + 31) / 32; }
inline size_t distill_smem(int vocab, int top) { return (size_t)(distill_bit_words(vocab) + 3 * top) * 4; }

// One warp reads a row's entries (bits cleared before).  An entry counts where
// its code is in range and stands for the first time; the order within a warp
// and from warp to warp of 32 is the list's, so the choice does not depend on timing.
template <class T>
__device__ void read_top(const DistillArgs &a, int64_t row, const T *z, int phase, const TopList &l) {
  const int lane = threadIdx.x & 31, top = a.dm.top;
  int bad = 0;
  for (int j0 = 0; j0 < top; j0 += 32) {
    const int j = j0 + lane;
    const int code = j < top ? a.top_codes[row * top + j] : -1;
    bool ok = code >= 0 && code < a.dm.vocab;
    const unsigned same = __match_any_sync(0xffffffffu, ok ? code : -1 - lane);
    ok = ok && __ffs(same) - 1 == lane;
    if (ok) {
      const int p = code + phase;
      const uint32_t bit = 1u << (p & 31);
      ok = !(atomicOr(&l.bits[p >> 5], bit) & bit);
    }
    bad += j < top && code != -1 && !ok;
    if (j < top) {
      l.code[j] = ok ? code : -1;
      l.t[j] = ok ? load_any(a.top_logits, a.dm.top_dtype, row * top + j) : -CUDART_INF_F;
      l.z[j] = ok ? to_float(z[code]) : -CUDART_INF_F;
    }
    __syncwarp();
  }
  if (a.bad_codes && __any_sync(0xffffffffu, bad)) {
    bad = __reduce_add_sync(0xffffffffu, bad);
    if (lane == 0) atomicAdd(reinterpret_cast<unsigned long long *>(a.bad_codes), (unsigned long long)bad);
  }
}

// What the gradient needs of a row: off the list e^((z - rest_m) / T) *
// rest_scale (rest_m = +inf: zero whatever z is), on it (p - q) * scale with
// p = e^((z - all.m) / T) / all.s and log q = (t - t_m) / T - t_log.
struct RowPlan {
  float rest_m, rest_scale, scale, loss, t_m, t_log;
  Sum all;
};
// Logarithms of the entries are natural ones: a logit of the type's lowest
// value, times log2(e), would be -inf.
__device__ __forceinline__ float log_q(const RowPlan &r, float t, float inv_t) {
  return fmaf(t - r.t_m, inv_t, -r.t_log);
}

// One warp: the row's plan from `sum`, the sum over every code (renormalised)
// or over the codes without an entry (with the tail).
__device__ RowPlan plan_row(const DistillArgs &a, int64_t row, float w, Sum sum, float c, const TopList &l) {
  const int lane = threadIdx.x & 31, top = a.dm.top;
  const float inv_t = 1.f / a.dm.temperature;
  const bool tail = a.teacher_lse != nullptr;
  bool any = false;
  Sum t = no_sum(), on = no_sum();
  for (int j = lane; j < top; j += 32) {
    if (l.code[j] < 0) continue;
    any = true;
    if (tail)
      on = join(on, {l.z[j], 1.f}, c);
    else
      t = join(t, {l.t[j], 1.f}, c);
  }
  any = __any_sync(0xffffffffu, any);
  RowPlan r;
  r.scale = w / a.dm.temperature;
  if (tail) {
    r.t_m = 0.f, r.t_log = a.teacher_lse[row];
    r.all = join(sum, warp_join(on, c), c);
  } else {
    t = warp_join(t, c);
    r.t_m = t.m, r.t_log = logf(t.s);
    r.all = sum;
  }
  if (!any || (!tail && t.s == 0.f)) {
    r.loss = r.rest_scale = r.scale = 0.f;
    r.rest_m = CUDART_INF_F;
    return r;
  }
  const bool empty = r.all.m == -CUDART_INF_F && r.all.s == 0.f;  // no code has a share
  const float log_all = logf(r.all.s);
  float q_sum = 0.f, loss = 0.f;
  for (int j = lane; j < top; j += 32) {
    if (l.code[j] < 0) continue;
    const float lq = log_q(r, l.t[j], inv_t), q = exp2_fast(lq * kLog2e);
    const float lp = empty ? -CUDART_INF_F : (l.z[j] - r.all.m) * inv_t - log_all;
    q_sum += q;
    if (q != 0.f) loss = fmaf(q, lq - lp, loss);  // a NaN goes on
  }
  q_sum = warp_sum(q_sum);
  loss = warp_sum(loss);
  r.rest_m = sum.m;
  r.rest_scale = r.scale / sum.s;
  if (tail) {
    float q_rest = 1.f - q_sum;
    if (q_rest <= kTailFloor) q_rest = 0.f;
    const bool none = sum.m == -CUDART_INF_F && sum.s == 0.f;
    const float lp_rest = none ? -CUDART_INF_F : (sum.m - r.all.m) * inv_t + (logf(sum.s) - log_all);
    if (q_rest != 0.f) loss = fmaf(q_rest, logf(q_rest) - lp_rest, loss);
    r.rest_scale *= exp2_fast(lp_rest * kLog2e) - q_rest;
  }
  if (sum.s == 0.f) r.rest_m = CUDART_INF_F, r.rest_scale = 0.f;  // no code off the list has a share
  r.loss = loss * w;
  return r;
}

// Entry j's gradient.
__device__ __forceinline__ float top_grad(const RowPlan &r, float t, float z, float c, float inv_t) {
  if (r.scale == 0.f) return 0.f;
  const float p = r.all.s == 0.f ? 0.f : share(z, r.all.m, c) / r.all.s;
  return (p - exp2_fast(log_q(r, t, inv_t) * kLog2e)) * r.scale;
}

// A row per block, read twice: once for the sum, once for the gradient (the
// second time from the L2).
template <class T>
__global__ void __launch_bounds__(256) k_distill(const DistillArgs a) {
  constexpr int N = 16 / (int)sizeof(T);
  extern __shared__ uint32_t smem[];
  __shared__ Sum box[8];
  __shared__ RowPlan plan;
  const int vocab = a.dm.vocab, top = a.dm.top, words = distill_bit_words(vocab);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const TopList l = {smem, reinterpret_cast<int32_t *>(smem + words), reinterpret_cast<float *>(smem + words + top),
                     reinterpret_cast<float *>(smem + words + 2 * top)};
  const float c = kLog2e / a.dm.temperature;
  const bool tail = a.teacher_lse != nullptr, known = a.sums_in != nullptr;
  for (int64_t row = blockIdx.x; row < a.dm.rows; row += gridDim.x) {
    const RowVectors<T> in(static_cast<const T *>(a.logits) + row * a.logits_stride, vocab);
    const int nv = in.count();
    T *out_row = a.dlogits ? static_cast<T *>(a.dlogits) + row * a.dlogits_stride : nullptr;
    const RowVectors<T> out(out_row, vocab);
    const float w = (a.weights ? a.weights[row] : 1.f);
    if (w == 0.f) {
      if (threadIdx.x == 0 && !known) {
        a.loss[row] = 0.f;
        if (a.sums) a.sums[2 * row] = a.sums[2 * row + 1] = 0.f;
      }
      const float zero[N] = {};
      if (out_row)
        for (int v = threadIdx.x; v < out.count(); v += blockDim.x) out.store(v, zero);
      continue;
    }
    __syncthreads();  // the row before is done with the shared memory
    for (int i = threadIdx.x; i < words; i += blockDim.x) l.bits[i] = 0;
    __syncthreads();
    if (warp == 0) read_top(a, row, static_cast<const T *>(a.logits) + row * a.logits_stride, in.phase, l);
    __syncthreads();
    Sum sum = no_sum();
    if (!known) {
      for (int v = threadIdx.x; v < nv; v += blockDim.x) {
        float f[N];
        unpack16<T>(in.load(v, from_float<T>(-CUDART_INF_F)), f);
        const uint32_t skip = tail ? l.bits[v * N >> 5] >> (v * N & 31) : 0;
        float m = -CUDART_INF_F;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (skip >> i & 1) f[i] = -CUDART_INF_F;
          m = fmaxf(m, f[i]);
        }
        const float at = m == -CUDART_INF_F ? 0.f : m;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) s += share(f[i], at, c);
        sum = join(sum, {m, s}, c);
      }
      sum = warp_join(sum, c);
      if (lane == 0) box[warp] = sum;
      __syncthreads();
    }
    if (warp == 0) {
      if (known)
        sum = {a.sums_in[2 * row], a.sums_in[2 * row + 1]};
      else
        sum = warp_join(lane < warps ? box[lane] : no_sum(), c);
      const RowPlan r = plan_row(a, row, known && a.grad_loss ? w * a.grad_loss[row] : w, sum, c, l);
      if (lane == 0) {
        plan = r;
        if (!known) {
          a.loss[row] = r.loss;
          if (a.sums) a.sums[2 * row] = sum.m, a.sums[2 * row + 1] = sum.s;
        }
      }
    }
    if (!out_row) continue;
    __syncthreads();
    const RowPlan r = plan;
    for (int v = threadIdx.x; v < nv; v += blockDim.x) {
      float f[N];
      unpack16<T>(in.load(v, from_float<T>(-CUDART_INF_F)), f);
#pragma unroll
      for (int i = 0; i < N; ++i)
        f[i] = r.rest_m == CUDART_INF_F && r.rest_scale == 0.f ? 0.f : share(f[i], r.rest_m, c) * r.rest_scale;
      if (out.phase == in.phase) {
        out.store(v, f);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int e = v * N + i - in.phase;
          if (e >= 0 && e < vocab) out_row[e] = from_float<T>(f[i]);
        }
      }
    }
    __syncthreads();  // the entries' gradients go over what was written in their place
    for (int j = threadIdx.x; j < top; j += blockDim.x)
      if (l.code[j] >= 0) out_row[l.code[j]] = from_float<T>(top_grad(r, l.t[j], l.z[j], c, 1.f / a.dm.temperature));
  }
}

template <class T>
cudaError_t launch_distill_typed(const DistillArgs &a, cudaStream_t st) {
  const size_t smem = distill_smem(a.dm.vocab, a.dm.top);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k_distill<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const int block = a.dm.vocab <= 2048 ? 128 : 256;
  k_distill<T><<<(unsigned)(a.dm.rows < (1 << 30) ? a.dm.rows : (1 << 30)), block, smem, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_distill(const DistillArgs &a, cudaStream_t st) {
  switch (a.dm.dtype) {
    case RVQ_DTYPE_F32: return launch_distill_typed<float>(a, st);
    case RVQ_DTYPE_BF16: return launch_distill_typed<__nv_bfloat16>(a, st);
    default: return launch_distill_typed<__half>(a, st);
  }
}

rvq_status check_distill(const DistillArgs &a) {
  const rvq_distill_dims &dm = a.dm;
  const int e = dtype_bytes(dm.dtype), te = dtype_bytes(dm.top_dtype);
  if (dm.rows < 0 || dm.vocab <= 0 || dm.top <= 0 || !e || !te) return RVQ_ERR_INVALID_ARG;
  if (!(dm.temperature > 0.f) || dm.temperature > 3.402823466e38f) return RVQ_ERR_INVALID_ARG;
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
