// Rows of 32- or 16-bit floats: element types, 16-byte vectors of them, and
// the reductions that the row operators (rvq_norm.cu, rvq_distill.cu,
// rvq_beam.cu) share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "rvq.h"

namespace rvq {

// Element sizes of RVQ_DTYPE_* (0: unknown).
inline int dtype_bytes(int32_t dtype) {
  return dtype == RVQ_DTYPE_F32 ? 4 : dtype == RVQ_DTYPE_BF16 || dtype == RVQ_DTYPE_F16 ? 2 : 0;
}
inline bool aligned_to(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
// Whether rows of `bytes`-sized elements at p, `stride` elements apart, all start on a 16-byte boundary.
inline bool rows_aligned16(const void *p, int64_t stride, int64_t rows, int bytes) {
  return aligned_to(p, 16) && (rows <= 1 || (stride * bytes) % 16 == 0);
}

// Lets a kernel take up to kMostSmem bytes of dynamic shared memory: asked of
// the runtime once per kernel and device, and always for the same size, so that
// no call lowers what another one needs.
constexpr int kMostSmem = 208 * 1024;  // of an SM's 227 KB; the rest is for static arrays
template <class K>
cudaError_t allow_smem(K kernel, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || done[dev & 63].load()) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
  if (e == cudaSuccess) done[dev & 63].store(true);
  return e;
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <class T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// A 16-byte vector (N = 16 / sizeof(T)) or one element (N = 1) as floats.
template <class T>
__device__ __forceinline__ void unpack16(const uint4 &v, float (&f)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 4) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        f[2 * i] = p.x, f[2 * i + 1] = p.y;
      }
    }
  }
}

template <class T>
__device__ __forceinline__ uint4 pack16(const float (&f)[16 / sizeof(T)]) {
  uint4 v;
  if constexpr (sizeof(T) == 4) {
    v = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&p);
      } else {
        const __half2 p = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&p);
      }
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return v;
}

// Two floats in one operation each (round to nearest, as the single ones).
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 floats(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// A vector as pairs of floats, and back.
template <class T>
__device__ __forceinline__ void unpack_pairs(const uint4 &v, F2 (&f)[8 / sizeof(T)]) {
  float e[16 / sizeof(T)];
  unpack16<T>(v, e);
#pragma unroll
  for (int i = 0; i < 8 / (int)sizeof(T); ++i) f[i] = f2(e[2 * i], e[2 * i + 1]);
}
template <class T>
__device__ __forceinline__ uint4 pack_pairs(const F2 (&f)[8 / sizeof(T)]) {
  float e[16 / sizeof(T)];
#pragma unroll
  for (int i = 0; i < 8 / (int)sizeof(T); ++i) {
    const float2 p = floats(f[i]);
    e[2 * i] = p.x, e[2 * i + 1] = p.y;
  }
  return pack16<T>(e);
}

// The largest element of a vector (a NaN is passed over).
template <class T>
__device__ __forceinline__ float largest_of(const uint4 &v) {
  if constexpr (sizeof(T) == 4) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  } else {
    using P = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const P *p = reinterpret_cast<const P *>(&v);
    const P m = __hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3]));
    return fmaxf(to_float(m.x), to_float(m.y));
  }
}

// A row cut at 16-byte boundaries: `head` elements before the first, `full`
// vectors, `tail` elements after the last.  The head and tail elements (under
// N each) go to 2 N threads, one each, so that no vector needs a check.
template <class T>
struct CutRow {
  static constexpr int N = 16 / (int)sizeof(T);
  const T *z;
  int width, head, full, tail;
  __device__ __forceinline__ CutRow(const T *row, int width_) : z(row), width(width_) {
    const int past = (int)(reinterpret_cast<uintptr_t>(z) & 15) / (int)sizeof(T);
    head = min(width, past ? N - past : 0);
    full = (width - head) / N;
    tail = width - head - full * N;
  }
  __device__ __forceinline__ uint4 vector(int v) const { return *reinterpret_cast<const uint4 *>(z + head + v * N); }
  // the element that thread t holds beside its vectors (-1: none)
  __device__ __forceinline__ int edge(int t) const {
    return t < head ? t : t >= N && t < N + tail ? head + full * N + t - N : -1;
  }
};

template <class T>
__device__ __forceinline__ uint4 all_low() {  // a vector of -inf
  const uint32_t w = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
  return make_uint4(w, w, w, w);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The largest of a warp's values, by one integer reduction over their order (a
// NaN's place in it is unspecified).
__device__ __forceinline__ float warp_max_order(float v) {
  const uint32_t b = __float_as_uint(v);
  const uint32_t o = __reduce_max_sync(0xffffffffu, b & 0x80000000u ? ~b : b | 0x80000000u);
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

// 2^x to about 2 units in the last place (subnormal results become zero).
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

}  // namespace rvq
