// Rows that are normalised: copies of the rows to come into shared memory, how a
// row lies over the threads of a warp or a block, and the sums over it
// (rvq_norm.cu, rvq_rms.cu, rvq_rms_backward.cu).
#pragma once

#include "rvq_rows.cuh"

namespace rvq {
namespace {

constexpr int kNormMaxWidth = 16384;
constexpr int kSms = 152;

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Read each time that it stands here: kept in registers between the two uses of
// a row, the values would spill.
__device__ __forceinline__ uint4 read16(const uint4 *p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"((uint32_t)__cvta_generic_to_shared(p)));
  return v;
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// The sum of K values over a row's group: LANES lanes of a warp, or (LANES 0)
// `tpr` threads, whole warps, through `box` (two halves used in turn, one
// barrier of the group a call).
template <int K, int LANES>
__device__ __forceinline__ void group_sum(float (&v)[K], float (*box)[K][16], int &turn, int group, int tpr) {
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int o = (LANES ? LANES : 32) / 2; o; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if constexpr (LANES == 0) {
    const int lane = threadIdx.x & 31, warp = (threadIdx.x % tpr) >> 5, warps = tpr >> 5;
    float(*at)[16] = box[group * 2 + (turn & 1)];
    ++turn;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) at[k][warp] = v[k];
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = lane < warps ? at[k][lane] : 0.f;
#pragma unroll
      for (int o = 8; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      v[k] = __shfl_sync(0xffffffffu, s, 0);
    }
  }
}

// A thread's columns: vectors t + j * tpr of the row's `full`, and perhaps one
// beside them.
template <int N, int NV>
struct Columns {
  int head, full, tail, tpr, t, edge;  // edge: the column beside the vectors, -1: none
  __device__ __forceinline__ Columns(const void *row, int bytes, int width, int tpr_, int t_) : tpr(tpr_), t(t_) {
    const int past = (int)(reinterpret_cast<uintptr_t>(row) & 15) / bytes;
    head = min(width, past ? N - past : 0);
    full = (width - head) / N;
    tail = width - head - full * N;
    edge = t < head ? t : t >= N && t < N + tail ? head + full * N + t - N : -1;
  }
  __device__ __forceinline__ bool has(int j) const { return t + j * tpr < full; }
  __device__ __forceinline__ int column(int j) const { return head + (t + j * tpr) * N; }
};

// How the `units` of a row, `n` elements each, are laid over threads: at most 32
// columns a thread.  Every column that is not in a unit needs a place of its own:
// the ring kernels have one beside the vectors (their units are the whole
// vectors), k_norm and k_norm_backward have none (a partial vector is a unit).
struct NormShape {
  int threads;  // of a row
  int columns;  // of a thread (C)
};
inline NormShape norm_shape(int units, int n, int least = 32) {
  int threads = least;
  while (threads * 32 < units * n) threads *= 2;
  const int c = ((units + threads - 1) / threads * n + 7) / 8 * 8;
  return {threads, c < 8 ? 8 : c};
}

}  // namespace
}  // namespace rvq
