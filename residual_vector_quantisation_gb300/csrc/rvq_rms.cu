// Root-mean-square norm over rows, with the residual's addition, dropout of
// what is added, and an output in 8 bits with scales (rvq_rms_norm).
//
//   h = round(residual + drop(x)),  r = 1 / sqrt(mean(h^2) + eps),  y = h r w
//
// The sum h is rounded to the tensors' type before it is normalised: that is
// what the layers after this one and the backward pass read, so all of them see
// the same value.
#include <cuda_fp8.h>

#include "rvq_rms.cuh"

namespace rvq {
namespace {

// A scale from the bits of a block's largest magnitude (NaN is above infinity),
// and its inverse: max / 448 (a product), at least 2^-126, so that a block of zeros
// has a scale and every scale an inverse; or the next power of two, read off the bits:
// 448 is 1.75 * 2^8.
struct Scale {
  float value, inverse;
  uint8_t exponent;  // of a power of two
};
__device__ __forceinline__ Scale scale_of(uint32_t most, bool power) {
  Scale s;
  if (power) {
    int e = (int)(most >> 23) - 8 + ((most & 0x7fffffu) > 0x600000u);
    e = most >= 0x7f800000u ? 255 : e < 1 ? 1 : e;  // infinity has no scale of this kind
    s.exponent = (uint8_t)e;
    s.value = 0.f;
    s.inverse = e == 255 ? CUDART_NAN_F : __uint_as_float((uint32_t)(254 - e) << 23);  // 1 <= e <= 247
  } else {
    s.value = __uint_as_float(most) * (1.f / 448.f);
    if (s.value < 1.17549435e-38f) s.value = 1.17549435e-38f;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.inverse) : "f"(s.value));  // (to a unit in the last place)
    s.exponent = 0;
  }
  return s;
}
// The larger of m and the magnitudes of a and b, NaN where one is NaN.
__device__ __forceinline__ float most3(float m, float a, float b) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void put_scale(const RmsArgs &a, int64_t row, int at, const Scale &s) {
  const int64_t i = row * a.scale_count + at;
  if (a.scale_type == RVQ_SCALE_E8M0)
    static_cast<uint8_t *>(a.scales)[i] = s.exponent;
  else
    static_cast<float *>(a.scales)[i] = s.value;
}
__device__ __forceinline__ uint32_t two_e4m3(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// ---------------------------------------------------------------------------
// rows through a ring in shared memory
// ---------------------------------------------------------------------------

// Places for the largest magnitudes of the blocks of a thread block's rows: a row of `threads` threads has up to
// 32 * threads + 14 columns, in blocks of 32 at least.
constexpr int kTable = kRmsThreads / 8 * (8 + 2);

// The largest of a group's values, as group_sum.
template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t v, uint32_t (*box)[16], int group, int tpr) {
  if constexpr (LANES != 0) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  } else {
    v = __reduce_max_sync(0xffffffffu, v);
    const int lane = threadIdx.x & 31;
    if (lane == 0) box[group][(threadIdx.x % tpr) >> 5] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
    return __reduce_max_sync(0xffffffffu, lane < tpr >> 5 ? box[group][lane] : 0u);
  }
}
template <int LANES>
__device__ __forceinline__ void group_barrier(int group, int tpr) {
  if constexpr (LANES != 0)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
}

// As for layer norm: a block stays on its SM and walks its rows; each thread
// copies its vectors of the rows to come into its own slots of shared memory, and
// keeps its columns' weights in registers.  All tensors of T start equally far
// from a 16-byte boundary in each row.
//
// Bandwidth and a row's chain share the bound (16 warps an SM): 60 000 x 1024 bf16
// with a residual 76 us, with dropout 81 (their bytes alone: 72); 16 384 x 4096 to
// 8 bits with a scale for 128 columns 88 (bytes: 69), where instructions count (34
// an element and lane) and each row has a barrier.
template <class T, int C, int LANES, bool DROP>
__global__ void __launch_bounds__(rms_threads<T>(), 1) k_rms_ring(const RmsArgs a, const int tpr_) {
  constexpr int N = 16 / (int)sizeof(T), NV = C / N;
  extern __shared__ uint4 ring[];
  __shared__ float box[2 * kRmsThreads / 32][1][16];
  __shared__ uint32_t high[kRmsThreads / 32][16], tables[kTable];
  const int tpr = LANES ? LANES : tpr_, group = threadIdx.x / tpr, groups = blockDim.x / tpr, width = a.dm.width;
  const int64_t rows = a.dm.rows, step = (int64_t)gridDim.x * groups, first = blockIdx.x + (int64_t)group * gridDim.x;
  const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
  const Columns<N, NV> c(x + (int64_t)blockIdx.x * a.xs, sizeof(T), width, tpr, threadIdx.x % tpr);
  const bool two = res != nullptr;
  const int arrays = two ? 2 : 1;
  const float inv = 1.f / (float)width;
  float g[NV][N], ge = c.edge >= 0 ? weight_at<T>(a, c.edge) : 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < N; ++i) g[j][i] = c.has(j) ? weight_at<T>(a, c.column(j) + i) : 0.f;
  uint4 *slot = ring + threadIdx.x;  // [stage][x, residual][j][thread]
  for (int i = 0; i < kStages * arrays * NV; ++i) slot[i * blockDim.x] = make_uint4(0, 0, 0, 0);
  auto fetch = [&](int64_t row, int stage) {
    if (row < rows) {
      uint4 *at = slot + stage * arrays * NV * blockDim.x;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (c.has(j)) {
          copy16((uint32_t)__cvta_generic_to_shared(at + j * blockDim.x), x + row * a.xs + c.column(j));
          if (two) copy16((uint32_t)__cvta_generic_to_shared(at + (NV + j) * blockDim.x), res + row * a.rs + c.column(j));
        }
    }
    copies_end();
  };
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) fetch(first + k * step, k);
  auto edge_of = [&](const T *p, int64_t stride, int64_t row) {
    return p && c.edge >= 0 && row < rows ? to_float(p[row * stride + c.edge]) : 0.f;
  };
  float e_next = edge_of(x, a.xs, first), re_next = edge_of(res, a.rs, first);
  const Dropped dropped(a.mask);
  int turn = 0, stage = 0;
  // the groups of a warp stay together: what a row past the end computes is stored nowhere
  constexpr int kPerWarp = LANES ? 32 / (LANES ? LANES : 32) : 1;
  const int64_t ahead = (int64_t)(group % kPerWarp) * gridDim.x;
  for (int64_t row = first; row - ahead < rows; row += step) {
    const bool there = row < rows;
    fetch(row + (kStages - 1) * step, (stage + kStages - 1) % kStages);
    float e = e_next;
    const float re = re_next;
    e_next = edge_of(x, a.xs, row + step), re_next = edge_of(res, a.rs, row + step);
    copies_wait<kStages - 1>();
    const uint4 *xv = slot + stage * arrays * NV * blockDim.x, *rv = xv + NV * blockDim.x;
    uint32_t gone = 0;  // of all the thread's vectors
    if constexpr (DROP) {
#pragma unroll 2
      for (int j = 0; j < NV; ++j) gone |= dropped.from<N>((uint64_t)(row * width + c.column(j))) << (j * N / 2);
    }
    float f[NV][N], s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      unpack16<T>(xv[j * blockDim.x], f[j]);
      if constexpr (DROP) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          f[j][i] = Dropped::at(gone >> (j * N / 2), i) ? 0.f : __fmul_rn(f[j][i], dropped.factor);
      }
      if (two) {
        float r[N];
        unpack16<T>(rv[j * blockDim.x], r);
#pragma unroll
        for (int i = 0; i < N; ++i) f[j][i] = __fadd_rn(f[j][i], r[i]);
      }
      if (two || DROP) {
        const uint4 sum = pack16<T>(f[j]);
        if (a.total && c.has(j) && there)
          *reinterpret_cast<uint4 *>(static_cast<T *>(a.total) + row * a.ts + c.column(j)) = sum;
        unpack16<T>(sum, f[j]);
      }
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) q = fmaf(f[j][i], f[j][i], q);
      if (c.has(j)) s[0] += q;
    }
    if (c.edge >= 0) {
      if constexpr (DROP) e = dropped.element((uint64_t)(row * width + c.edge)) ? 0.f : __fmul_rn(e, dropped.factor);
      if (two) e = __fadd_rn(e, re);
      if (two || DROP) {
        const T sum = from_float<T>(e);
        if (a.total && there) static_cast<T *>(a.total)[row * a.ts + c.edge] = sum;
        e = to_float(sum);
      }
      s[0] = fmaf(e, e, s[0]);
    }
    group_sum<1, LANES>(s, box, turn, group, tpr);
    const float r = 1.f / sqrtf(fmaf(s[0], inv, a.dm.eps));
    if (a.rstd && c.t == 0 && there) a.rstd[row] = r;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < N; ++i) f[j][i] = f[j][i] * r * g[j][i];
      if (a.y && c.has(j) && there)
        *reinterpret_cast<uint4 *>(static_cast<T *>(a.y) + row * a.ys + c.column(j)) = pack16<T>(f[j]);
    }
    e = e * r * ge;
    if (a.y && c.edge >= 0 && there) static_cast<T *>(a.y)[row * a.ys + c.edge] = from_float<T>(e);
    stage = (stage + 1) % kStages;
    if (a.q == nullptr) continue;

    uint8_t *q = a.q + row * a.qs;
    const bool power = a.scale_type == RVQ_SCALE_E8M0;
    const bool words = ((reinterpret_cast<uintptr_t>(q) + c.head) & (N - 1)) == 0;
    auto put = [&](int j, const float (&inverse)[N]) {
      uint32_t w[N / 4];
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const uint32_t p = two_e4m3(f[j][i] * inverse[i], f[j][i + 1] * inverse[i + 1]);
        w[i / 4] = i % 4 ? w[i / 4] | p << 16 : p;
      }
      uint8_t *at = q + c.column(j);
      if (!c.has(j) || !there) return;
      if (!words) {
#pragma unroll
        for (int i = 0; i < N; ++i) at[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
      } else if constexpr (N == 8) {
        *reinterpret_cast<uint2 *>(at) = make_uint2(w[0], w[1]);
      } else {
        *reinterpret_cast<uint32_t *>(at) = w[0];
      }
    };
    auto put_all = [&](int j, float inverse) {
      float all[N];
#pragma unroll
      for (int i = 0; i < N; ++i) all[i] = inverse;
      put(j, all);
    };
    auto put_edge = [&](float inverse) {
      if (c.edge >= 0 && there) q[c.edge] = (uint8_t)two_e4m3(e * inverse, 0.f);
    };
    auto most_all = [&](int j) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < N; i += 2) m = most3(m, f[j][i], f[j][i + 1]);
      return c.has(j) ? __float_as_uint(m) : 0u;
    };
    auto most_of = [&](int j, int from, int to) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i >= from && i < to) m = max(m, __float_as_uint(f[j][i]) & 0x7fffffffu);
      return m;
    };
    if (a.block == 0) {
      uint32_t m = c.edge >= 0 ? __float_as_uint(e) & 0x7fffffffu : 0u;
#pragma unroll
      for (int j = 0; j < NV; ++j) m = max(m, most_all(j));
      const Scale sc = scale_of(group_max<LANES>(m, high, group, tpr), power);
      if (c.t == 0 && there) put_scale(a, row, 0, sc);
#pragma unroll
      for (int j = 0; j < NV; ++j) put_all(j, sc.inverse);
      put_edge(sc.inverse);
    } else if (c.head == 0 && c.tail == 0) {
      // a block is 4 to 32 neighbouring lanes of one vector number
      const int lanes = a.block / N;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        uint32_t m = most_all(j);
        for (int o = lanes / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const Scale sc = scale_of(m, power);
        const int v = c.t + j * tpr;
        if (v % lanes == 0 && c.has(j) && there) put_scale(a, row, v / lanes, sc);
        put_all(j, sc.inverse);
      }
    } else {
      // blocks end inside vectors, or have the elements beside them: a table in shared memory
      uint32_t *table = tables + group * (tpr + 2);
      const int count = a.scale_count;
      group_barrier<LANES>(group, tpr);  // the row before has been read
      for (int i = c.t; i < count; i += tpr) table[i] = 0;
      group_barrier<LANES>(group, tpr);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!c.has(j)) continue;
        const int b = c.column(j) / a.block, in = (b + 1) * a.block - c.column(j);  // columns of the first block
        atomicMax(&table[b], most_of(j, 0, in));
        if (in < N) atomicMax(&table[b + 1], most_of(j, in, N));
      }
      if (c.edge >= 0) atomicMax(&table[c.edge / a.block], __float_as_uint(e) & 0x7fffffffu);
      group_barrier<LANES>(group, tpr);
      for (int i = c.t; i < count; i += tpr)
        if (there) put_scale(a, row, i, scale_of(table[i], power));
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!c.has(j)) continue;
        const int b = c.column(j) / a.block, in = (b + 1) * a.block - c.column(j);
        const float one = scale_of(table[b], power).inverse;
        const float other = in < N ? scale_of(table[b + 1], power).inverse : one;
        float all[N];
#pragma unroll
        for (int i = 0; i < N; ++i) all[i] = i < in ? one : other;
        put(j, all);
      }
      if (c.edge >= 0) put_edge(scale_of(table[c.edge / a.block], power).inverse);
    }
  }
}

// ---------------------------------------------------------------------------
// any rows: the sum in shared memory, element by element
// ---------------------------------------------------------------------------

// A warp's rows (WARP, up to 1024 columns, 4 a block) or a block's.  A warp takes
// 256 columns at a time, 8 elements a lane in flight.  Latency of one row after the
// other: 60 000 x 1024 bf16 122 us (bytes alone: 36), 58 536 x 1025, a block of 512
// threads a row, 549 (35), 5000 x 16384 f32 with a residual 276 (193).
constexpr int kAnyWidth = 1024, kAnyWarps = 4, kAnyThreads = 512;
template <class T, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kAnyWarps : kAnyThreads)
    k_rms_any(const RmsArgs a, const bool drop, const int64_t row0) {
  extern __shared__ float sums[];  // [row][width], then [row][scale_count]
  __shared__ float box[16];
  __shared__ uint32_t most;
  const int width = a.dm.width, lane = threadIdx.x & 31;
  const int warp = WARP ? 0 : threadIdx.x >> 5, warps = WARP ? 1 : blockDim.x >> 5;
  const int team = WARP ? threadIdx.x >> 5 : 0, t = WARP ? lane : threadIdx.x, threads = WARP ? 32 : blockDim.x;
  const int64_t row = row0 + (WARP ? blockIdx.x * (int64_t)kAnyWarps + team : blockIdx.x);
  if (row >= a.dm.rows) return;  // (a warp's, or the block's)
  auto barrier = [] {
    if constexpr (WARP)
      __syncwarp();
    else
      __syncthreads();
  };
  float *h = sums + team * width;
  uint32_t *table = reinterpret_cast<uint32_t *>(sums + (WARP ? kAnyWarps : 1) * width) + team * a.scale_count;
  const T *x = static_cast<const T *>(a.x) + row * a.xs;
  const T *res = a.residual ? static_cast<const T *>(a.residual) + row * a.rs : nullptr;
  const Dropped dropped(a.mask);
  float s = 0.f;
  for (int c0 = warp * 256; c0 < width; c0 += warps * 256) {
    float f[8], r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + i * 32 + lane;
      f[i] = c < width ? to_float(x[c]) : 0.f;
      r[i] = res && c < width ? to_float(res[c]) : 0.f;
    }
    if (drop) {
      const uint64_t e0 = (uint64_t)(row * width + c0);
      const int at = (int)(e0 & 7);
      const uint32_t bits = dropped.group((e0 >> 3) + lane), last = dropped.group((e0 >> 3) + 32);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = at + i * 32 + lane;
        uint32_t b = __shfl_sync(0xffffffffu, bits, (e >> 3) & 31);
        if (e >= 256) b = last;
        f[i] = Dropped::at(b, e & 7) ? 0.f : __fmul_rn(f[i], dropped.factor);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + i * 32 + lane;
      if (c >= width) continue;
      if (res) f[i] = __fadd_rn(f[i], r[i]);
      if (res || drop) {
        const T sum = from_float<T>(f[i]);
        if (a.total) static_cast<T *>(a.total)[row * a.ts + c] = sum;
        f[i] = to_float(sum);
      }
      h[c] = f[i];
      s = fmaf(f[i], f[i], s);
    }
  }
  s = warp_sum(s);
  if constexpr (!WARP) {
    if (lane == 0) box[warp] = s;
    if (threadIdx.x == 0) most = 0;
    __syncthreads();
    s = warp_sum(lane < warps ? box[lane] : 0.f);
  }
  const float r = 1.f / sqrtf(fmaf(s, 1.f / (float)width, a.dm.eps));
  if (a.rstd && t == 0) a.rstd[row] = r;
  if (a.q && a.block) {
    for (int i = t; i < a.scale_count; i += threads) table[i] = 0;
    barrier();
  }
  uint32_t high = 0;
  for (int c0 = warp * 256; c0 < width; c0 += warps * 256)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + i * 32 + lane;
      const float y = c < width ? h[c] * r * weight_at<T>(a, c) : 0.f;
      if (a.y && c < width) static_cast<T *>(a.y)[row * a.ys + c] = from_float<T>(y);
      if (a.q == nullptr) continue;
      if (c < width) h[c] = y;
      const uint32_t m = __float_as_uint(y) & 0x7fffffffu;
      high = max(high, m);
      if (a.block && c - lane < width) {  // the warp's 32 columns are of one block
        const uint32_t all = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) atomicMax(&table[c / a.block], all);
      }
    }
  if (a.q == nullptr) return;
  const bool power = a.scale_type == RVQ_SCALE_E8M0;
  Scale sc{};
  if (a.block == 0) {
    high = __reduce_max_sync(0xffffffffu, high);
    if constexpr (!WARP) {
      if (lane == 0) atomicMax(&most, high);
      __syncthreads();
      high = most;
    }
    sc = scale_of(high, power);
    if (t == 0) put_scale(a, row, 0, sc);
  } else {
    barrier();
    for (int i = t; i < a.scale_count; i += threads) put_scale(a, row, i, scale_of(table[i], power));
  }
  uint8_t *q = a.q + row * a.qs;
  for (int c0 = warp * 256; c0 < width; c0 += warps * 256)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + i * 32 + lane;
      if (c >= width) continue;
      if (a.block) sc = scale_of(table[c / a.block], power);
      q[c] = (uint8_t)two_e4m3(h[c] * sc.inverse, 0.f);
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

template <class T>
size_t rms_thread_bytes(const RmsArgs &a, int columns) {
  return (size_t)kStages * (a.residual ? 2 : 1) * columns * sizeof(T);
}

template <class T, int C, int LANES, bool DROP>
cudaError_t launch_ring(const RmsArgs &a, const RmsShape &s, cudaStream_t st) {
  const size_t thread = rms_thread_bytes<T>(a, C);
  const RmsGrid grid = rms_grid<T>(a.dm.rows, s, thread);
  const auto kernel = k_rms_ring<T, C, LANES, DROP>;
  static std::atomic<bool> allowed[64];
  const cudaError_t e = allow_smem(kernel, allowed);
  if (e != cudaSuccess) return e;
  const int block = grid.groups * s.threads;
  kernel<<<(unsigned)grid.blocks, block, block * thread, st>>>(a, s.threads);
  return cudaGetLastError();
}
template <class T, bool DROP>
cudaError_t launch_ring_shape(const RmsArgs &a, const RmsShape &s, cudaStream_t st) {
  if (s.lanes == 8) return s.columns == 16 ? launch_ring<T, 16, 8, DROP>(a, s, st) : launch_ring<T, 32, 8, DROP>(a, s, st);
  if (s.lanes == 16) return launch_ring<T, 32, 16, DROP>(a, s, st);
  if (s.lanes == 32) return s.columns == 24 ? launch_ring<T, 24, 32, DROP>(a, s, st) : launch_ring<T, 32, 32, DROP>(a, s, st);
  return launch_ring<T, 32, 0, DROP>(a, s, st);
}
template <class T>
cudaError_t launch_any(const RmsArgs &a, bool drop, cudaStream_t st) {
  const bool warp = a.dm.width <= kAnyWidth;
  const int per = warp ? kAnyWarps : 1;
  const size_t smem = (size_t)per * (a.dm.width + a.scale_count) * sizeof(float);
  const auto kernel = warp ? k_rms_any<T, true> : k_rms_any<T, false>;
  static std::atomic<bool> allowed[2][64];
  cudaError_t e = allow_smem(kernel, allowed[warp]);
  constexpr int64_t kMost = (int64_t)1 << 30;  // blocks of a launch
  for (int64_t row0 = 0; e == cudaSuccess && row0 < a.dm.rows; row0 += kMost * per) {
    const int64_t blocks = (a.dm.rows - row0 + per - 1) / per;
    kernel<<<(unsigned)(blocks < kMost ? blocks : kMost), warp ? 32 * kAnyWarps : kAnyThreads, smem, st>>>(a, drop, row0);
    e = cudaGetLastError();
  }
  return e;
}

template <class T>
cudaError_t launch_rms_typed(const RmsArgs &a, bool drop, cudaStream_t st) {
  constexpr int e = sizeof(T), N = 16 / e;
  const int64_t rows = a.dm.rows;
  // a block of columns with a scale of its own is block / N lanes
  const RmsShape s = rms_shape(a.dm.width, e, rows_aligned16(a.x, a.xs, rows, e) && a.dm.width % N == 0, a.q ? a.block / N : 8);
  auto alike = [&](const void *p, int64_t stride) { return rows_alike(p, stride, a.x, a.xs, rows, e); };
  if (!alike(a.residual, a.rs) || !alike(a.total, a.ts) || !alike(a.y, a.ys) ||
      s.threads > rms_threads<T>() || rms_thread_bytes<T>(a, s.columns) * s.threads > kMostSmem)
    return launch_any<T>(a, drop, st);
  return drop ? launch_ring_shape<T, true>(a, s, st) : launch_ring_shape<T, false>(a, s, st);
}

cudaError_t launch_rms(const RmsArgs &a, bool drop, cudaStream_t st) {
  switch (a.dm.dtype) {
    case RVQ_DTYPE_F32: return launch_rms_typed<float>(a, drop, st);
    case RVQ_DTYPE_BF16: return launch_rms_typed<__nv_bfloat16>(a, drop, st);
    default: return launch_rms_typed<__half>(a, drop, st);
  }
}

}  // namespace
}  // namespace rvq

extern "C" {

RVQ_API rvq_status rvq_rms_norm(rvq_norm_dims dims, const void *x, int64_t x_stride, const void *residual,
                                int64_t residual_stride, const rvq_dropout_mask *mask, const void *weight, void *total,
                                int64_t total_stride, void *y, int64_t y_stride, float *rstd, const rvq_rms_8bit *q,
                                rvq_stream_t stream) {
  using namespace rvq;
  const rvq_status s = check_rms(dims);
  if (s != RVQ_OK) return s;
  RmsArgs a{};
  a.dm = dims, a.x = x, a.xs = x_stride, a.residual = residual, a.rs = residual_stride, a.weight = weight;
  a.total = total, a.ts = total_stride, a.y = y, a.ys = y_stride, a.rstd = rstd;
  if (mask && !dropout_mask(*mask, a.mask)) return RVQ_ERR_INVALID_ARG;
  int se = 0;
  if (q) {
    if (q->block != 0 && q->block != 32 && q->block != 64 && q->block != 128) return RVQ_ERR_INVALID_ARG;
    if (q->scale_type != RVQ_SCALE_F32 && q->scale_type != RVQ_SCALE_E8M0) return RVQ_ERR_INVALID_ARG;
    a.q = static_cast<uint8_t *>(q->values), a.qs = q->stride, a.scales = q->scales;
    a.block = q->block, a.scale_type = q->scale_type;
    a.scale_count = q->block ? (dims.width + q->block - 1) / q->block : 1;
    se = q->scale_type == RVQ_SCALE_F32 ? 4 : 1;
  }
  const int64_t rows = dims.rows;
  if (rows == 0) return RVQ_OK;
  const int e = dtype_bytes(dims.dtype), pe = dtype_bytes(dims.param_dtype);
  auto ok = [&](const void *p, int64_t stride) { return aligned_to(p, e) && (stride >= dims.width || rows <= 1); };
  if (!x || (!y && !q && !total) || !ok(x, x_stride) || (residual && !ok(residual, residual_stride)) ||
      (total && !ok(total, total_stride)) || (y && !ok(y, y_stride)))
    return RVQ_ERR_INVALID_ARG;
  if (!aligned_to(weight, pe) || !aligned_to(rstd, 4)) return RVQ_ERR_INVALID_ARG;
  if (q && (!q->values || !q->scales || !aligned_to(q->scales, se) || (q->stride < dims.width && rows > 1)))
    return RVQ_ERR_INVALID_ARG;
  // without a residual and dropout the sum is x: there is nothing to write
  if (total && !residual && !mask) return RVQ_ERR_INVALID_ARG;
  const Touched written[] = {rows_at(total, total_stride, dims), rows_at(y, y_stride, dims), bytes_at(rstd, rows * 4),
                             {row_set(a.q, dims.width, rows, a.qs), false},
                             bytes_at(a.scales, rows * a.scale_count * se)};
  const Touched read[] = {rows_at(x, x_stride, dims), rows_at(residual, residual_stride, dims),
                          bytes_at(weight, (int64_t)dims.width * pe), bytes_at(mask ? mask->step : nullptr, 8)};
  if (!rms_apart(written, read)) return RVQ_ERR_INVALID_ARG;
  return launch_rms(a, mask != nullptr, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? RVQ_OK : RVQ_ERR_CUDA;
}

}  // extern "C"
