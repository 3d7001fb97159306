// Layer norm over rows, forward and backward (rvq_layer_norm,
// rvq_layer_norm_backward).
//
// A row is read once: 8, 16 or 32 lanes per row up to 1024 columns, a group of
// 64 .. 512 threads per row above, up to 32 columns a thread.  The variance is the mean
// square of the centred values, so a row with a large mean loses nothing.
//
// k_norm_ring and k_norm_backward_ring (up to 8192 columns) are what bandwidth
// asks for.  A block stays on its SM and walks its rows; each thread copies its
// 16-byte vectors of the rows to come into its own slots of shared memory
// (cp.async, no barrier), so that loads are in flight without holding
// registers, and keeps its columns' parameters and the sums of their gradients
// in registers.  Rows that start inside a 16-byte vector (odd widths and
// strides) take the same path: a block's rows are a multiple of 8 apart, so
// all of them start equally far from a boundary, and a thread's columns stay
// its own.  What is needed for that is that x, y (dy, dx) are equally far from
// a boundary in each row; else, and above 8192 columns, k_norm and
// k_norm_backward hold a row in registers.
#include "rvq_internal.cuh"
#include "rvq_overlap.h"
#include "rvq_rows.cuh"
#include "sm103_ptx.cuh"

namespace rvq {
namespace {

constexpr int kNormMaxWidth = 16384;
constexpr int kNormWarpWidth = 1024;   // widest row that one warp holds
constexpr int kNormWarps = 4;          // rows (warps) of a block up to that width
constexpr int kSms = 152;

// One thread's piece of a row: unit u holds the columns [u * N, u * N + N).
template <class T, int N>
struct Unit {
  static_assert(N == 16 / (int)sizeof(T), "a unit is a 16-byte vector");
  uint4 raw;
  __device__ __forceinline__ void load(const T *row, int u, int width) {
    if ((u + 1) * N <= width) {
      raw = *reinterpret_cast<const uint4 *>(row + (int64_t)u * N);
    } else {
      union {
        uint4 v;
        T t[N];
      } r;
      r.v = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (u * N + i < width) r.t[i] = row[u * N + i];
      raw = r.v;
    }
  }
  __device__ __forceinline__ void get(float (&f)[N]) const { unpack16<T>(raw, f); }
};
template <class T>
struct Unit<T, 1> {
  T raw;
  __device__ __forceinline__ void load(const T *row, int u, int width) { raw = u < width ? row[u] : from_float<T>(0.f); }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = to_float(raw); }
};

template <class T, int N>
__device__ __forceinline__ void store_unit(T *row, int u, int width, const float (&f)[N]) {
  if constexpr (N == 1) {
    if (u < width) row[u] = from_float<T>(f[0]);
  } else if ((u + 1) * N <= width) {
    *reinterpret_cast<uint4 *>(row + (int64_t)u * N) = pack16<T>(f);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (u * N + i < width) row[u * N + i] = from_float<T>(f[i]);
  }
}

// N parameters of unit u (`none` where p is null).
template <class P, int N>
__device__ __forceinline__ void load_params(const P *p, int u, int width, float none, float (&f)[N]) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = none;
    return;
  }
  constexpr int M = 16 / (int)sizeof(P);
  if constexpr (N >= M) {
    if ((u + 1) * N <= width) {
#pragma unroll
      for (int j = 0; j < N / M; ++j) {
        float g[M];
        unpack16<P>(*reinterpret_cast<const uint4 *>(p + (int64_t)u * N + j * M), g);
#pragma unroll
        for (int i = 0; i < M; ++i) f[j * M + i] = g[i];
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = u * N + i < width ? to_float(p[u * N + i]) : none;
}

// The sum of K values over a row's threads, in every one of them: a warp's, or
// a block's through `box` (two halves used in turn, so that one barrier a call
// is enough).
template <int K, bool WARP>
__device__ __forceinline__ void row_sum(float (&v)[K], float *box, int &turn) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  if constexpr (!WARP) {
    float *at = box + (turn & 1) * K * 16;
    ++turn;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) at[k * 16 + warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = warp_sum(lane < warps ? at[k * 16 + lane] : 0.f);
  }
}

template <class T, class P, int N, int C, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kNormWarps : 512)
    k_norm(const T *x, int64_t xs, const P *__restrict__ weight, const P *__restrict__ bias, float eps,
           int64_t rows, int width, T *y, int64_t ys, float *mean, float *rstd) {
  constexpr int NV = C / N;
  __shared__ float box[2 * 16];
  const int tpr = WARP ? 32 : blockDim.x, t = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int64_t first = WARP ? (int64_t)blockIdx.x * kNormWarps + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t step = (int64_t)gridDim.x * (WARP ? kNormWarps : 1);
  const float inv = 1.f / (float)width;
  int turn = 0;
  for (int64_t row = first; row < rows; row += step) {
    const T *xr = x + row * xs;
    Unit<T, N> in[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) in[j].load(xr, j * tpr + t, width);
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[N];
      in[j].get(f);
#pragma unroll
      for (int i = 0; i < N; ++i) s[0] += f[i];
    }
    row_sum<1, WARP>(s, box, turn);
    const float mu = s[0] * inv;
    s[0] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[N];
      in[j].get(f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float d = (j * tpr + t) * N + i < width ? f[i] - mu : 0.f;
        s[0] = fmaf(d, d, s[0]);
      }
    }
    row_sum<1, WARP>(s, box, turn);
    const float r = 1.f / sqrtf(fmaf(s[0], inv, eps));
    if (t == 0) {
      if (mean) mean[row] = mu;
      if (rstd) rstd[row] = r;
    }
    T *yr = y + row * ys;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int u = j * tpr + t;
      if (u * N >= width) continue;
      float f[N], g[N], b[N];
      in[j].get(f);
      load_params<P, N>(weight, u, width, 1.f, g);
      load_params<P, N>(bias, u, width, 0.f, b);
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = fmaf((f[i] - mu) * r, g[i], b[i]);
      store_unit<T, N>(yr, u, width, f);
    }
  }
}

// dx per row, and each block's sums of dy * h and dy over its rows into
// part[block][2][width].
template <class T, class P, int N, int C, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kNormWarps : 512)
    k_norm_backward(const T *dy, int64_t dys, const T *x, int64_t xs, const P *__restrict__ weight,
                    const float *__restrict__ mean, const float *__restrict__ rstd, int64_t rows, int width, T *dx,
                    int64_t dxs, float *part) {
  constexpr int NV = C / N;
  __shared__ float box[2 * 2 * 16];
  const int tpr = WARP ? 32 : blockDim.x, t = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int64_t first = WARP ? (int64_t)blockIdx.x * kNormWarps + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t step = (int64_t)gridDim.x * (WARP ? kNormWarps : 1);
  const float inv = 1.f / (float)width;
  float dw[C], db[C];
#pragma unroll
  for (int c = 0; c < C; ++c) dw[c] = db[c] = 0.f;
  int turn = 0;
  for (int64_t row = first; row < rows; row += step) {
    const T *xr = x + row * xs, *dyr = dy + row * dys;
    Unit<T, N> in[NV], up[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      in[j].load(xr, j * tpr + t, width);
      up[j].load(dyr, j * tpr + t, width);
    }
    const float mu = mean[row], r = rstd[row];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[N], d[N], g[N];
      in[j].get(f);
      up[j].get(d);
      load_params<P, N>(weight, j * tpr + t, width, 1.f, g);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float h = (f[i] - mu) * r, a = d[i] * g[i];  // columns past the width have d = 0
        s[0] += a;
        s[1] = fmaf(a, h, s[1]);
        dw[j * N + i] = fmaf(d[i], h, dw[j * N + i]);
        db[j * N + i] += d[i];
      }
    }
    row_sum<2, WARP>(s, box, turn);
    if (dx == nullptr) continue;
    const float m1 = s[0] * inv, m2 = s[1] * inv;
    T *dxr = dx + row * dxs;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int u = j * tpr + t;
      if (u * N >= width) continue;
      float f[N], d[N], g[N];
      in[j].get(f);
      up[j].get(d);
      load_params<P, N>(weight, u, width, 1.f, g);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float h = (f[i] - mu) * r;
        f[i] = r * (d[i] * g[i] - m1 - h * m2);
      }
      store_unit<T, N>(dxr, u, width, f);
    }
  }
  if (part == nullptr) return;
  float *mine = part + (int64_t)blockIdx.x * 2 * width;
  if constexpr (WARP) {
    // the warps' sums, added in their order
    __shared__ float sums[2 * kNormWarpWidth];
    for (int w = 0; w < kNormWarps; ++w) {
      if ((threadIdx.x >> 5) == w)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int c = (j * 32 + t) * N + i;
            if (c < width) {
              sums[c] = (w ? sums[c] : 0.f) + dw[j * N + i];
              sums[kNormWarpWidth + c] = (w ? sums[kNormWarpWidth + c] : 0.f) + db[j * N + i];
            }
          }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < width; c += blockDim.x) {
      mine[c] = sums[c];
      mine[width + c] = sums[kNormWarpWidth + c];
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (j * tpr + t) * N + i;
        if (c < width) {
          mine[c] = dw[j * N + i];
          mine[width + c] = db[j * N + i];
        }
      }
  }
}

// ---------------------------------------------------------------------------
// rows through a ring in shared memory
// ---------------------------------------------------------------------------

constexpr int kRingWidth = 8192;
constexpr int kRingThreads = 384;  // of a block of the backward pass, one on an SM (168 registers a thread)
constexpr int kRingForward = 256;  // of the forward pass, two on an SM

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

template <class P, int N, int NV>
__device__ __forceinline__ void load_columns(const P *p, const Columns<N, NV> &c, float none, float (&f)[NV][N], float &edge) {
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < N; ++i) f[j][i] = p && c.has(j) ? to_float(p[c.column(j) + i]) : none;
  edge = p && c.edge >= 0 ? to_float(p[c.edge]) : none;
}

// Shared memory: `stages` x `arrays` x NV vectors of every thread, and, for
// the backward pass, 8 bytes of every thread and stage.
inline size_t ring_bytes(int threads, int stages, int arrays, int nv) {
  return (size_t)threads * stages * (arrays * nv * 16 + (arrays > 1 ? 8 : 0));
}

template <class T, class P, int C, int LANES, int STAGES>
__global__ void __launch_bounds__(kRingForward, 2)
    k_norm_ring(const T *x, int64_t xs, const P *__restrict__ weight, const P *__restrict__ bias, float eps,
                int64_t rows, int width, T *y, int64_t ys, float *mean, float *rstd, int tpr_) {
  constexpr int N = 16 / (int)sizeof(T), NV = C / N;
  extern __shared__ uint4 ring[];
  __shared__ float box[2 * kRingThreads / 64][1][16];
  const int tpr = LANES ? LANES : tpr_, group = threadIdx.x / tpr, groups = blockDim.x / tpr;
  const int64_t step = (int64_t)gridDim.x * groups, first = blockIdx.x + (int64_t)group * gridDim.x;
  const Columns<N, NV> c(x + (int64_t)blockIdx.x * xs, sizeof(T), width, tpr, threadIdx.x % tpr);
  const float inv = 1.f / (float)width;
  float g[NV][N], b[NV][N], ge, be;
  load_columns<P, N, NV>(weight, c, 1.f, g, ge);
  load_columns<P, N, NV>(bias, c, 0.f, b, be);
  uint4 *slot = ring + threadIdx.x;  // [stage][j][thread]
#pragma unroll
  for (int i = 0; i < STAGES * NV; ++i) slot[i * blockDim.x] = make_uint4(0, 0, 0, 0);
  auto fetch = [&](int64_t row, int stage) {
    if (row < rows) {
      const T *xr = x + row * xs;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (c.has(j)) copy16((uint32_t)__cvta_generic_to_shared(slot + (stage * NV + j) * blockDim.x), xr + c.column(j));
    } else if (LANES) {
#pragma unroll
      for (int j = 0; j < NV; ++j) slot[(stage * NV + j) * blockDim.x] = make_uint4(0, 0, 0, 0);
    }
    copies_end();
  };
#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) fetch(first + k * step, k);
  float e_next = c.edge >= 0 && first < rows ? to_float(x[first * xs + c.edge]) : 0.f;
  int turn = 0, stage = 0;
  // the groups of a warp stay together: a row past the end holds zeros and leaves nothing
  constexpr int kPerWarp = LANES ? 32 / (LANES ? LANES : 32) : 1;
  const int64_t ahead = (int64_t)(group % kPerWarp) * gridDim.x;
  for (int64_t row = first; row - ahead < rows; row += step) {
    const bool there = row < rows;
    fetch(row + (STAGES - 1) * step, (stage + STAGES - 1) % STAGES);
    const float e = e_next;
    e_next = c.edge >= 0 && row + step < rows ? to_float(x[(row + step) * xs + c.edge]) : 0.f;
    copies_wait<STAGES - 1>();
    float f[NV][N], s[1] = {e};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      unpack16<T>(slot[(stage * NV + j) * blockDim.x], f[j]);
#pragma unroll
      for (int i = 0; i < N; ++i) s[0] += f[j][i];
    }
    group_sum<1, LANES>(s, box, turn, group, tpr);
    const float mu = s[0] * inv;
    s[0] = c.edge >= 0 ? (e - mu) * (e - mu) : 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        f[j][i] -= mu;
        q = fmaf(f[j][i], f[j][i], q);
      }
      if (c.has(j)) s[0] += q;
    }
    group_sum<1, LANES>(s, box, turn, group, tpr);
    const float r = 1.f / sqrtf(fmaf(s[0], inv, eps));
    if (c.t == 0 && there) {
      if (mean) mean[row] = mu;
      if (rstd) rstd[row] = r;
    }
    T *yr = y + row * ys;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!c.has(j) || !there) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) f[j][i] = fmaf(f[j][i] * r, g[j][i], b[j][i]);
      *reinterpret_cast<uint4 *>(yr + c.column(j)) = pack16<T>(f[j]);
    }
    if (c.edge >= 0 && there) yr[c.edge] = from_float<T>(fmaf((e - mu) * r, ge, be));
    stage = (stage + 1) % STAGES;
  }
}

// dx per row, and each block's sums of dy * h and dy over its rows into
// part[block][2][width].
template <class T, class P, int C, int LANES, int STAGES>
__global__ void __launch_bounds__(kRingThreads)
    k_norm_backward_ring(const T *dy, int64_t dys, const T *x, int64_t xs, const P *__restrict__ weight,
                         const float *__restrict__ mean, const float *__restrict__ rstd, int64_t rows, int width, T *dx,
                         int64_t dxs, float *part, int tpr_) {
  constexpr int N = 16 / (int)sizeof(T), NV = C / N, H = N / 2;
  extern __shared__ uint4 ring[];
  __shared__ float box[2 * kRingThreads / 64][2][16];
  const int tpr = LANES ? LANES : tpr_, group = threadIdx.x / tpr, groups = blockDim.x / tpr;
  const int64_t step = (int64_t)gridDim.x * groups, first = blockIdx.x + (int64_t)group * gridDim.x;
  const Columns<N, NV> c(x + (int64_t)blockIdx.x * xs, sizeof(T), width, tpr, threadIdx.x % tpr);
  const float inv = 1.f / (float)width;
  const F2 zero = f2(0.f, 0.f);
  F2 g[NV][H], dw[NV][H], db[NV][H];
  float ge, dwe = 0.f, dbe = 0.f;
  {
    float w[NV][N];
    load_columns<P, N, NV>(weight, c, 1.f, w, ge);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < H; ++i) {
        g[j][i] = f2(w[j][2 * i], w[j][2 * i + 1]);
        dw[j][i] = db[j][i] = zero;
      }
  }
  uint4 *slot = ring + threadIdx.x;  // [stage][x, dy][j][thread], then [stage][thread] of mean and rstd
  float2 *stat = reinterpret_cast<float2 *>(ring + STAGES * 2 * NV * blockDim.x) + threadIdx.x;
#pragma unroll
  for (int i = 0; i < STAGES * 2 * NV; ++i) slot[i * blockDim.x] = make_uint4(0, 0, 0, 0);
  auto fetch = [&](int64_t row, int stage) {
    if (row < rows) {
      const T *xr = x + row * xs, *dyr = dy + row * dys;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (c.has(j)) {
          copy16((uint32_t)__cvta_generic_to_shared(slot + (stage * 2 * NV + j) * blockDim.x), xr + c.column(j));
          copy16((uint32_t)__cvta_generic_to_shared(slot + (stage * 2 * NV + NV + j) * blockDim.x), dyr + c.column(j));
        }
      const uint32_t at = (uint32_t)__cvta_generic_to_shared(stat + stage * blockDim.x);
      copy4(at, mean + row);
      copy4(at + 4, rstd + row);
    } else if (LANES) {
      asm volatile("" ::: "memory");  // after the last reading of these slots
#pragma unroll
      for (int j = 0; j < 2 * NV; ++j) slot[(stage * 2 * NV + j) * blockDim.x] = make_uint4(0, 0, 0, 0);
      stat[stage * blockDim.x] = make_float2(0.f, 0.f);
    }
    copies_end();
  };
#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) fetch(first + k * step, k);
  float xe_next = 0.f, de_next = 0.f;
  if (c.edge >= 0 && first < rows)
    xe_next = to_float(x[first * xs + c.edge]), de_next = to_float(dy[first * dys + c.edge]);
  int turn = 0, stage = 0;
  // the groups of a warp stay together: a row past the end holds zeros and leaves nothing
  constexpr int kPerWarp = LANES ? 32 / (LANES ? LANES : 32) : 1;
  const int64_t ahead = (int64_t)(group % kPerWarp) * gridDim.x;
  for (int64_t row = first; row - ahead < rows; row += step) {
    const bool there = row < rows;
    fetch(row + (STAGES - 1) * step, (stage + STAGES - 1) % STAGES);
    const float xe = xe_next, de = de_next;
    xe_next = de_next = 0.f;
    if (c.edge >= 0 && row + step < rows)
      xe_next = to_float(x[(row + step) * xs + c.edge]), de_next = to_float(dy[(row + step) * dys + c.edge]);
    copies_wait<STAGES - 1>();
    const float2 ms = stat[stage * blockDim.x];
    const float r = ms.y;
    const F2 mu2 = f2(-ms.x, -ms.x), r2 = f2(r, r);
    const uint4 *xv = slot + stage * 2 * NV * blockDim.x, *dv = xv + NV * blockDim.x;
    F2 s0 = zero, s1 = zero;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      F2 f[H], d[H];
      unpack_pairs<T>(read16(xv + j * blockDim.x), f);
      unpack_pairs<T>(read16(dv + j * blockDim.x), d);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const F2 h = (f[i] + mu2) * r2, a = d[i] * g[j][i];  // no column: d = 0
        s0 = s0 + a;
        s1 = fma2(a, h, s1);
        dw[j][i] = fma2(d[i], h, dw[j][i]);
        db[j][i] = db[j][i] + d[i];
      }
    }
    const float he = (xe - ms.x) * r;
    if (c.edge >= 0) {
      dwe = fmaf(de, he, dwe);
      dbe += de;
    }
    if (dx != nullptr) {
      const float2 a0 = floats(s0), a1 = floats(s1);
      float s[2] = {a0.x + a0.y, a1.x + a1.y};
      if (c.edge >= 0) s[0] += de * ge, s[1] = fmaf(de * ge, he, s[1]);
      group_sum<2, LANES>(s, box, turn, group, tpr);
      if constexpr (LANES != 0) __syncwarp();  // the second reading of the row stays below: moved up, it spills
      const float m1 = s[0] * inv, m2 = s[1] * inv;
      const F2 minus1 = f2(-m1, -m1), minus2 = f2(-m2, -m2);
      T *dxr = dx + row * dxs;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!c.has(j) || !there) continue;
        F2 f[H], d[H];
        unpack_pairs<T>(read16(xv + j * blockDim.x), f);
        unpack_pairs<T>(read16(dv + j * blockDim.x), d);
#pragma unroll
        for (int i = 0; i < H; ++i)
          f[i] = fma2((f[i] + mu2) * r2, minus2, fma2(d[i], g[j][i], minus1)) * r2;
        *reinterpret_cast<uint4 *>(dxr + c.column(j)) = pack_pairs<T>(f);
      }
      if (c.edge >= 0 && there) dxr[c.edge] = from_float<T>(r * (fmaf(de, ge, -m1) - he * m2));
    }
    stage = (stage + 1) % STAGES;
  }
  if (part == nullptr || blockIdx.x >= rows) return;  // (a block without rows has no part in the workspace)
  copies_wait<0>();
  __syncthreads();
  // the groups' sums through shared memory, added in their order
  float *sums = reinterpret_cast<float *>(ring), *mine = part + (int64_t)blockIdx.x * 2 * width;
  float *own = groups > 1 ? sums + (int64_t)group * 2 * width : mine;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (c.has(j))
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float2 w = floats(dw[j][i]), b = floats(db[j][i]);
        own[c.column(j) + 2 * i] = w.x, own[c.column(j) + 2 * i + 1] = w.y;
        own[width + c.column(j) + 2 * i] = b.x, own[width + c.column(j) + 2 * i + 1] = b.y;
      }
  if (c.edge >= 0) own[c.edge] = dwe, own[width + c.edge] = dbe;
  if (groups == 1) return;
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * width; i += blockDim.x) {
    float v = 0.f;
    for (int k = 0; k < groups; ++k) v += sums[k * 2 * width + i];
    mine[i] = v;
  }
}

// The blocks' sums, added in a fixed order: 32 columns a block, 32 lanes of
// parts.  Brought up while the kernel before it ends, which still writes `part`
// then: not a read-only pointer, and read through the L2.
constexpr int kSumRows = 32;
template <class P>
__global__ void __launch_bounds__(32 * kSumRows)
    k_norm_params(const float *part, int parts, int width, P *dweight, P *dbias) {
  __shared__ float box[kSumRows][33];
  P *out = blockIdx.y ? dbias : dweight;
  ptx::griddep_wait();
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const float *p = part + (int64_t)blockIdx.y * width + c;
  float s = 0.f;
  if (c < width)
#pragma unroll 4
    for (int i = ty; i < parts; i += kSumRows) s += __ldcg(p + (int64_t)i * 2 * width);
  box[ty][lane] = s;
  __syncthreads();
  if (ty == 0 && c < width) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kSumRows; ++i) s += box[i][lane];
    out[c] = from_float<P>(s);
  }
}

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

// Blocks of the backward pass: of the ring kernel, one an SM; of the other, as
// many as give each SM 512 threads.  The workspace holds a part of each.
inline int norm_parts(int64_t rows, int width) {
  const int threads = norm_shape(width, 1).threads;
  const int most = kSms * (threads == 32 ? 512 / (32 * kNormWarps) : 512 / threads);
  return rows < most ? (int)rows : most;
}

struct NormArgs {
  rvq_norm_dims dm;
  const void *dy;
  int64_t dys;
  const void *x;
  int64_t xs;
  const void *weight, *bias;
  const float *mean, *rstd;
  void *out;  // y or dx
  int64_t outs;
  float *mean_out, *rstd_out, *part;
  int parts;  // blocks of the backward pass, set by the launch
};

template <class T, class P, int N, int C, bool WARP>
cudaError_t launch_norm_shape(NormArgs &a, int threads, bool backward, cudaStream_t st) {
  const int block = WARP ? 32 * kNormWarps : threads;
  if (backward) {
    a.parts = norm_parts(a.dm.rows, a.dm.width);
    k_norm_backward<T, P, N, C, WARP><<<a.parts, block, 0, st>>>(
        static_cast<const T *>(a.dy), a.dys, static_cast<const T *>(a.x), a.xs, static_cast<const P *>(a.weight),
        a.mean, a.rstd, a.dm.rows, a.dm.width, static_cast<T *>(a.out), a.outs, a.part);
  } else {
    const int64_t blocks = WARP ? (a.dm.rows + kNormWarps - 1) / kNormWarps : a.dm.rows;
    k_norm<T, P, N, C, WARP><<<(unsigned)(blocks < (1 << 30) ? blocks : (1 << 30)), block, 0, st>>>(
        static_cast<const T *>(a.x), a.xs, static_cast<const P *>(a.weight), static_cast<const P *>(a.bias), a.dm.eps,
        a.dm.rows, a.dm.width, static_cast<T *>(a.out), a.outs, a.mean_out, a.rstd_out);
  }
  return cudaGetLastError();
}

template <class T, class P, int C, int LANES>  // LANES of a row, or 0: whole warps
cudaError_t launch_ring_shape(NormArgs &a, int threads, bool backward, cudaStream_t st) {
  constexpr int NV = C * (int)sizeof(T) / 16;
  constexpr int kForwardStages = sizeof(T) == 4 ? 3 : 4, kBackwardStages = sizeof(T) == 4 ? 2 : 3;
  // no more groups a block than there are rows for the SMs, and a multiple of 8 blocks, so that a block's rows
  // start equally far from a 16-byte boundary
  const int sms = backward ? kSms : 2 * kSms, most = (backward ? kRingThreads : kRingForward) / threads;
  int64_t groups = (a.dm.rows + sms - 1) / sms;
  groups = groups > most ? most : groups;
  constexpr int kPerWarp = LANES ? 32 / (LANES ? LANES : 32) : 1;
  groups = (groups + kPerWarp - 1) / kPerWarp * kPerWarp;  // whole warps
  int64_t blocks = ((a.dm.rows + groups - 1) / groups + 7) / 8 * 8;
  blocks = blocks > sms ? sms : blocks;
  const int block = (int)groups * threads;
  cudaError_t e;
  if (backward) {
    const size_t smem = ring_bytes(block, kBackwardStages, 2, NV);
    const auto kernel = k_norm_backward_ring<T, P, C, LANES, kBackwardStages>;
    a.parts = (int)(blocks < a.dm.rows ? blocks : a.dm.rows);
    static std::atomic<bool> allowed[64];
    if ((e = allow_smem(kernel, allowed)) != cudaSuccess) return e;
    kernel<<<(unsigned)blocks, block, smem, st>>>(
        static_cast<const T *>(a.dy), a.dys, static_cast<const T *>(a.x), a.xs, static_cast<const P *>(a.weight),
        a.mean, a.rstd, a.dm.rows, a.dm.width, static_cast<T *>(a.out), a.outs, a.part, threads);
  } else {
    const size_t smem = ring_bytes(block, kForwardStages, 1, NV);
    const auto kernel = k_norm_ring<T, P, C, LANES, kForwardStages>;
    static std::atomic<bool> allowed[64];
    if ((e = allow_smem(kernel, allowed)) != cudaSuccess) return e;
    kernel<<<(unsigned)blocks, block, smem, st>>>(
        static_cast<const T *>(a.x), a.xs, static_cast<const P *>(a.weight), static_cast<const P *>(a.bias), a.dm.eps,
        a.dm.rows, a.dm.width, static_cast<T *>(a.out), a.outs, a.mean_out, a.rstd_out, threads);
  }
  return cudaGetLastError();
}

enum NormPath { kRing, kVectors, kElements };

template <class T, class P>
cudaError_t launch_norm_typed(NormArgs &a, NormPath path, bool backward, cudaStream_t st) {
  constexpr int N = 16 / (int)sizeof(T);
  if (path == kRing) {
    // narrow rows share a warp: 8 or 16 lanes each.  The elements beside the vectors need 2 N threads.
    const bool whole = rows_aligned16(a.x, a.xs, a.dm.rows, sizeof(T)) && a.dm.width % N == 0;
    const NormShape s = norm_shape(a.dm.width / N, N, whole || N == 4 ? 8 : 16);
    if (s.threads > 32)  // a thread holds more than 16 columns
      return s.columns <= 24 ? launch_ring_shape<T, P, 24, 0>(a, s.threads, backward, st)
                             : launch_ring_shape<T, P, 32, 0>(a, s.threads, backward, st);
    if (s.threads == 32)
      return s.columns <= 24 ? launch_ring_shape<T, P, 24, 32>(a, 32, backward, st)
                             : launch_ring_shape<T, P, 32, 32>(a, 32, backward, st);
    if (s.threads == 16)
      switch (s.columns) {
        case 8: return launch_ring_shape<T, P, 8, 16>(a, 16, backward, st);
        case 16: return launch_ring_shape<T, P, 16, 16>(a, 16, backward, st);
        case 24: return launch_ring_shape<T, P, 24, 16>(a, 16, backward, st);
        default: return launch_ring_shape<T, P, 32, 16>(a, 16, backward, st);
      }
    switch (s.columns) {
      case 8: return launch_ring_shape<T, P, 8, 8>(a, 8, backward, st);
      case 16: return launch_ring_shape<T, P, 16, 8>(a, 8, backward, st);
      case 24: return launch_ring_shape<T, P, 24, 8>(a, 8, backward, st);
      default: return launch_ring_shape<T, P, 32, 8>(a, 8, backward, st);
    }
  }
  const NormShape s = path == kElements ? norm_shape(a.dm.width, 1) : norm_shape((a.dm.width + N - 1) / N, N);
  if (path == kVectors)  // above kRingWidth
    return s.columns <= 24 ? launch_norm_shape<T, P, N, 24, false>(a, s.threads, backward, st)
                           : launch_norm_shape<T, P, N, 32, false>(a, s.threads, backward, st);
  if (s.threads > 32)
    return s.columns <= 24 ? launch_norm_shape<T, P, 1, 24, false>(a, s.threads, backward, st)
                           : launch_norm_shape<T, P, 1, 32, false>(a, s.threads, backward, st);
  switch (s.columns) {
    case 8: return launch_norm_shape<T, P, 1, 8, true>(a, 32, backward, st);
    case 16: return launch_norm_shape<T, P, 1, 16, true>(a, 32, backward, st);
    case 24: return launch_norm_shape<T, P, 1, 24, true>(a, 32, backward, st);
    default: return launch_norm_shape<T, P, 1, 32, true>(a, 32, backward, st);
  }
}

cudaError_t launch_norm(NormArgs &a, bool backward, cudaStream_t st) {
  const int e = dtype_bytes(a.dm.dtype);
  const int64_t rows = a.dm.rows;
  // every row of p equally far from a 16-byte boundary as that row of x?
  auto like_x = [&](const void *p, int64_t stride) {
    return p == nullptr || (((reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(a.x)) & 15) == 0 &&
                            (rows <= 1 || ((stride - a.xs) * e) % 16 == 0));
  };
  NormPath path = kElements;
  if (a.dm.width <= kRingWidth) {
    if (like_x(a.out, a.outs) && like_x(a.dy, a.dys)) path = kRing;
  } else if (rows_aligned16(a.x, a.xs, rows, e) && like_x(a.out, a.outs) && like_x(a.dy, a.dys) &&
             aligned_to(a.weight, 16) && aligned_to(a.bias, 16)) {
    path = kVectors;
  }
  const bool same = a.dm.param_dtype != RVQ_DTYPE_F32;
  switch (a.dm.dtype) {
    case RVQ_DTYPE_F32: return launch_norm_typed<float, float>(a, path, backward, st);
    case RVQ_DTYPE_BF16:
      return same ? launch_norm_typed<__nv_bfloat16, __nv_bfloat16>(a, path, backward, st)
                  : launch_norm_typed<__nv_bfloat16, float>(a, path, backward, st);
    default:
      return same ? launch_norm_typed<__half, __half>(a, path, backward, st)
                  : launch_norm_typed<__half, float>(a, path, backward, st);
  }
}

template <class P>
cudaError_t launch_params(const NormArgs &a, void *dweight, void *dbias, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.dm.width + 31) / 32, 2);
  cfg.blockDim = dim3(32 * kSumRows);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_norm_params<P>, (const float *)a.part, a.parts, (int)a.dm.width,
                            static_cast<P *>(dweight), static_cast<P *>(dbias));
}

rvq_status check_norm(const rvq_norm_dims &dm) {
  if (dm.rows < 0 || dm.width <= 0 || !dtype_bytes(dm.dtype) || !dtype_bytes(dm.param_dtype)) return RVQ_ERR_INVALID_ARG;
  if (!(dm.eps >= 0.f)) return RVQ_ERR_INVALID_ARG;
  if (dm.param_dtype != RVQ_DTYPE_F32 && dm.param_dtype != dm.dtype) return RVQ_ERR_INVALID_ARG;
  if (dm.width > kNormMaxWidth) return RVQ_ERR_UNSUPPORTED;
  return RVQ_OK;
}
// A tensor of rows: not null, aligned to its elements, rows that do not overlap.
bool rows_ok(const void *p, int64_t stride, const rvq_norm_dims &dm) {
  return p && aligned_to(p, dtype_bytes(dm.dtype)) && (stride >= dm.width || dm.rows <= 1);
}
// Rows that may be written where the rows of `in` are read: blocks take rows in any order.
bool apart(const void *out, int64_t out_stride, const void *in, int64_t in_stride, const rvq_norm_dims &dm) {
  const int e = dtype_bytes(dm.dtype);
  return rows_apart(out, out_stride * e, in, in_stride * e, dm.rows, (int64_t)dm.width * e);
}

}  // namespace
}  // namespace rvq

extern "C" {

RVQ_API rvq_status rvq_layer_norm(rvq_norm_dims dims, const void *x, int64_t x_stride, const void *weight,
                                  const void *bias, void *y, int64_t y_stride, float *mean, float *rstd,
                                  rvq_stream_t stream) {
  using namespace rvq;
  const rvq_status s = check_norm(dims);
  if (s != RVQ_OK || dims.rows == 0) return s;
  const int pe = dtype_bytes(dims.param_dtype);
  if (!rows_ok(x, x_stride, dims) || !rows_ok(y, y_stride, dims) || !apart(y, y_stride, x, x_stride, dims))
    return RVQ_ERR_INVALID_ARG;
  if (!aligned_to(weight, pe) || !aligned_to(bias, pe) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return RVQ_ERR_INVALID_ARG;
  NormArgs a{};
  a.dm = dims, a.x = x, a.xs = x_stride, a.weight = weight, a.bias = bias, a.out = y, a.outs = y_stride;
  a.mean_out = mean, a.rstd_out = rstd;
  return launch_norm(a, false, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? RVQ_OK : RVQ_ERR_CUDA;
}

RVQ_API size_t rvq_layer_norm_workspace_bytes(int64_t rows, int32_t width) {
  if (rows < 0 || width <= 0 || width > rvq::kNormMaxWidth) return 0;
  return rvq::align_up(((size_t)rvq::norm_parts(rows, width) + (rows == 0)) * 2 * (size_t)width * sizeof(float));
}

RVQ_API rvq_status rvq_layer_norm_backward(rvq_norm_dims dims, const void *dy, int64_t dy_stride, const void *x,
                                           int64_t x_stride, const void *weight, const float *mean, const float *rstd,
                                           void *dx, int64_t dx_stride, void *dweight, void *dbias, void *workspace,
                                           size_t workspace_bytes, rvq_stream_t stream) {
  using namespace rvq;
  const rvq_status s = check_norm(dims);
  if (s != RVQ_OK) return s;
  const int pe = dtype_bytes(dims.param_dtype);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!aligned_to(weight, pe) || !aligned_to(dweight, pe) || !aligned_to(dbias, pe)) return RVQ_ERR_INVALID_ARG;
  if (dims.rows == 0) {
    const size_t bytes = (size_t)dims.width * pe;
    if (dweight && cudaMemsetAsync(dweight, 0, bytes, st) != cudaSuccess) return RVQ_ERR_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, bytes, st) != cudaSuccess) return RVQ_ERR_CUDA;
    return RVQ_OK;
  }
  if (!rows_ok(dy, dy_stride, dims) || !rows_ok(x, x_stride, dims) || (dx && !rows_ok(dx, dx_stride, dims)))
    return RVQ_ERR_INVALID_ARG;
  if (dx && (!apart(dx, dx_stride, dy, dy_stride, dims) || !apart(dx, dx_stride, x, x_stride, dims)))
    return RVQ_ERR_INVALID_ARG;
  if (!mean || !rstd || !aligned_to(mean, 4) || !aligned_to(rstd, 4)) return RVQ_ERR_INVALID_ARG;
  const bool params = dweight || dbias;
  if (params && (!workspace || !aligned_to(workspace, 16) ||
                 workspace_bytes < rvq_layer_norm_workspace_bytes(dims.rows, dims.width)))
    return RVQ_ERR_INVALID_ARG;
  if (!dx && !params) return RVQ_OK;
  NormArgs a{};
  a.dm = dims, a.dy = dy, a.dys = dy_stride, a.x = x, a.xs = x_stride, a.weight = weight, a.mean = mean, a.rstd = rstd;
  a.out = dx, a.outs = dx_stride, a.part = params ? static_cast<float *>(workspace) : nullptr;
  if (launch_norm(a, true, st) != cudaSuccess) return RVQ_ERR_CUDA;
  if (!params) return RVQ_OK;
  const cudaError_t e = dims.param_dtype == RVQ_DTYPE_F32    ? launch_params<float>(a, dweight, dbias, st)
                        : dims.param_dtype == RVQ_DTYPE_BF16 ? launch_params<__nv_bfloat16>(a, dweight, dbias, st)
                                                             : launch_params<__half>(a, dweight, dbias, st);
  return e == cudaSuccess ? RVQ_OK : RVQ_ERR_CUDA;
}

}  // extern "C"
