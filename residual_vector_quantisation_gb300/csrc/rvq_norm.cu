// Layer norm over rows, forward and backward (rvq_layer_norm,
// rvq_layer_norm_backward).
//
// A row's elements are held in registers from one read: a warp per row up to
// 1024 columns, a block of 64 .. 512 threads per row above, C columns a thread
// (8, 16, 24 or 32, the fewest that hold the row).  The variance is the mean
// square of the centred values, so a row with a large mean loses nothing.
// The columns of a thread come as 16-byte vectors (N = 4 or 8 elements) where
// every row and parameter starts on a 16-byte boundary, else one by one
// (N = 1, neighbouring threads on neighbouring elements).
#include "rvq_internal.cuh"
#include "rvq_rows.cuh"

namespace rvq {
namespace {

constexpr int kNormMaxWidth = 16384;
constexpr int kNormWarpWidth = 1024;   // widest row that one warp holds
constexpr int kNormWarps = 4;          // rows (warps) of a block up to that width
constexpr int kNormParts = 608;        // most blocks of the backward pass (four on each of 152 SMs)
constexpr int kNormPartsWide = 304;    // ... above kNormWarpWidth

inline int norm_parts(int64_t rows, int width) {
  const int most = width <= kNormWarpWidth ? kNormParts : kNormPartsWide;
  return rows < most ? (int)rows : most;
}

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

// The blocks' sums, added in a fixed order: 32 columns a block, 16 lanes of rows.
constexpr int kSumRows = 16;
template <class P>
__global__ void __launch_bounds__(32 * kSumRows)
    k_norm_params(const float *__restrict__ part, int parts, int width, P *dweight, P *dbias) {
  __shared__ float box[kSumRows][33];
  P *out = blockIdx.y ? dbias : dweight;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const float *p = part + (int64_t)blockIdx.y * width + c;
  float s = 0.f;
  if (c < width)
    for (int i = ty; i < parts; i += kSumRows) s += p[(int64_t)i * 2 * width];
  box[ty][lane] = s;
  __syncthreads();
  if (ty == 0 && c < width) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kSumRows; ++i) s += box[i][lane];
    out[c] = from_float<P>(s);
  }
}

// How a row of `width` columns is laid over threads.
struct NormShape {
  int threads;  // of a row
  int columns;  // of a thread (C)
};
inline NormShape norm_shape(int width) {
  int threads = 32;
  while (threads * 32 < width) threads *= 2;
  int c = ((width + threads - 1) / threads + 7) / 8 * 8;
  return {threads, c};
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
  int parts;
};

template <class T, class P, int N, int C, bool WARP>
cudaError_t launch_norm_shape(const NormArgs &a, int threads, bool backward, cudaStream_t st) {
  const int block = WARP ? 32 * kNormWarps : threads;
  if (backward) {
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

template <class T, class P, int N>
cudaError_t launch_norm_typed(const NormArgs &a, bool backward, cudaStream_t st) {
  const NormShape s = norm_shape(a.dm.width);
  if (s.threads == 32) {
    switch (s.columns) {
      case 8: return launch_norm_shape<T, P, N, 8, true>(a, 32, backward, st);
      case 16: return launch_norm_shape<T, P, N, 16, true>(a, 32, backward, st);
      case 24: return launch_norm_shape<T, P, N, 24, true>(a, 32, backward, st);
      default: return launch_norm_shape<T, P, N, 32, true>(a, 32, backward, st);
    }
  }
  // above 1024 columns a thread holds more than 16 of them
  if (s.columns <= 24) return launch_norm_shape<T, P, N, 24, false>(a, s.threads, backward, st);
  return launch_norm_shape<T, P, N, 32, false>(a, s.threads, backward, st);
}

template <class T, class P>
cudaError_t launch_norm_aligned(const NormArgs &a, bool vectors, bool backward, cudaStream_t st) {
  return vectors ? launch_norm_typed<T, P, 16 / (int)sizeof(T)>(a, backward, st)
                 : launch_norm_typed<T, P, 1>(a, backward, st);
}

cudaError_t launch_norm(const NormArgs &a, bool vectors, bool backward, cudaStream_t st) {
  const bool same = a.dm.param_dtype != RVQ_DTYPE_F32;
  switch (a.dm.dtype) {
    case RVQ_DTYPE_F32: return launch_norm_aligned<float, float>(a, vectors, backward, st);
    case RVQ_DTYPE_BF16:
      return same ? launch_norm_aligned<__nv_bfloat16, __nv_bfloat16>(a, vectors, backward, st)
                  : launch_norm_aligned<__nv_bfloat16, float>(a, vectors, backward, st);
    default:
      return same ? launch_norm_aligned<__half, __half>(a, vectors, backward, st)
                  : launch_norm_aligned<__half, float>(a, vectors, backward, st);
  }
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

}  // namespace
}  // namespace rvq

extern "C" {

RVQ_API rvq_status rvq_layer_norm(rvq_norm_dims dims, const void *x, int64_t x_stride, const void *weight,
                                  const void *bias, void *y, int64_t y_stride, float *mean, float *rstd,
                                  rvq_stream_t stream) {
  using namespace rvq;
  const rvq_status s = check_norm(dims);
  if (s != RVQ_OK || dims.rows == 0) return s;
  const int e = dtype_bytes(dims.dtype), pe = dtype_bytes(dims.param_dtype);
  if (!rows_ok(x, x_stride, dims) || !rows_ok(y, y_stride, dims)) return RVQ_ERR_INVALID_ARG;
  if (!aligned_to(weight, pe) || !aligned_to(bias, pe) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return RVQ_ERR_INVALID_ARG;
  const bool vectors = rows_aligned16(x, x_stride, dims.rows, e) && rows_aligned16(y, y_stride, dims.rows, e) &&
                       aligned_to(weight, 16) && aligned_to(bias, 16);
  NormArgs a{};
  a.dm = dims, a.x = x, a.xs = x_stride, a.weight = weight, a.bias = bias, a.out = y, a.outs = y_stride;
  a.mean_out = mean, a.rstd_out = rstd;
  return launch_norm(a, vectors, false, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? RVQ_OK : RVQ_ERR_CUDA;
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
  const int e = dtype_bytes(dims.dtype), pe = dtype_bytes(dims.param_dtype);
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
  if (!mean || !rstd || !aligned_to(mean, 4) || !aligned_to(rstd, 4)) return RVQ_ERR_INVALID_ARG;
  const bool params = dweight || dbias;
  if (params && (!workspace || !aligned_to(workspace, 16) ||
                 workspace_bytes < rvq_layer_norm_workspace_bytes(dims.rows, dims.width)))
    return RVQ_ERR_INVALID_ARG;
  if (!dx && !params) return RVQ_OK;
  const bool vectors = rows_aligned16(x, x_stride, dims.rows, e) && rows_aligned16(dy, dy_stride, dims.rows, e) &&
                       (!dx || rows_aligned16(dx, dx_stride, dims.rows, e)) && aligned_to(weight, 16);
  NormArgs a{};
  a.dm = dims, a.dy = dy, a.dys = dy_stride, a.x = x, a.xs = x_stride, a.weight = weight, a.mean = mean, a.rstd = rstd;
  a.out = dx, a.outs = dx_stride, a.part = params ? static_cast<float *>(workspace) : nullptr;
  a.parts = norm_parts(dims.rows, dims.width);
  if (launch_norm(a, vectors, true, st) != cudaSuccess) return RVQ_ERR_CUDA;
  if (!params) return RVQ_OK;
  const dim3 grid((unsigned)(dims.width + 31) / 32, 2);
  if (dims.param_dtype == RVQ_DTYPE_F32)
    k_norm_params<float><<<grid, 32 * kSumRows, 0, st>>>(a.part, a.parts, dims.width, static_cast<float *>(dweight),
                                                        static_cast<float *>(dbias));
  else if (dims.param_dtype == RVQ_DTYPE_BF16)
    k_norm_params<__nv_bfloat16><<<grid, 32 * kSumRows, 0, st>>>(a.part, a.parts, dims.width,
                                                                static_cast<__nv_bfloat16 *>(dweight),
                                                                static_cast<__nv_bfloat16 *>(dbias));
  else
    k_norm_params<__half><<<grid, 32 * kSumRows, 0, st>>>(a.part, a.parts, dims.width, static_cast<__half *>(dweight),
                                                         static_cast<__half *>(dbias));
  return cudaGetLastError() == cudaSuccess ? RVQ_OK : RVQ_ERR_CUDA;
}

}  // extern "C"
