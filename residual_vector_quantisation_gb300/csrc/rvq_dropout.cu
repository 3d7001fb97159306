// Dropout with a mask that is never stored (rvq_dropout): y = x / (1 - p) where
// the element stays, 0 where it does not, plus a residual.  The gradient is the
// same call on dy.
#include "rvq_dropout.cuh"
#include "rvq_internal.cuh"
#include "rvq_overlap.h"

namespace rvq {
namespace {

struct DropoutArgs {
  const void *x, *residual;
  void *y;
  int64_t xs, rs, ys;  // strides in elements
  int64_t rows, width;
  DropoutMask mask;
};

constexpr int kThreads = 256;

// Groups of 8 elements that are whole vectors of a row (width a multiple of 8,
// rows on 16-byte boundaries); one group a thread at a time.  Bound by bandwidth:
// 192 000 x 1024 bf16, forward with a residual and backward, 299 us (97 % of a
// copy's rate); the generator's 60 or so instructions for 8 elements are hidden.
template <class T>
__global__ void __launch_bounds__(kThreads) k_dropout(const DropoutArgs a) {
  constexpr int N = 16 / (int)sizeof(T), V = 8 / N;
  const Dropped drop(a.mask);
  const int64_t each = a.width / 8, groups = a.rows * each;
  for (int64_t g = blockIdx.x * (int64_t)kThreads + threadIdx.x; g < groups; g += (int64_t)gridDim.x * kThreads) {
    const int64_t row = a.rows == 1 ? 0 : g / each, col = (g - row * each) * 8;
    const T *x = static_cast<const T *>(a.x) + row * a.xs + col;
    T *y = static_cast<T *>(a.y) + row * a.ys + col;
    uint4 in[V], add[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      in[v] = reinterpret_cast<const uint4 *>(x)[v];
      add[v] = a.residual ? reinterpret_cast<const uint4 *>(static_cast<const T *>(a.residual) + row * a.rs + col)[v]
                          : make_uint4(0, 0, 0, 0);
    }
    const uint32_t bits = drop.group((uint64_t)g);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f[N], r[N];
      unpack16<T>(in[v], f);
      unpack16<T>(add[v], r);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        f[i] = Dropped::at(bits, v * N + i) ? 0.f : __fmul_rn(f[i], drop.factor);
        if (a.residual) f[i] = __fadd_rn(f[i], r[i]);
      }
      reinterpret_cast<uint4 *>(y)[v] = pack16<T>(f);
    }
  }
}

// Anything else (rows with gaps of no whole vectors, or without gaps and with
// elements beside the last whole group): a warp takes 256 elements, each lane
// working out one group of them, so that lanes next to one another read and write
// next to one another.  Bound by instructions: 58 536 x 1025 bf16, rows 1031 apart,
// 127 us (bytes alone 35).
template <class T>
__global__ void __launch_bounds__(kThreads) k_dropout_elements(const DropoutArgs a) {
  const Dropped drop(a.mask);
  const int lane = threadIdx.x & 31;
  const int64_t all = a.rows * a.width, warps = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t e0 = (blockIdx.x * (int64_t)(kThreads / 32) + (threadIdx.x >> 5)) * 256; e0 < all; e0 += warps * 256) {
    const uint32_t bits = drop.group((uint64_t)(e0 / 8 + lane));
    // Where the lane's elements lie, 32 apart: one division, then sums.  All are read before any is written (y may be
    // x, so that the compiler keeps reads behind the writes that stand before them).
    const int64_t row0 = (e0 + lane) / a.width, col0 = e0 + lane - row0 * a.width;
    const int left = (int)min(all - e0 - lane, (int64_t)256);  // element i is there: i * 32 < left
    auto walk = [&](int64_t stride, auto at) {
      int64_t col = col0, place = row0 * stride + col0;
      const int64_t gap = stride - a.width;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i * 32 < left) at(i, place);
        place += 32;
        for (col += 32; col >= a.width; col -= a.width) place += gap;
      }
    };
    float f[8], r[8] = {};
    walk(a.xs, [&](int i, int64_t place) { f[i] = to_float(static_cast<const T *>(a.x)[place]); });
    if (a.residual) walk(a.rs, [&](int i, int64_t place) { r[i] = to_float(static_cast<const T *>(a.residual)[place]); });
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[i] = Dropped::at(__shfl_sync(0xffffffffu, bits, i * 4 + lane / 8), lane & 7) ? 0.f : __fmul_rn(f[i], drop.factor);
      if (a.residual) f[i] = __fadd_rn(f[i], r[i]);
    }
    walk(a.ys, [&](int i, int64_t place) { static_cast<T *>(a.y)[place] = from_float<T>(f[i]); });
  }
}

template <class T>
cudaError_t launch_dropout(DropoutArgs a, cudaStream_t st) {
  // rows without anything between them are one row
  if ((a.xs == a.width && a.ys == a.width && (!a.residual || a.rs == a.width)) || a.rows == 1)
    a.width *= a.rows, a.rows = 1;
  const auto aligned = [&](const void *p, int64_t stride) { return rows_aligned16(p, stride, a.rows, sizeof(T)); };
  const bool vectors = a.width % 8 == 0 && aligned(a.x, a.xs) && aligned(a.y, a.ys) && (!a.residual || aligned(a.residual, a.rs));
  const int64_t items = (a.rows * a.width + 7) / 8;
  const int64_t want = (items + kThreads - 1) / kThreads, most = 152 * 8 * 16;
  const unsigned blocks = (unsigned)(want < most ? want : most);
  if (vectors)
    k_dropout<T><<<blocks, kThreads, 0, st>>>(a);
  else
    k_dropout_elements<T><<<blocks, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace rvq

extern "C" {

RVQ_API rvq_status rvq_dropout(rvq_dropout_dims dims, const void *x, int64_t x_stride, const void *residual,
                               int64_t residual_stride, const rvq_dropout_mask *mask, void *y, int64_t y_stride,
                               rvq_stream_t stream) {
  using namespace rvq;
  const int64_t rows = dims.rows, width = dims.width;
  const int e = dtype_bytes(dims.dtype);
  DropoutArgs a{x, residual, y, x_stride, residual_stride, y_stride, rows, width, {}};
  if (rows < 0 || width < 0 || !e || !mask || !dropout_mask(*mask, a.mask)) return RVQ_ERR_INVALID_ARG;
  if (rows > 0 && width > ((int64_t)1 << 48) / rows) return RVQ_ERR_UNSUPPORTED;
  if (rows == 0 || width == 0) return RVQ_OK;
  const auto ok = [&](const void *p, int64_t stride) { return p && aligned_to(p, e) && (rows <= 1 || stride >= width); };
  if (!ok(x, x_stride) || !ok(y, y_stride) || (residual && !ok(residual, residual_stride))) return RVQ_ERR_INVALID_ARG;
  if (!rows_apart(y, y_stride * e, x, x_stride * e, rows, width * e) ||
      (residual && !rows_apart(y, y_stride * e, residual, residual_stride * e, rows, width * e)) ||
      (mask->step && overlap(row_set(y, width * e, rows, y_stride * e), row_set(mask->step, 8, 1, 0)) != Overlap::kNone))
    return RVQ_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = dims.dtype == RVQ_DTYPE_F32    ? launch_dropout<float>(a, st)
                          : dims.dtype == RVQ_DTYPE_BF16 ? launch_dropout<__nv_bfloat16>(a, st)
                                                         : launch_dropout<__half>(a, st);
  return err == cudaSuccess ? RVQ_OK : RVQ_ERR_CUDA;
}

}  // extern "C"
