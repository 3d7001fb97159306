// What the two passes of the root-mean-square norm share (rvq_rms.cu,
// rvq_rms_backward.cu): arguments, launch shapes, and the checks of a call.
#pragma once

#include "rvq_dropout.cuh"
#include "rvq_internal.cuh"
#include "rvq_norm_rows.cuh"
#include "rvq_overlap.h"
#include "sm103_ptx.cuh"

namespace rvq {
namespace {

struct RmsArgs {
  rvq_norm_dims dm;
  const void *x, *residual;  // forward
  const void *dy, *dtotal;   // backward
  void *total;               // the sum: written by the forward pass (nullable), read by the backward pass
  void *y;                   // forward: y; backward: dresidual (nullable)
  void *dx;                  // backward, through the dropout (nullable)
  int64_t xs, rs, dys, dts, ts, ys, dxs;
  const void *weight;
  float *rstd;
  uint8_t *q;  // nullable
  int64_t qs;
  void *scales;
  int32_t block, scale_type, scale_count;
  DropoutMask mask;
  float *part;
  int parts;
};

// The weight at column c, in whichever type it is (one where there is none).
template <class T>
__device__ __forceinline__ float weight_at(const RmsArgs &a, int c) {
  if (a.weight == nullptr) return 1.f;
  return a.dm.param_dtype == RVQ_DTYPE_F32 ? static_cast<const float *>(a.weight)[c]
                                           : to_float(static_cast<const T *>(a.weight)[c]);
}

// Threads of a block of the ring kernels, one on an SM: 128 registers each, or 168 in 32 bits, whose slots leave no room
// for more threads.
constexpr int kRmsThreads = 512;
template <class T>
constexpr int rms_threads() { return sizeof(T) == 4 ? 384 : kRmsThreads; }

// Rows that a thread has slots for: the one it works on and the next.  (Three leave room for fewer warps: 192 000 x 1024
// bf16 with dropout, both passes, 691 us against 558.)
constexpr int kStages = 2;

// How a row lies in a ring kernel: over `threads`, `lanes` of a warp or (lanes 0)
// whole warps, at most `columns` a thread.  Each shape is an instance of its own
// in three types, with and without a mask, in both passes; those that are here
// are for rows that fill them.  8 and 16 lanes have no 24 columns, as layer norm's
// table does, and widths between lose by it, most with a mask, which is worked out
// for empty columns too (60 000 000 bf16 elements with a residual, forward and
// backward pass; 32 columns a lane, 24): 264 wide 77 + 98 us, 83 + 86; with a mask
// 144 + 187, 121 + 161; 320 wide 87 + 82, 85 + 78; with a mask 120 + 157, 101 + 135;
// 384 f32 with a mask 152 + 234, 174 + 222.  Whole warps are as many as the row
// needs, so that 32 columns are nearly full there.
struct RmsShape {
  int lanes, columns, threads;
};
inline RmsShape rms_shape(int width, int bytes, bool whole, int least) {
  // the elements beside the vectors need 2 N lanes of their own
  const int n = 16 / bytes, units = width / n;
  least = least < 8 ? 8 : least;
  if (!whole && least < 2 * n) least = 2 * n;
  const NormShape s = norm_shape(units, n, least);
  if (s.threads <= 8) return {8, s.columns <= 16 ? 16 : 32, 8};
  if (s.threads <= 16) return {16, 32, 16};
  if (s.threads <= 32) return {32, s.columns <= 24 ? 24 : 32, 32};
  return {0, 32, ((units * n + 31) / 32 + 31) / 32 * 32};
}

// Whether rows at p start as far from a 16-byte boundary as those at `like`.
inline bool rows_alike(const void *p, int64_t stride, const void *like, int64_t like_stride, int64_t rows, int bytes) {
  return p == nullptr || (((reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(like)) & 15) == 0 &&
                          (rows <= 1 || ((stride - like_stride) * bytes) % 16 == 0));
}

// The rows (groups) of a block and the blocks of a ring kernel: no more rows a
// block than there are for the SMs, whole warps, and a multiple of 8 blocks, so
// that a block's rows start equally far from a 16-byte boundary.
struct RmsGrid {
  int groups;
  int64_t blocks;
};
template <class T>
RmsGrid rms_grid(int64_t rows, const RmsShape &s, size_t thread_bytes) {
  int most = rms_threads<T>() / s.threads;
  const int fit = (int)(kMostSmem / (thread_bytes * s.threads));
  most = most < fit ? most : fit;
  const int per_warp = s.lanes ? 32 / s.lanes : 1;
  most = most / per_warp * per_warp;
  int64_t groups = (rows + kSms - 1) / kSms;
  groups = groups > most ? most : groups;
  groups = (groups + per_warp - 1) / per_warp * per_warp;
  const int64_t blocks = ((rows + groups - 1) / groups + 7) / 8 * 8;
  return {(int)groups, blocks > kSms ? kSms : blocks};
}

rvq_status check_rms(const rvq_norm_dims &dm) {
  if (dm.rows < 0 || dm.width <= 0 || !dtype_bytes(dm.dtype) || !dtype_bytes(dm.param_dtype)) return RVQ_ERR_INVALID_ARG;
  if (!(dm.eps >= 0.f)) return RVQ_ERR_INVALID_ARG;
  if (dm.param_dtype != RVQ_DTYPE_F32 && dm.param_dtype != dm.dtype) return RVQ_ERR_INVALID_ARG;
  if (dm.width > kNormMaxWidth) return RVQ_ERR_UNSUPPORTED;
  return RVQ_OK;
}

// Whether what a call writes meets what else it writes or reads.  Blocks take
// rows in any order, so a tensor of rows may lie over one that is read row by
// row, and nothing in any other way.  (A set at null is none.)
struct Touched {
  RowSet set;
  bool rows;  // a tensor of the norm's rows
};
inline Touched rows_at(const void *p, int64_t stride, const rvq_norm_dims &dm) {
  const int e = dtype_bytes(dm.dtype);
  return {row_set(p, (int64_t)dm.width * e, dm.rows, stride * e), true};
}
inline Touched bytes_at(const void *p, int64_t bytes) { return {row_set(p, bytes, 1, 0), false}; }
template <int W, int R>
bool rms_apart(const Touched (&written)[W], const Touched (&read)[R]) {
  for (int i = 0; i < W; ++i) {
    const Touched &w = written[i];
    if (!w.set.base) continue;
    for (int j = i + 1; j < W; ++j)
      if (written[j].set.base && overlap(w.set, written[j].set) != Overlap::kNone) return false;
    for (const Touched &r : read) {
      if (!r.set.base) continue;
      const auto &x = w.set.axis[0], &y = r.set.axis[0];
      if (w.rows && r.rows && w.set.base == r.set.base && (x.count <= 1 || x.stride == y.stride)) continue;
      if (overlap(w.set, r.set) != Overlap::kNone) return false;
    }
  }
  return true;
}

}  // namespace
}  // namespace rvq
