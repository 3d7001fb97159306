// Gradients of the root-mean-square norm (rvq_rms_norm_backward).
//
//   u = h r,  g = dy w,  dh = r (g - u mean(g u)) + dtotal,  dx = drop(dh),  dw = sum of dy u
#include "rvq_rms.cuh"

namespace rvq {
namespace {

// Rows through a ring in shared memory, as in the forward pass: dresidual and dx
// per row, and each block's sums of dy u over its rows into part[block][width].
// 60 000 x 1024 bf16 with the sum's gradient: 81 us (bytes alone: 72), with
// dropout, one tensor more, 108 (90).
template <class T, int C, int LANES, bool DROP>
__global__ void __launch_bounds__(rms_threads<T>(), 1) k_rms_backward_ring(const RmsArgs a, const int tpr_) {
  constexpr int N = 16 / (int)sizeof(T), NV = C / N, H = N / 2;
  extern __shared__ uint4 ring[];
  __shared__ float box[2 * kRmsThreads / 32][1][16];
  const int tpr = LANES ? LANES : tpr_, group = threadIdx.x / tpr, groups = blockDim.x / tpr, width = a.dm.width;
  const int64_t rows = a.dm.rows, step = (int64_t)gridDim.x * groups, first = blockIdx.x + (int64_t)group * gridDim.x;
  const T *hp = static_cast<const T *>(a.total), *dp = static_cast<const T *>(a.dy), *tp = static_cast<const T *>(a.dtotal);
  const Columns<N, NV> c(hp + (int64_t)blockIdx.x * a.ts, sizeof(T), width, tpr, threadIdx.x % tpr);
  const bool three = tp != nullptr;
  const int arrays = three ? 3 : 2;
  const float inv = 1.f / (float)width;
  const F2 zero = f2(0.f, 0.f);
  F2 g[NV][H], dw[NV][H];
  float ge = c.edge >= 0 ? weight_at<T>(a, c.edge) : 0.f, dwe = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < H; ++i) {
      g[j][i] = c.has(j) ? f2(weight_at<T>(a, c.column(j) + 2 * i), weight_at<T>(a, c.column(j) + 2 * i + 1)) : zero;
      dw[j][i] = zero;
    }
  uint4 *slot = ring + threadIdx.x;  // [stage][h, dy, dtotal][j][thread], then [stage][thread] of rstd
  float *stat = reinterpret_cast<float *>(ring + kStages * arrays * NV * blockDim.x) + threadIdx.x;
  for (int i = 0; i < kStages * arrays * NV; ++i) slot[i * blockDim.x] = make_uint4(0, 0, 0, 0);
  auto fetch = [&](int64_t row, int stage) {
    uint4 *at = slot + stage * arrays * NV * blockDim.x;
    if (row < rows) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (c.has(j)) {
          copy16((uint32_t)__cvta_generic_to_shared(at + j * blockDim.x), hp + row * a.ts + c.column(j));
          copy16((uint32_t)__cvta_generic_to_shared(at + (NV + j) * blockDim.x), dp + row * a.dys + c.column(j));
          if (three) copy16((uint32_t)__cvta_generic_to_shared(at + (2 * NV + j) * blockDim.x), tp + row * a.dts + c.column(j));
        }
      copy4((uint32_t)__cvta_generic_to_shared(stat + stage * blockDim.x), a.rstd + row);
    } else if (LANES) {  // a row past the end has nothing to add to the sums
      asm volatile("" ::: "memory");  // after the last reading of these slots
#pragma unroll
      for (int j = 0; j < 2 * NV; ++j) at[j * blockDim.x] = make_uint4(0, 0, 0, 0);
      stat[stage * blockDim.x] = 0.f;
    }
    copies_end();
  };
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) fetch(first + k * step, k);
  auto edge_of = [&](const T *p, int64_t stride, int64_t row) {
    return p && c.edge >= 0 && row < rows ? to_float(p[row * stride + c.edge]) : 0.f;
  };
  float he_next = edge_of(hp, a.ts, first), de_next = edge_of(dp, a.dys, first), te_next = edge_of(tp, a.dts, first);
  const Dropped dropped(a.mask);
  int turn = 0, stage = 0;
  // the groups of a warp stay together
  constexpr int kPerWarp = LANES ? 32 / (LANES ? LANES : 32) : 1;
  const int64_t ahead = (int64_t)(group % kPerWarp) * gridDim.x;
  for (int64_t row = first; row - ahead < rows; row += step) {
    const bool there = row < rows;
    fetch(row + (kStages - 1) * step, (stage + kStages - 1) % kStages);
    const float he = he_next, de = de_next, te = te_next;
    he_next = edge_of(hp, a.ts, row + step), de_next = edge_of(dp, a.dys, row + step), te_next = edge_of(tp, a.dts, row + step);
    copies_wait<kStages - 1>();
    // what is dropped of all the thread's vectors, in one word, one group after the other: worked out where it is used,
    // it spilled 124 bytes a thread (instances of several warps a row still spill up to 32, without a mask those of 16
    // bits in one warp 4 to 12)
    uint32_t gone = 0;
    if constexpr (DROP) {
      if (a.dx)
#pragma unroll 1
        for (int j = 0; j < NV; ++j) gone |= dropped.from<N>((uint64_t)(row * width + c.column(j))) << (j * H);
    }
    const float r = stat[stage * blockDim.x];
    const F2 r2 = f2(r, r);
    const uint4 *hv = slot + stage * arrays * NV * blockDim.x, *dv = hv + NV * blockDim.x, *tv = dv + NV * blockDim.x;
    F2 s2 = zero;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      F2 h[H], d[H];
      unpack_pairs<T>(read16(hv + j * blockDim.x), h);
      unpack_pairs<T>(read16(dv + j * blockDim.x), d);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const F2 u = h[i] * r2;  // no column: d = 0
        s2 = fma2(d[i] * g[j][i], u, s2);
        dw[j][i] = fma2(d[i], u, dw[j][i]);
      }
    }
    const float ue = he * r;
    if (c.edge >= 0) dwe = fmaf(de, ue, dwe);
    if (a.y != nullptr || a.dx != nullptr) {
      const float2 both = floats(s2);
      float s[1] = {both.x + both.y};
      if (c.edge >= 0) s[0] = fmaf(de * ge, ue, s[0]);
      group_sum<1, LANES>(s, box, turn, group, tpr);
      if constexpr (LANES != 0) __syncwarp();  // the second reading of the row stays below: moved up, it spills
      const float m = s[0] * inv;
      const F2 minus = f2(-m, -m);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        F2 h[H], d[H];
        unpack_pairs<T>(read16(hv + j * blockDim.x), h);
        unpack_pairs<T>(read16(dv + j * blockDim.x), d);
#pragma unroll
        for (int i = 0; i < H; ++i) h[i] = fma2(h[i] * r2, minus, d[i] * g[j][i]) * r2;
        if (three) {
          unpack_pairs<T>(read16(tv + j * blockDim.x), d);
#pragma unroll
          for (int i = 0; i < H; ++i) h[i] = h[i] + d[i];
        }
        const bool store = c.has(j) && there;
        if (a.y && store) *reinterpret_cast<uint4 *>(static_cast<T *>(a.y) + row * a.ys + c.column(j)) = pack_pairs<T>(h);
        if constexpr (DROP) {
          if (a.dx && store) {
            float f[N];
#pragma unroll
            for (int i = 0; i < H; ++i) {
              const float2 p = floats(h[i]);
              f[2 * i] = gone >> (j * H + i) & 1 ? 0.f : p.x * dropped.factor;
              f[2 * i + 1] = gone >> (16 + j * H + i) & 1 ? 0.f : p.y * dropped.factor;
            }
            *reinterpret_cast<uint4 *>(static_cast<T *>(a.dx) + row * a.dxs + c.column(j)) = pack16<T>(f);
          }
        }
      }
      if (c.edge >= 0 && there) {
        const float dh = fmaf(ue, -m, de * ge) * r + te;
        if (a.y) static_cast<T *>(a.y)[row * a.ys + c.edge] = from_float<T>(dh);
        if (DROP && a.dx)
          static_cast<T *>(a.dx)[row * a.dxs + c.edge] =
              from_float<T>(dropped.element((uint64_t)(row * width + c.edge)) ? 0.f : dh * dropped.factor);
      }
    }
    stage = (stage + 1) % kStages;
  }
  if (a.part == nullptr || blockIdx.x >= rows) return;  // (a block without rows has no part in the workspace)
  copies_wait<0>();
  __syncthreads();
  // the groups' sums through shared memory, added in their order
  float *sums = reinterpret_cast<float *>(ring), *mine = a.part + (int64_t)blockIdx.x * width;
  float *own = groups > 1 ? sums + (int64_t)group * width : mine;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (c.has(j))
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float2 w = floats(dw[j][i]);
        own[c.column(j) + 2 * i] = w.x, own[c.column(j) + 2 * i + 1] = w.y;
      }
  if (c.edge >= 0) own[c.edge] = dwe;
  if (groups == 1) return;
  __syncthreads();
  for (int i = threadIdx.x; i < width; i += blockDim.x) {
    float v = 0.f;
    for (int k = 0; k < groups; ++k) v += sums[k * width + i];
    mine[i] = v;
  }
}

// Any rows, element by element: a warp's (up to 1024 columns, 4 a block) or a
// block's, read twice (the second time from the L1 or L2); the sums of dy u in
// shared memory, each column's by one thread.  At most 304 blocks, whose latency
// bounds it: 60 000 x 1024 bf16 356 us (bytes alone: 54), 58 536 x 1025 365 (53).
constexpr int kAnyWidth = 1024, kAnyWarps = 4, kAnyThreads = 512;
template <class T, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kAnyWarps : kAnyThreads) k_rms_backward_any(const RmsArgs a, const bool drop) {
  extern __shared__ float sums[];  // [team][width]
  __shared__ float box[2][16];
  const int width = a.dm.width, lane = threadIdx.x & 31;
  const int warp = WARP ? 0 : threadIdx.x >> 5, warps = WARP ? 1 : blockDim.x >> 5;
  const int team = WARP ? threadIdx.x >> 5 : 0;
  constexpr int kTeams = WARP ? kAnyWarps : 1;
  float *dw = sums + team * width;
  const Dropped dropped(a.mask);
  const float inv = 1.f / (float)width;
  for (int c = WARP ? lane : threadIdx.x; c < width; c += WARP ? 32 : blockDim.x) dw[c] = 0.f;
  if constexpr (WARP)
    __syncwarp();
  else
    __syncthreads();
  int turn = 0;
  for (int64_t row = blockIdx.x * (int64_t)kTeams + team; row < a.dm.rows; row += (int64_t)gridDim.x * kTeams) {
    const T *h = static_cast<const T *>(a.total) + row * a.ts, *dy = static_cast<const T *>(a.dy) + row * a.dys;
    const T *dt = a.dtotal ? static_cast<const T *>(a.dtotal) + row * a.dts : nullptr;
    const float r = a.rstd[row];
    float s = 0.f;
    for (int c0 = warp * 256; c0 < width; c0 += warps * 256) {
      float u[8], d[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = c0 + i * 32 + lane;
        u[i] = c < width ? to_float(h[c]) * r : 0.f;
        d[i] = c < width ? to_float(dy[c]) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = c0 + i * 32 + lane;
        if (c >= width) continue;
        s = fmaf(d[i] * weight_at<T>(a, c), u[i], s);
        dw[c] = fmaf(d[i], u[i], dw[c]);
      }
    }
    if (a.y == nullptr && a.dx == nullptr) continue;
    s = warp_sum(s);
    if constexpr (!WARP) {
      float *at = box[turn++ & 1];
      if (lane == 0) at[warp] = s;
      __syncthreads();
      s = warp_sum(lane < warps ? at[lane] : 0.f);
    }
    const float m = s * inv;
    for (int c0 = warp * 256; c0 < width; c0 += warps * 256) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = c0 + i * 32 + lane;
        f[i] = 0.f;
        if (c < width) {
          f[i] = fmaf(to_float(h[c]) * r, -m, to_float(dy[c]) * weight_at<T>(a, c)) * r;
          if (dt) f[i] += to_float(dt[c]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = c0 + i * 32 + lane;
        if (a.y && c < width) static_cast<T *>(a.y)[row * a.ys + c] = from_float<T>(f[i]);
      }
      if (!drop || a.dx == nullptr) continue;
      const uint64_t e0 = (uint64_t)(row * width + c0);
      const int at = (int)(e0 & 7);
      const uint32_t bits = dropped.group((e0 >> 3) + lane), last = dropped.group((e0 >> 3) + 32);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = c0 + i * 32 + lane, e = at + i * 32 + lane;
        uint32_t b = __shfl_sync(0xffffffffu, bits, (e >> 3) & 31);
        if (e >= 256) b = last;
        if (c < width) static_cast<T *>(a.dx)[row * a.dxs + c] = from_float<T>(Dropped::at(b, e & 7) ? 0.f : f[i] * dropped.factor);
      }
    }
  }
  if (a.part == nullptr) return;
  __syncthreads();
  float *mine = a.part + (int64_t)blockIdx.x * width;
  for (int c = threadIdx.x; c < width; c += blockDim.x) {
    float v = sums[c];
    for (int k = 1; k < kTeams; ++k) v += sums[k * width + c];
    mine[c] = v;
  }
}

// The blocks' sums, added in a fixed order: 32 columns a block, 32 lanes of parts.
constexpr int kSumRows = 32;
template <class P>
__global__ void __launch_bounds__(32 * kSumRows) k_rms_weight(const float *part, int parts, int width, P *dweight) {
  __shared__ float box[kSumRows][33];
  ptx::griddep_wait();  // brought up while the kernel before it ends, which still writes `part`
  const int lane = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < width)
#pragma unroll 4
    for (int i = ty; i < parts; i += kSumRows) s += __ldcg(part + (int64_t)i * width + c);
  box[ty][lane] = s;
  __syncthreads();
  if (ty == 0 && c < width) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kSumRows; ++i) s += box[i][lane];
    dweight[c] = from_float<P>(s);
  }
}

// Blocks of the backward pass at most: the workspace holds a part of each.
inline int rms_parts(int64_t rows) { return (int)(rows < 2 * kSms ? rows : 2 * kSms); }

// Shared memory of a thread: its slots and a place for rstd.
template <class T>
size_t rms_thread_bytes(const RmsArgs &a, int columns) {
  return (size_t)kStages * ((a.dtotal ? 3 : 2) * columns * sizeof(T) + 4);
}

template <class T, int C, int LANES, bool DROP>
cudaError_t launch_ring(RmsArgs &a, const RmsShape &s, cudaStream_t st) {
  const size_t thread = rms_thread_bytes<T>(a, C);
  const RmsGrid grid = rms_grid<T>(a.dm.rows, s, thread);
  const auto kernel = k_rms_backward_ring<T, C, LANES, DROP>;
  static std::atomic<bool> allowed[64];
  const cudaError_t e = allow_smem(kernel, allowed);
  if (e != cudaSuccess) return e;
  a.parts = (int)(grid.blocks < a.dm.rows ? grid.blocks : a.dm.rows);
  const int block = grid.groups * s.threads;
  kernel<<<(unsigned)grid.blocks, block, block * thread, st>>>(a, s.threads);
  return cudaGetLastError();
}
template <class T, bool DROP>
cudaError_t launch_ring_shape(RmsArgs &a, const RmsShape &s, cudaStream_t st) {
  if (s.lanes == 8) return s.columns == 16 ? launch_ring<T, 16, 8, DROP>(a, s, st) : launch_ring<T, 32, 8, DROP>(a, s, st);
  if (s.lanes == 16) return launch_ring<T, 32, 16, DROP>(a, s, st);
  if (s.lanes == 32) return s.columns == 24 ? launch_ring<T, 24, 32, DROP>(a, s, st) : launch_ring<T, 32, 32, DROP>(a, s, st);
  return launch_ring<T, 32, 0, DROP>(a, s, st);
}
template <class T>
cudaError_t launch_any(RmsArgs &a, bool drop, cudaStream_t st) {
  const bool warp = a.dm.width <= kAnyWidth;
  const int per = warp ? kAnyWarps : 1;
  const size_t smem = (size_t)per * a.dm.width * sizeof(float);
  const auto kernel = warp ? k_rms_backward_any<T, true> : k_rms_backward_any<T, false>;
  static std::atomic<bool> allowed[2][64];
  const cudaError_t e = allow_smem(kernel, allowed[warp]);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (a.dm.rows + per - 1) / per;
  a.parts = (int)(blocks < rms_parts(a.dm.rows) ? blocks : rms_parts(a.dm.rows));
  kernel<<<(unsigned)a.parts, warp ? 32 * kAnyWarps : kAnyThreads, smem, st>>>(a, drop);
  return cudaGetLastError();
}

template <class T>
cudaError_t launch_rms_typed(RmsArgs &a, bool drop, cudaStream_t st) {
  constexpr int e = sizeof(T), N = 16 / e;
  const int64_t rows = a.dm.rows;
  const RmsShape s = rms_shape(a.dm.width, e, rows_aligned16(a.total, a.ts, rows, e) && a.dm.width % N == 0, 8);
  auto alike = [&](const void *p, int64_t stride) { return rows_alike(p, stride, a.total, a.ts, rows, e); };
  if (!alike(a.dy, a.dys) || !alike(a.dtotal, a.dts) || !alike(a.y, a.ys) || !alike(a.dx, a.dxs) ||
      s.threads > rms_threads<T>() || rms_thread_bytes<T>(a, s.columns) * s.threads > kMostSmem)
    return launch_any<T>(a, drop, st);
  return drop ? launch_ring_shape<T, true>(a, s, st) : launch_ring_shape<T, false>(a, s, st);
}

cudaError_t launch_rms(RmsArgs &a, bool drop, cudaStream_t st) {
  switch (a.dm.dtype) {
    case RVQ_DTYPE_F32: return launch_rms_typed<float>(a, drop, st);
    case RVQ_DTYPE_BF16: return launch_rms_typed<__nv_bfloat16>(a, drop, st);
    default: return launch_rms_typed<__half>(a, drop, st);
  }
}

template <class P>
cudaError_t launch_weight(const RmsArgs &a, void *dweight, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.dm.width + 31) / 32);
  cfg.blockDim = dim3(32 * kSumRows);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_rms_weight<P>, (const float *)a.part, a.parts, (int)a.dm.width,
                            static_cast<P *>(dweight));
}

}  // namespace
}  // namespace rvq

extern "C" {

RVQ_API size_t rvq_rms_norm_workspace_bytes(int64_t rows, int32_t width) {
  if (rows < 0 || width <= 0 || width > rvq::kNormMaxWidth) return 0;
  return rvq::align_up(((size_t)rvq::rms_parts(rows) + (rows == 0)) * (size_t)width * sizeof(float));
}

RVQ_API rvq_status rvq_rms_norm_backward(rvq_norm_dims dims, const void *dy, int64_t dy_stride, const void *dtotal,
                                         int64_t dtotal_stride, const void *total, int64_t total_stride,
                                         const rvq_dropout_mask *mask, const void *weight, const float *rstd,
                                         void *dresidual, int64_t dresidual_stride, void *dx, int64_t dx_stride,
                                         void *dweight, void *workspace, size_t workspace_bytes, rvq_stream_t stream) {
  using namespace rvq;
  const rvq_status s = check_rms(dims);
  if (s != RVQ_OK) return s;
  RmsArgs a{};
  a.dm = dims, a.dy = dy, a.dys = dy_stride, a.dtotal = dtotal, a.dts = dtotal_stride;
  a.total = const_cast<void *>(total), a.ts = total_stride, a.weight = weight, a.rstd = const_cast<float *>(rstd);
  a.y = dresidual, a.ys = dresidual_stride, a.dx = dx, a.dxs = dx_stride;
  if (mask && !dropout_mask(*mask, a.mask)) return RVQ_ERR_INVALID_ARG;
  if (dx && !mask) return RVQ_ERR_INVALID_ARG;  // it is dresidual
  const int e = dtype_bytes(dims.dtype), pe = dtype_bytes(dims.param_dtype);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!aligned_to(weight, pe) || !aligned_to(dweight, pe)) return RVQ_ERR_INVALID_ARG;
  const int64_t rows = dims.rows;
  if (rows == 0) {
    if (dweight && cudaMemsetAsync(dweight, 0, (size_t)dims.width * pe, st) != cudaSuccess) return RVQ_ERR_CUDA;
    return RVQ_OK;
  }
  auto ok = [&](const void *p, int64_t stride) { return aligned_to(p, e) && (stride >= dims.width || rows <= 1); };
  if (!dy || !total || !ok(dy, dy_stride) || !ok(total, total_stride) || (dtotal && !ok(dtotal, dtotal_stride)) ||
      (dresidual && !ok(dresidual, dresidual_stride)) || (dx && !ok(dx, dx_stride)))
    return RVQ_ERR_INVALID_ARG;
  if (!rstd || !aligned_to(rstd, 4)) return RVQ_ERR_INVALID_ARG;
  const size_t need = rvq_rms_norm_workspace_bytes(rows, dims.width);
  if (dweight && (!workspace || !aligned_to(workspace, 16) || workspace_bytes < need)) return RVQ_ERR_INVALID_ARG;
  const Touched written[] = {rows_at(dresidual, dresidual_stride, dims), rows_at(dx, dx_stride, dims),
                             bytes_at(dweight, (int64_t)dims.width * pe),
                             bytes_at(dweight ? workspace : nullptr, (int64_t)need)};
  const Touched read[] = {rows_at(dy, dy_stride, dims), rows_at(total, total_stride, dims),
                          rows_at(dtotal, dtotal_stride, dims), bytes_at(weight, (int64_t)dims.width * pe),
                          bytes_at(rstd, rows * 4), bytes_at(mask ? mask->step : nullptr, 8)};
  if (!rms_apart(written, read)) return RVQ_ERR_INVALID_ARG;
  if (!dresidual && !dx && !dweight) return RVQ_OK;
  a.part = dweight ? static_cast<float *>(workspace) : nullptr;
  if (launch_rms(a, mask != nullptr, st) != cudaSuccess) return RVQ_ERR_CUDA;
  if (!dweight) return RVQ_OK;
  const cudaError_t err = dims.param_dtype == RVQ_DTYPE_F32    ? launch_weight<float>(a, dweight, st)
                          : dims.param_dtype == RVQ_DTYPE_BF16 ? launch_weight<__nv_bfloat16>(a, dweight, st)
                                                               : launch_weight<__half>(a, dweight, st);
  return err == cudaSuccess ? RVQ_OK : RVQ_ERR_CUDA;
}

}  // extern "C"
