// The best entries of a row, in order, by a warp (rvq_beam.cu, rvq_log_probs.cu).
#pragma once

#include "rvq_rows.cuh"

namespace rvq {

constexpr int kMostKept = 64;  // entries that a row keeps at most
constexpr int kRoom = 128;     // entries that a warp puts in order at once, beside those it holds

// An entry's place in the order: the larger value (of raw values: value + score,
// rounded) first, then the lower code.  0 is no entry (NaN and -inf have none).
__device__ __forceinline__ uint32_t order_of(float v) {
  if (!(v > -CUDART_INF_F)) return 0;
  const uint32_t b = __float_as_uint(v + 0.f);  // -0 becomes 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float v, int code) {
  const uint32_t o = order_of(v);
  return o ? (uint64_t)o << 32 | (uint32_t)~code : 0;
}

// A warp's shared memory: the entries to be put in order, and the best so far.
struct WarpRoom {
  uint64_t room[kRoom + kMostKept], best[kMostKept];
  int count;
};

// The n-th largest of the lanes' values (n <= 32): for few by taking the
// largest away, else by sorting (15 exchanges).
__device__ __forceinline__ uint32_t warp_nth(uint32_t v, int n) {
  const int lane = threadIdx.x & 31;
  if (n <= 8) {
    uint32_t top = 0;
    for (int i = 0; i < n; ++i) {
      top = __reduce_max_sync(0xffffffffu, v);
      const unsigned at = __ballot_sync(0xffffffffu, v == top);
      if (lane == __ffs(at) - 1) v = 0;
    }
    return top;
  }
#pragma unroll
  for (int k = 2; k <= 32; k *= 2)
#pragma unroll
    for (int j = k / 2; j; j /= 2) {
      const uint32_t o = __shfl_xor_sync(0xffffffffu, v, j);
      const bool high = ((lane & k) == 0) == ((lane & j) == 0);
      v = high ? max(v, o) : min(v, o);
    }
  return __shfl_sync(0xffffffffu, v, n - 1);
}

// The pieces `first`, `first` + `step`, ... of a row, NV vectors a lane each:
// the best n entries in order in r.best (0: none).  `sum(z, edge, high)` is
// given each piece before its entries are looked for: the vectors (-inf where
// there are none), the lane's element beside them and the largest of the lane's
// elements.  `add` is added to every value first.  PARTS: the parts of a lane's
// elements whose largest values may make the bar, 2, or 4 where more than 32 are
// kept: two live values more, which cost the beam step's block for a group its
// last registers (12000 groups of 4 rows of 1024 floats, 4 kept: 51.3 us against
// 48.8 with two; 2000 of 12 rows of 1025 bf16, 24 kept: 88.7 against 74.7), and
// which pay where many are kept (500 of 64 rows of 1024 floats, 64 kept: 5.35 ms
// against 7.06).
template <class T, int NV, int PARTS, class Sum>
__device__ __forceinline__ void warp_pieces(const CutRow<T> &in, int first, int step, int n, float add, WarpRoom &r,
                                            Sum sum) {
  constexpr int N = 16 / (int)sizeof(T);
  const int lane = threadIdx.x & 31;
  for (int i = lane; i < kMostKept; i += 32) r.best[i] = 0;
  if (lane == 0) r.count = 0;
  __syncwarp();
  bool held = false;
  for (int p = first; p == 0 || p * NV * 32 < in.full; p += step) {
    uint4 z[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = (p * NV + j) * 32 + lane;
      z[j] = v < in.full ? in.vector(v) : all_low<T>();
    }
    const int edge_at = p == 0 ? in.edge(lane) : -1;
    const float edge = edge_at >= 0 ? to_float(in.z[edge_at]) + add : -CUDART_INF_F;
    // each vector's largest, and the largest of each part of the lane's elements (z + add: add is 0 where the sum is
    // wanted).  Once the sum is taken the vectors are done with: the few that hold an entry worth ordering are
    // read again, by their lanes at the same time.
    float most[NV], part[PARTS];
#pragma unroll
    for (int i = 0; i < PARTS; ++i) part[i] = -CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      most[j] = largest_of<T>(z[j]) + add;
      part[j * PARTS / NV] = fmaxf(part[j * PARTS / NV], most[j]);
    }
    part[0] = fmaxf(part[0], edge);
    float half[2];
    if constexpr (PARTS == 4)
      half[0] = fmaxf(part[0], part[1]), half[1] = fmaxf(part[2], part[3]);
    else
      half[0] = part[0], half[1] = part[1];
    const float high = fmaxf(half[0], half[1]);
    sum(z, edge, high);
    const uint64_t last = held ? r.best[n - 1] : 0;  // an entry counts if it is above this
    const uint32_t last_value = (uint32_t)(last >> 32);
    if (!__any_sync(0xffffffffu, order_of(high) > 0 && order_of(high) >= last_value)) continue;
    // n entries reach the bar: the n-th of the lanes' largest, or, for more, half as far down among the largest of
    // their halves, or a quarter among those of their quarters.  (The 32nd of 32 is a low one: it let through more
    // than there is room for, and 6 rows of 65536 f16 with 32 kept took 338 us against 18.  Two searches cost more than
    // a low bar up to 18: 2000 groups of 12 rows of 1025 bf16, 17 kept: 56.5 us against 58.5.)
    uint32_t bar;
    if (n <= 18) {
      bar = warp_nth(order_of(high), n);
    } else if (PARTS == 2 || n <= 32) {
      const int at = (n + 1) / 2;
      bar = min(warp_nth(order_of(half[0]), at), warp_nth(order_of(half[1]), at));
    } else {
      bar = 0xffffffffu;
#pragma unroll
      for (int i = 0; i < PARTS; ++i) bar = min(bar, warp_nth(order_of(part[i]), (n + PARTS - 1) / PARTS));
    }
    bar = max(bar, last_value);
    const float line = bar ? value_of(bar) : -3.402823466e38f;
    auto offer = [&](float v, int code) {
      const uint64_t k = key_of(v, code);
      if (k <= last) return;
      const int at = atomicAdd(&r.count, 1);
      if (at < kRoom) r.room[at] = k;
    };
    uint32_t wanted = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) wanted |= (uint32_t)(most[j] >= line) << j;
    if (edge >= line) offer(edge, edge_at);
    while (wanted) {
      const int v = (p * NV + __ffs(wanted) - 1) * 32 + lane;
      wanted &= wanted - 1;
      float f[N];
      unpack16<T>(in.vector(v), f);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (f[i] + add >= line) offer(f[i] + add, in.head + v * N + i);
    }
    __syncwarp();
    if (r.count > kRoom) {
      // many equal values at the bar: the best n one after the other
      __syncwarp();
      uint64_t below = ~0ull;
      for (int c = 0; c < n; ++c) {
        uint64_t k = key_of(edge, edge_at);
        if (k >= below) k = 0;
        for (int j = 0; j < NV; ++j) {
          const int v = (p * NV + j) * 32 + lane;
          if (v >= in.full) break;
          float f[N];
          unpack16<T>(in.vector(v), f);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const uint64_t e = key_of(f[i] + add, in.head + v * N + i);
            if (e < below && e > k) k = e;
          }
        }
        const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
        const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
        below = (uint64_t)hi << 32 | lo;
        if (lane == 0 && c == 0) r.count = 0;
        if (below <= last) break;
        if (lane == 0) r.room[c] = below, r.count = c + 1;
      }
    }
    __syncwarp();
    // every entry's place among the new ones and those held
    const int fresh = r.count;
    if (fresh) {
      const int all = held ? fresh + n : fresh;
      if (held)
        for (int i = lane; i < n; i += 32) r.room[fresh + i] = r.best[i];
      __syncwarp();
      for (int i = lane; i < all; i += 32) {
        const uint64_t k = r.room[i];
        int place = 0;
        for (int j = 0; j < all; ++j) place += r.room[j] > k;
        if (k && place < n) r.best[place] = k;
      }
      held = true;
      if (lane == 0) r.count = 0;
      __syncwarp();
    }
  }
}

}  // namespace rvq
