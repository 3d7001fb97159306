// The dropout mask (rvq_dropout_mask): a function of an element's index, the
// seed and the call, computed where it is needed and never stored.
//
// Eight elements share one call of Philox4x32 with ten rounds (Salmon, Moraes,
// Dror, Shaw: Parallel random numbers: as easy as 1, 2, 3; 2011): counter
// (e / 8, offset + 2^32 * step), key seed; 16 of its 128 bits each.  An element
// is dropped where its 16 bits are below round(p * 2^16), so that the factor
// 2^16 / (2^16 - that) is exact to the probability that is used.  16 bits and not
// 32: ten rounds are 20 wide products, and at 8 elements a call that is 2.5 an
// element.
#pragma once

#include "rvq_rows.cuh"

namespace rvq {

struct DropoutMask {
  uint64_t seed, offset;
  const int64_t *step;  // null: 0
  uint32_t drop;        // of 2^16
  float factor;         // of what stays (0 where nothing does)
};

// What a call's mask becomes; false: not valid.
inline bool dropout_mask(const rvq_dropout_mask &m, DropoutMask &out) {
  if (!(m.p >= 0.f && m.p <= 1.f) || !aligned_to(m.step, 8)) return false;
  const uint32_t drop = (uint32_t)((double)m.p * 65536.0 + 0.5);
  out = {m.seed, m.offset, m.step, drop, drop < 65536 ? (float)(65536.0 / (65536 - drop)) : 0.f};
  return true;
}

// The mask of one launch, its call's counter read.  What is dropped of 8 elements
// comes as one bit each, the even ones' in the lower half of a word and the odd
// ones' in the upper: a pair is compared at once, by 16-bit maxima.
struct Dropped {
  uint32_t k0, k1, u0, u1, limit, all;
  float factor;
  __device__ __forceinline__ explicit Dropped(const DropoutMask &m)
      : k0((uint32_t)m.seed), k1((uint32_t)(m.seed >> 32)), limit((m.drop & 0xffffu) * 0x10001u),
        all(m.drop > 0xffffu ? 0x000f000fu : 0u), factor(m.factor) {
    const uint64_t upper = m.offset + (m.step ? (uint64_t)*m.step << 32 : 0);
    u0 = (uint32_t)upper, u1 = (uint32_t)(upper >> 32);
  }
  static __device__ __forceinline__ uint32_t below(uint32_t w, uint32_t limit) {  // of each half: 1 where w < limit
    uint32_t m, d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(m) : "r"(w), "r"(limit));
    asm("min.u16x2 %0, %1, %2;" : "=r"(d) : "r"(m ^ w), "r"(0x00010001u));
    return d;
  }
  // Of group g: bit i: element 2 i, bit 16 + i: element 2 i + 1 (i < 4).
  __device__ __forceinline__ uint32_t group(uint64_t g) const {
    uint32_t a = (uint32_t)g, b = (uint32_t)(g >> 32), c = u0, d = u1, x = k0, y = k1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const uint64_t p = (uint64_t)a * 0xD2511F53u, q = (uint64_t)c * 0xCD9E8D57u;
      a = (uint32_t)(q >> 32) ^ b ^ x, b = (uint32_t)q;
      c = (uint32_t)(p >> 32) ^ d ^ y, d = (uint32_t)p;
      x += 0x9E3779B9u, y += 0xBB67AE85u;
    }
    return below(a, limit) + below(b, limit) * 2 + below(c, limit) * 4 + below(d, limit) * 8 | all;
  }
  // Whether element i of the 8 that `bits` is of is dropped.
  static __device__ __forceinline__ bool at(uint32_t bits, int i) { return bits >> (i / 2 + (i & 1) * 16) & 1; }
  __device__ __forceinline__ bool element(uint64_t e) const { return at(group(e >> 3), (int)(e & 7)); }
  // In the same form, elements e to e + N - 1 (N 4 or 8): one group, or two where they do not start at one (the norm
  // with dropout, both passes: 60 000 x 1024 bf16 188 us, bytes alone 163; 58 536 x 1025, rows 1031 apart, 283 and 159).
  template <int N>
  __device__ __forceinline__ uint32_t from(uint64_t e) const {
    const int i = (int)(e & 7);
    uint32_t w = group(e >> 3);
    if (i + N > 8) w |= group((e >> 3) + 1) << 4;
    if (i & 1) w = w >> 16 | (w & 0xffffu) >> 1 << 16;  // the odd ones become the even ones
    return w >> (i / 2) & (N == 8 ? 0x000f000fu : 0x00030003u);
  }
};

}  // namespace rvq
