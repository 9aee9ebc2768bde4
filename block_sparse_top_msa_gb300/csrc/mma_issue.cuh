// What the attention kernels that issue their products by whole warps share: the
// order of a segment's tiles, MMAs and commits by an elected lane, rings, and
// row maxima that keep NaN.
#pragma once

#include "common.cuh"

namespace msa {

// Tile x of the 2 n tiles of a segment, in the order the products want them:
// K0, K1, V0, K2, V1, ... V(n-1). Returns the block, and whether it is V.
MSA_DEV int tile_order(int x, int n, bool& is_v) {
  if (x == 0) {
    is_v = false;
    return 0;
  }
  const int i = x >> 1;
  if (x & 1) {
    is_v = i + 1 >= n;
    return is_v ? n - 1 : i + 1;
  }
  is_v = true;
  return i - 1;
}

// MMAs and commits issued by the one lane whose `el` is not 0. Descriptors as
// low word and high word.
MSA_DEV uint32_t elect_one() {
  uint32_t el;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(el));
  return el;
}
MSA_DEV void mma_ss_if(uint32_t el, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 q, %0, 0;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%2, %4};\n\tmov.b64 b, {%3, %4};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%1], a, b, %5, p;\n\t}" ::"r"(el),
      "r"(d), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
MSA_DEV void mma_ts_if(uint32_t el, uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\tsetp.ne.b32 q, %0, 0;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 b, {%3, %4};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], b, %5, p;\n\t}" ::"r"(el),
      "r"(d), "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
MSA_DEV void commit_if(uint32_t el, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %0, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n\t}" ::"r"(el),
      "r"(smem_u32(bar))
      : "memory");
}

// Slot and phase of a position in a ring of N slots.
template <int N>
struct Ring {
  int idx = 0;
  uint32_t phase = 0;
  MSA_DEV void next() {
    if (++idx == N) {
      idx = 0;
      phase ^= 1u;
    }
  }
};
// The largest of three, NaN if one is: a NaN among keys that are masked
// otherwise has to show.
MSA_DEV float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <int N>
MSA_DEV float row_max(const float* v) {
  float m0 = v[0], m1 = v[1], m2 = v[2], m3 = v[3];
#pragma unroll
  for (int c = 4; c + 8 <= N; c += 8) {
    m0 = max3_nan(m0, v[c], v[c + 1]);
    m1 = max3_nan(m1, v[c + 2], v[c + 3]);
    m2 = max3_nan(m2, v[c + 4], v[c + 5]);
    m3 = max3_nan(m3, v[c + 6], v[c + 7]);
  }
  m0 = max3_nan(m0, v[N - 4], v[N - 3]);
  m1 = max3_nan(m1, v[N - 2], v[N - 1]);
  return max3_nan(max3_nan(m0, m1, m2), m3, m3);
}

}  // namespace msa
