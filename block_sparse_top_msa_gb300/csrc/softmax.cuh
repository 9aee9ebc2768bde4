// The online softmax of one block over a row of scores in TMEM, shared by the
// attention kernels.
#pragma once

#include <math.h>

#include "common.cuh"
#include "tmem_wide.cuh"

namespace msa {

constexpr float kRescaleLog2 = 8.0f;

MSA_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

MSA_DEV float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Max of 64 values with four independent three-input chains.
MSA_DEV float row_max64(const float* v) {
  float m0 = v[0], m1 = v[1], m2 = v[2], m3 = v[3];
#pragma unroll
  for (int c = 4; c + 8 <= 64; c += 8) {
    m0 = fmax3(m0, v[c], v[c + 1]);
    m1 = fmax3(m1, v[c + 2], v[c + 3]);
    m2 = fmax3(m2, v[c + 4], v[c + 5]);
    m3 = fmax3(m3, v[c + 6], v[c + 7]);
  }
  m0 = fmax3(m0, v[60], v[61]);
  m1 = fmax3(m1, v[62], v[63]);
  return fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
}

// Running-max update of one row for a block whose raw max logit is mx. The
// reference max only moves when the new max exceeds it by more than 2^8, so
// O is rescaled rarely; P stays <= 2^8, exact enough for bf16 and fp32 sums.
MSA_DEV void update_max(bool mem, float mx, float scale_log2, float& m_ref, float& l,
                        float& alpha, bool& rescale) {
  if (!mem) return;
  const float m_new = mx * scale_log2;
  if (m_ref == -INFINITY || m_new > m_ref + kRescaleLog2) {
    if (m_ref != -INFINITY) {
      alpha = ex2(m_ref - m_new);
      rescale = true;
      l *= alpha;
    }
    m_ref = m_new;
  }
}

// P = 2^(s * scale_log2 + neg_m) for N columns, packed to 16-bit pairs (the
// type of V) and stored to TMEM at pcol (N/2 columns); the fp32 values are
// summed into acc. P <= 2^8, well inside the f16 range.
template <int N, bool F16 = false>
MSA_DEV void exp_pack_store(const float* sv, float2 sc2, float neg_m, float2& acc, uint32_t pcol) {
  uint32_t pk[N / 2];
  const float2 nm2 = make_float2(neg_m, neg_m);
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const float2 x = __ffma2_rn(make_float2(sv[c], sv[c + 1]), sc2, nm2);
    const float p0 = ex2(x.x), p1 = ex2(x.y);
    acc = __fadd2_rn(acc, make_float2(p0, p1));
    pk[c >> 1] = pack_x2<F16>(p0, p1);
  }
  if (N == 64) tmem_st32(pcol, pk);
}

}  // namespace msa
