// Steps that the kernels on SM pairs (cta_group::2, 128 query rows per CTA,
// key tiles of 128) share: operand descriptors and the softmax of a key tile.
#pragma once

#include "internal.h"
#include "tc_util.cuh"

namespace cpattn {

constexpr int kKHalfBytes = 64 * 64 * 2;  // one 64-column box of a CTA's 64 keys

// Descriptor of K-step kk (16 bf16 along the head dimension) of this CTA's
// 64-key half of a key tile: two 128-byte-swizzled 64-column boxes of 8 KB.
__device__ __forceinline__ uint64_t khalf_step(uint64_t base_desc, int kk) {
  return base_desc + uint64_t((((kk >> 2) * kKHalfBytes) + (kk & 3) * 32) >> 4);
}

// Maximum of the raw scores of a row (keys lo <= j < lo + span when
// kMasked, span >= 0), over four independent chains.
template <bool kMasked>
__device__ __forceinline__ float row_max(const uint32_t* sr, int lo, uint32_t span) {
  float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int j = 0; j < kTile; j += 2) {
    float s0 = __uint_as_float(sr[j]), s1 = __uint_as_float(sr[j + 1]);
    if (kMasked) {
      s0 = uint32_t(j - lo) < span ? s0 : -INFINITY;
      s1 = uint32_t(j + 1 - lo) < span ? s1 : -INFINITY;
    }
    m4[(j >> 1) & 3] = tc::fmax3(m4[(j >> 1) & 3], s0, s1);
  }
  return tc::fmax3(fmaxf(m4[0], m4[1]), m4[2], m4[3]);
}

// P = exp2(s * scale_log2 - mu) over the 128 scores of a row: bf16 pairs are
// written over the row's S columns (keys 2c, 2c+1 -> column c) and the row
// sum of the fp32 values is returned.  kMasked keeps keys lo <= j < lo + span.
template <bool kMasked>
__device__ __forceinline__ float p_pass(const uint32_t* sr, int lo, uint32_t span, float mu, uint64_t sl2x2,
                                        uint32_t tS) {
  const uint64_t nmu = tc::f32x2(-mu, -mu);
  uint64_t ls[4] = {tc::f32x2(0.f, 0.f), tc::f32x2(0.f, 0.f), tc::f32x2(0.f, 0.f), tc::f32x2(0.f, 0.f)};
#pragma unroll
  for (int cc = 0; cc < 4; ++cc) {
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int j0 = cc * 32 + 2 * e;
      float x0, x1;
      tc::f32x2_split(tc::ffma2(tc::f32x2(__uint_as_float(sr[j0]), __uint_as_float(sr[j0 + 1])), sl2x2, nmu), x0,
                      x1);
      if (kMasked) {
        x0 = uint32_t(j0 - lo) < span ? x0 : -INFINITY;
        x1 = uint32_t(j0 + 1 - lo) < span ? x1 : -INFINITY;
      }
      const float p0 = tc::ex2(x0), p1 = tc::ex2(x1);
      ls[e & 3] = tc::fadd2(ls[e & 3], tc::f32x2(p0, p1));
      pk[e] = tc::pack_bf16x2(p0, p1);
    }
    tc::tmem_st16(tS + cc * 16, pk);
  }
  float x, y;
  tc::f32x2_split(tc::fadd2(tc::fadd2(ls[0], ls[1]), tc::fadd2(ls[2], ls[3])), x, y);
  return x + y;
}

}  // namespace cpattn
