// The slice kernel (slice.cuh) over packed keys: tensor map and launch, for the
// translation units that build it in bf16 and in float32.
#pragma once

#include "cross.h"
#include "slice.cuh"

namespace cpattn {

// [1][rows][heads][d] of K or V: the layout of a cache of one page.
inline bool make_tmap_keys(CUtensorMap* map, const CrossArgs& a, bool of_v, int box) {
  auto enc = tmap_encoder();
  if (!enc) return false;
  const cuuint64_t size = a.dtype == CP_BF16 ? 2 : 4, stride = cuuint64_t(of_v ? a.v_stride : a.k_stride) * size;
  const cuuint64_t dims[4] = {cuuint64_t(a.d), cuuint64_t(a.Hkv), cuuint64_t(a.rows_k > 0 ? a.rows_k : 1), 1};
  const cuuint64_t strides[3] = {cuuint64_t(a.d) * size, stride, stride};
  const cuuint32_t b[4] = {cuuint32_t(128 / size), 1, cuuint32_t(box), 1}, es[4] = {1, 1, 1, 1};
  // one head's row of less than 256 bytes: see make_tmap_pages
  return enc(map, a.dtype == CP_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4,
             const_cast<void*>(of_v ? a.v : a.k), dims, strides, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B,
             a.d * size < 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool B, bool Dr>
CrossArgsOf<B, Dr> as(const CrossArgs& a) {
  CrossArgsOf<B, Dr> x;
  static_cast<CrossArgs&>(x) = a;
  return x;
}

template <typename S, int D, int R>
cp_status run(const CrossArgs& a, bool early, cudaStream_t s) {
  return a.rel ? few::run_slice<S, D, R>(as<true, false>(a), early, s)
               : few::run_slice<S, D, R>(as<false, false>(a), early, s);
}
template <typename S, int D, int R>
cp_status run_f32(const CrossArgs& a, bool early, cudaStream_t s) {
  return a.rng ? few::run_slice<S, D, R>(as<true, true>(a), early, s) : run<S, D, R>(a, early, s);
}

}  // namespace cpattn
