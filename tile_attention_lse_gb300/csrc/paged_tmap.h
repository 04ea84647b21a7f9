// Host helper: TMA tensor map of a paged cache.
#pragma once

#include "paged.h"
#include "tmap.h"

namespace cpattn {

// [pages][page][heads][d] with the token and head dimensions in ascending
// order of stride (head first where head_stride <= token_stride); box: 128
// bytes of one head (128-byte swizzle) of `box` tokens of one page.  Page
// number n_pages lies outside: zeros, no access.  Where a head's 128 bytes stand
// alone (bf16 of head_dim 64, heads side by side), fetching 256 bytes of memory for
// them brings in half of the next head's (64 single tokens over about 1808 keys: 73 us, 61 without).
// Returns false on failure.
inline bool make_tmap_pages(CUtensorMap* map, const void* base, const PagedArgs& a, int box) {
  auto enc = tmap_encoder();
  if (!enc) return false;
  const bool head_inner = a.head_stride <= a.token_stride;
  const cuuint64_t size = a.dtype == CP_BF16 ? 2 : 4;
  const cuuint64_t page = cuuint64_t(1) << a.page_shift, heads = cuuint64_t(a.Hkv);
  const cuuint64_t dims[4] = {cuuint64_t(a.d), head_inner ? heads : page, head_inner ? page : heads,
                              cuuint64_t(a.n_pages)};
  const cuuint64_t hs = cuuint64_t(a.head_stride) * size, ts = cuuint64_t(a.token_stride) * size;
  cuuint64_t ps = cuuint64_t(a.page_stride) * size;
  if (a.n_pages == 1 && ps == 0) ps = page * ts;
  const cuuint64_t strides[3] = {head_inner ? hs : ts, head_inner ? ts : hs, ps};
  const cuuint32_t b[4] = {cuuint32_t(128 / size), head_inner ? 1u : cuuint32_t(box),
                           head_inner ? cuuint32_t(box) : 1u, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const cuuint64_t row = cuuint64_t(a.d) * size, run = !head_inner && ts == row ? page * row : row;  // bytes of a head side by side
  return enc(map, a.dtype == CP_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4,
             const_cast<void*>(base), dims, strides, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             run < 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool make_tmap_keys(CUtensorMap* map, const PagedArgs& a, bool of_v, int box) {
  return make_tmap_pages(map, of_v ? a.v : a.k, a, box);
}

}  // namespace cpattn
