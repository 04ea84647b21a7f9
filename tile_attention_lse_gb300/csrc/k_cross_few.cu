// Cross attention of few rows in bf16 on the slice kernel, and the merge of cut
// tiles of any launch.
#include "cross_few.cuh"

namespace cpattn {

cp_status launch_cross_few(const CrossArgs& a, PagedKernel k, bool early, cudaStream_t s) {
  if (a.dtype == CP_F32) return launch_cross_few_f32(a, k, early, s);
  if (a.rng) return CP_ERR_UNSUPPORTED;  // the pair kernel's
  if (k == kPagedSlice16)
    return a.d == 128 ? run<few::SliceBf16<128, 16>, 128, 16>(a, early, s)
                      : run<few::SliceBf16<64, 16>, 64, 16>(a, early, s);
  if (k == kPagedSlice32)
    return a.d == 128 ? run<few::SliceBf16<128, 32>, 128, 32>(a, early, s)
                      : run<few::SliceBf16<64, 32>, 64, 32>(a, early, s);
  return CP_ERR_UNSUPPORTED;
}

cp_status launch_cross_merge(const CrossArgs& a, bool pair, cudaStream_t s) {
  CrossArgs none = a;
  none.grid = 0;
  const CrossArgs &p = pair ? a : none, &q = pair ? none : a;
  if (a.dtype == CP_BF16)
    return a.d == 128 ? few::run_merge<__nv_bfloat16, 128>(p, q, s) : few::run_merge<__nv_bfloat16, 64>(p, q, s);
  return a.d == 128 ? few::run_merge<float, 128>(p, q, s) : few::run_merge<float, 64>(p, q, s);
}

}  // namespace cpattn
