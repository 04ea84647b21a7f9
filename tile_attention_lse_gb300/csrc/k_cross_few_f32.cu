// Cross attention in float32 on the slice kernel.
#include "cross_few.cuh"

namespace cpattn {

cp_status launch_cross_few_f32(const CrossArgs& a, PagedKernel k, bool early, cudaStream_t s) {
  if (k == kPagedSlice4)
    return a.d == 128 ? run_f32<few::SliceF32<128, 4>, 128, 4>(a, early, s)
                      : run_f32<few::SliceF32<64, 4>, 64, 4>(a, early, s);
  if (k == kPagedSlice16)
    return a.d == 128 ? run_f32<few::SliceF32<128, 16>, 128, 16>(a, early, s)
                      : run_f32<few::SliceF32<64, 16>, 64, 16>(a, early, s);
  return CP_ERR_UNSUPPORTED;
}

}  // namespace cpattn
