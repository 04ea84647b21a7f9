// Attention of a request's new tokens over its pages: the slice kernel and the
// merge of cut tiles.
//
// For a query row at position i of a request with kv cached keys:
//   S_j = scale q . k_j over the visible keys (j < kv; causal: j <= i; window
//   W: i - j < W), L = log sum_j exp S_j, O = sum_j exp(S_j - L) v_j, and O = 0,
//   L = -inf for a row that sees none.  One pass over the keys with a running
//   maximum and sum per row.  The sum is 0 for a row that sees nothing and NaN
//   where a score is NaN or +inf (the maximum passes over NaN): both states keep
//   that through every join.
//
// What bounds it: a single token per request reads 4 d bytes (bf16) of K and V
// per key and kv-head and does 8 d G flops on them, so HBM is the bound; the
// kernel's job is to keep enough loads in flight on every SM.  Warps have parts:
//   producers walk the block's share, up to four pieces ahead, and load it, one
//             K (and Q by 16-byte copies), one V: by TMA, a box per page and 128
//             bytes of the head, into a ring of stages of 32 KB (of
//             128 keys at head_dim 64).  A box costs its issuer about 55 ns whatever it
//             holds, 2 KB at pages of 16: two issuers share them;
//   workers   take the stages in turn (bf16: four or eight of them each, float32: one or two); a worker has its own
//             slice of a stage's keys and its own running maximum, sum and O, so
//             no barrier stands between them; at the end of a piece it leaves its state
//             in shared memory and goes on with the next one;
//   joiners   join the workers' states of a piece and write it out meanwhile.
// Pages that no row sees are loaded from outside the map: zeros, without
// touching memory.  Keys outside a tile's range that share a page with others
// are masked out of S, and their V is masked to zero before the second product (0 times
// what the rest of a page holds need not be 0).
//
// bf16: mma.sync m16n8k16, rows of the tile on M (16 or 32, G query heads of a
//   kv-head packed), so K and V are read once for all of them; P is rounded
//   to bf16 for the second product (relative 2^-8, the inputs' own
//   precision), its row sum is taken in float32 before that.  The legacy
//   tensor path is chosen here because these tiles have too few rows to be
//   bound by it.
// float32: FFMA throughout, for the arithmetic's sake.
#include "slice.cuh"

namespace cpattn {

int paged_slice_grid() { return num_sms(); }

cp_status launch_paged_slice(const PagedArgs& a, PagedKernel k, bool after_pair, cudaStream_t s) {
  if (a.dtype == CP_BF16) {
    if (k == kPagedSlice16)
      return a.d == 128 ? few::run_slice<few::SliceBf16<128, 16>, 128, 16>(a, after_pair, s)
                        : few::run_slice<few::SliceBf16<64, 16>, 64, 16>(a, after_pair, s);
    if (k == kPagedSlice32)
      return a.d == 128 ? few::run_slice<few::SliceBf16<128, 32>, 128, 32>(a, after_pair, s)
                        : few::run_slice<few::SliceBf16<64, 32>, 64, 32>(a, after_pair, s);
    return CP_ERR_UNSUPPORTED;
  }
  if (k == kPagedSlice4)
    return a.d == 128 ? few::run_slice<few::SliceF32<128, 4>, 128, 4>(a, after_pair, s)
                      : few::run_slice<few::SliceF32<64, 4>, 64, 4>(a, after_pair, s);
  if (k == kPagedSlice16)
    return a.d == 128 ? few::run_slice<few::SliceF32<128, 16>, 128, 16>(a, after_pair, s)
                      : few::run_slice<few::SliceF32<64, 16>, 64, 16>(a, after_pair, s);
  return CP_ERR_UNSUPPORTED;
}

cp_status launch_paged_merge(const PagedArgs& pair, const PagedArgs& slice, cudaStream_t s) {
  const PagedArgs& a = pair.grid > 0 ? pair : slice;
  if (pair.grid > 0 && a.dtype != CP_BF16) return CP_ERR_UNSUPPORTED;
  if (a.dtype == CP_BF16)
    return a.d == 128 ? few::run_merge<__nv_bfloat16, 128>(pair, slice, s) : few::run_merge<__nv_bfloat16, 64>(pair, slice, s);
  return a.d == 128 ? few::run_merge<float, 128>(pair, slice, s) : few::run_merge<float, 64>(pair, slice, s);
}

}  // namespace cpattn
