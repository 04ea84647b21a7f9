// Attention of packed query sequences over packed key sequences of other
// lengths (cp_cross_attn_fwd, cp_cross_attn_bwd): arguments and launchers.
//
// A sequence is what paged.h calls a request, its keys rows of a packed tensor
// instead of pages; the forward's work is divided as there.  The position of query i
// of a sequence of nq queries and nk keys is i + nk - nq: the ends are aligned.
#pragma once

#include "paged.h"

namespace cpattn {

// The bias of relative position x = key position - query position of head h, in log2 units (times
// log2 e), is rel[h * rel_stride + rel_zero + x] for |x| <= reach + kRelPad; it
// is the same for all x <= -reach, and for all x >= reach.
constexpr int kRelPad = 256;  // a tile of 128 rows and 128 keys that touches the part that varies

struct CrossArgs : PagedArgs {
  static constexpr bool kDense = true;
  const int32_t* cu_k;   // [n_reqs + 1]
  const int32_t* len_q;  // [n_reqs] or null
  const int32_t* len_k;
  int64_t k_stride, v_stride, rows_k;
  const float* rel;  // null: no bias
  int32_t rel_stride, rel_zero, reach;
  void* rest;  // bf16: what o lost, [rows][H][d]: with a bias to both roundings (P's and its own), else to its own; null: not asked for
  const uint64_t* rng;  // {seed, offset}; null: no dropout
  uint32_t drop_min;    // pieces below it drop their probability
  float drop_scale;     // 1 / (1 - drop_min / 2^15)
};
template <bool B, bool D>
struct CrossArgsOf : CrossArgs {
  static constexpr bool kBias = B, kDrop = D;
};

CPATTN_HD int32_t paged_key_row(const CrossArgs& a, int r) { return clamp_i32(a.cu_k[r], 0, int32_t(a.rows_k)); }

CPATTN_HD PagedReq paged_req(const CrossArgs& a, int r) {
  PagedReq q;
  q.q0 = clamp_i32(a.cu[r], 0, int32_t(a.rows));
  q.nq = clamp_i32(a.cu[r + 1], q.q0, int32_t(a.rows)) - q.q0;
  if (a.len_q) q.nq = clamp_i32(a.len_q[r], 0, q.nq);
  const int32_t k0 = paged_key_row(a, r);
  q.kv = clamp_i32(a.cu_k[r + 1], k0, int32_t(a.rows_k)) - k0;
  if (a.len_k) q.kv = clamp_i32(a.len_k[r], 0, q.kv);
  return q;
}

#ifdef __CUDACC__
__device__ __forceinline__ float rel_bias(const CrossArgs& a, int head, int x) {
  if (!a.rel) return 0.f;  // float32 with dropout is built once, with a bias
  return a.rel[int64_t(head) * a.rel_stride + a.rel_zero + min(max(x, -a.reach), a.reach)];
}
#endif

// First distances of the buckets of one direction, ascending: a distance is in
// the last bucket that starts at or before it.
constexpr int kMaxBuckets = 64;
struct RelStarts {
  int32_t per;   // buckets of a direction
  int32_t both;  // keys behind the query have buckets of their own, from `per` on
  int32_t start[kMaxBuckets];
};

// Spreads the table [buckets][heads] over the relative positions.
struct RelSpread {
  const void* table;
  float* rel;
  int32_t heads, rel_stride, rel_zero;
  RelStarts starts;
};
cp_status launch_rel_spread(const RelSpread& a, cp_dtype dtype, cudaStream_t s);

// early: the launch before on the stream is launch_rel_spread, which it may overlap.
cp_status launch_cross_few(const CrossArgs& a, PagedKernel k, bool early, cudaStream_t s);
cp_status launch_cross_few_f32(const CrossArgs& a, PagedKernel k, bool early, cudaStream_t s);
cp_status launch_cross_pair(const CrossArgs& a, bool early, cudaStream_t s);
cp_status cross_pair_grid(const CrossArgs& a, int32_t* pairs);
// Joins the cut tiles of the launch before.
cp_status launch_cross_merge(const CrossArgs& a, bool pair, cudaStream_t s);

// ---- backward ----
//
// With P_ij = exp2(s_ij - L2_i), dP_ij = dO_i . v_j, D_i = dO_i . O_i, keep and r = drop_scale:
//   dV_j = r sum_i keep P dO_i,   dS = P (r keep dP - D),
//   dQ_i = scale sum_j dS_ij k_j, dK_j = scale sum_i dS_ij q_i,   dtable[b][h] = sum of dS_ij over bucket(ij) = b.
// The kernels form dS / r = P (keep dP - D / r) and multiply by r at the end.
// One work item is a tile of keys of a sequence and one kv-head with all queries of its
// group, so dK and dV are complete in it; the tiles are listed on the device by the
// preparation, those with the most query tiles first (and, in float32, tiles of queries
// for dQ likewise).
struct CrossTile {
  int32_t seq, first;  // sequence, first row (counted in it)
  int32_t id;          // place in the order of the sequences, which sums go by
  int32_t pad;
};
struct CrossTiles {
  CrossTile* list;
  int32_t* count;  // tiles listed
  int32_t most;    // places of the list
  int32_t size;    // rows of a tile
};
struct CrossBwd : CrossArgs {
  const void* dout;
  int64_t do_stride;
  float* delta;  // [H][rows]: D / r
  float* lse2;   // [H][rows]: lse * log2(e), +inf for a row that sees no key
  float* dq_acc;  // bf16: float32 sums [H][rows][d]
  void *dq, *dk, *dv, *dtable;
  float* part;         // partial sums of the table's gradient, [key tile][H][parts][bucket_stride]
  int32_t parts, buckets, bucket_stride;
  CrossTiles k_tiles, q_tiles;
  RelStarts starts;
  float scale;
};

// First query that sees a key of the tile from key k0 on.
CPATTN_HD int32_t cross_first_query(const CrossArgs& a, const PagedReq& q, int32_t k0) {
  return a.causal ? clamp_i32(k0 - (q.kv - q.nq), 0, q.nq) : 0;
}

// Relative positions lo .. hi (ends included) that belong to bucket b.
CPATTN_HD void rel_range(const RelStarts& s, int32_t b, int32_t* lo, int32_t* hi) {
  const int32_t far = 1 << 30;
  const bool fore = s.both && b >= s.per;
  const int32_t n = fore ? b - s.per : b;
  const int32_t first = s.start[n], last = n + 1 < s.per ? s.start[n + 1] - 1 : far;
  if (fore) {
    *lo = first > 1 ? first : 1;
    *hi = last;
  } else {
    *lo = -last;
    *hi = !s.both && n == 0 ? far : -first;
  }
}

// Tiles, D, L2, zeros where sums begin and in rows that no sequence owns.
cp_status launch_cross_bwd_prep(const CrossBwd& a, cudaStream_t s);
cp_status launch_cross_bwd(const CrossBwd& a, cudaStream_t s);      // bf16
cp_status launch_cross_bwd_f32(const CrossBwd& a, cudaStream_t s);
// dQ from its sums (bf16) and the table's gradient.
cp_status launch_cross_bwd_post(const CrossBwd& a, cudaStream_t s);

}  // namespace cpattn
