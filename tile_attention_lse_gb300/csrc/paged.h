// Attention over a paged K/V cache: arguments, the division of the work over
// the blocks of a launch, and the launchers.
//
// The lengths of the requests live in device memory only, so the division is
// computed on the device, by every block for itself.  The new tokens of a
// request times the G query heads of a kv-head are its packed rows (row =
// token * G + head in group: all of them read the same keys), cut into tiles
// of R rows.  A tile's visible keys are walked in units of U keys and cost n
// units plus E for its start and its end.  The units of all (request,
// kv-head, tile) triples, in that order, form one axis, and block c of N takes
// the c-th of N runs of it (T / N units, the first T % N blocks one more):
// equal shares whatever the lengths.  A tile
// whose units fall to one block is written to the outputs by it; a tile that
// is cut leaves one partial state (O, L) per block in the workspace, at most
// two per block (its first and its last piece), and the merge kernel joins
// them in the order of the blocks, so the result does not depend on timing.
#pragma once

#include "internal.h"

namespace cpattn {

struct PagedArgs {
  static constexpr bool kDense = false, kBias = false, kDrop = false;
  const void* q;  // [rows][H][d], q_stride elements between rows
  int64_t q_stride;
  const void* k;  // pages: element (page, token, head, i) at page * page_stride + ...
  const void* v;
  int64_t page_stride, token_stride, head_stride;
  const int32_t* table;  // [n_reqs][max_blocks]
  const int32_t* cu;     // [n_reqs + 1]
  const int32_t* lens;   // [n_reqs]
  void* o;               // [rows][H][d]
  float* lse;            // [rows][H]
  float* part_o;         // [2 grid][R][d]
  float* part_l;         // [2 grid][R]
  int32_t n_reqs, max_blocks, n_pages, page_shift;
  int64_t rows;
  int32_t max_keys;  // max_blocks * page_size
  int32_t H, Hkv, G, d;
  int32_t R;  // packed rows of a tile
  uint32_t g_inv, r_inv;  // paged_inverse of G and R
  int32_t row_min, row_max;  // requests of fewer or more packed rows are another launch's
  // that launch, where the call has one (other_R 0: none)
  int32_t other_R, other_min, other_max;
  uint32_t other_r_inv;
  int32_t pairs, blocks;  // what the pair launch and the slice launch have at most
  int32_t pair_cost, slice_cost;  // SM time of a unit of either (ns)
  int32_t causal, window;
  float scale_log2;  // softmax scale * log2(e)
  cp_dtype dtype;
  int32_t grid;  // blocks (or pairs of blocks) of the launch
  int* err;
};

// Device error codes beside the waits' (see read_and_clear_device_error).
constexpr int kErrBadPage = 3;

#ifdef __CUDACC__
#define CPATTN_HD __host__ __device__ __forceinline__
#else
#define CPATTN_HD inline
#endif

// Quotients by numbers that the host knows: a division is 20 instructions, and
// every block makes a dozen of them before it can ask for its first key (with
// the barriers set up by a thread each: one token over 777 keys 12.0 -> 11.4 us, 300 over
// 100 61.9 -> 57.6, 7 short float32 chunks 28.1 -> 26.1).  For
// x < 2^31 the product with floor((2^32 - 1) / n) falls short of x / n by less
// than x / 2^32 < 1/2, so its whole part is the quotient or one less.
CPATTN_HD uint32_t paged_inverse(uint32_t n) { return 0xffffffffu / n; }
CPATTN_HD int32_t paged_quot(uint32_t x, uint32_t n, uint32_t inv) {
  const uint32_t q = uint32_t((uint64_t(x) * inv) >> 32);
  return int32_t(q + (x - q * n >= n ? 1 : 0));
}
// The token of a packed row.
CPATTN_HD int32_t paged_token(const PagedArgs& a, int32_t row) { return paged_quot(uint32_t(row), uint32_t(a.G), a.g_inv); }

struct PagedReq {
  int32_t q0, nq, kv;  // first row of q, new tokens, cached keys (new ones among them)
};

CPATTN_HD int32_t clamp_i32(int32_t x, int32_t lo, int32_t hi) { return x < lo ? lo : (x > hi ? hi : x); }

CPATTN_HD PagedReq paged_req(const PagedArgs& a, int r) {
  PagedReq q;
  q.q0 = clamp_i32(a.cu[r], 0, int32_t(a.rows));
  q.nq = clamp_i32(a.cu[r + 1], q.q0, int32_t(a.rows)) - q.q0;
  if (q.nq * a.G < a.row_min || q.nq * a.G > a.row_max) q.nq = 0;
  q.kv = clamp_i32(a.lens[r], 0, a.max_keys);
  return q;
}

// Tile t of a request: packed rows row0 .. row0 + nrows - 1 and the units
// b0 .. b0 + n - 1 of its keys; lo .. hi - 1: the keys that some row sees.
struct PagedTile {
  int32_t row0, nrows, b0, n, lo, hi;
};

template <class A>
CPATTN_HD int32_t paged_tiles(const A& a, const PagedReq& q) {
  return paged_quot(uint32_t(q.nq) * uint32_t(a.G) + uint32_t(a.R) - 1, uint32_t(a.R), a.r_inv);  // rows * G < 2^31 - R
}

template <int U, class A>
CPATTN_HD PagedTile paged_tile(const A& a, const PagedReq& q, int t) {
  PagedTile x;
  x.row0 = t * a.R;
  const int32_t left = q.nq * a.G - x.row0;
  x.nrows = left < a.R ? left : a.R;
  const int32_t pos0 = q.kv - q.nq + paged_token(a, x.row0), pos1 = q.kv - q.nq + paged_token(a, x.row0 + x.nrows - 1);
  x.hi = a.causal ? (pos1 + 1 < q.kv ? pos1 + 1 : q.kv) : q.kv;
  if (x.hi < 0) x.hi = 0;
  x.lo = a.window > 0 && pos0 - a.window + 1 > 0 ? pos0 - a.window + 1 : 0;
  if (x.lo > x.hi) x.lo = x.hi;
  x.b0 = x.lo / U;
  x.n = x.hi > x.lo ? (x.hi + U - 1) / U - x.b0 : 0;
  return x;
}

// Units of one kv-head of a request.
template <int U, int E, class A>
CPATTN_HD int64_t paged_req_units(const A& a, const PagedReq& q) {
  const int nt = paged_tiles(a, q);
  int64_t s = 0;
  for (int t = 0; t < nt; ++t) s += paged_tile<U>(a, q, t).n + E;
  return s;
}

// Quotient of values below 2^62; the 32-bit division where both fit is several times faster.
CPATTN_HD int64_t paged_div(int64_t x, int64_t y) {
  return ((x | y) >> 31) == 0 ? int64_t(uint32_t(x) / uint32_t(y)) : x / y;
}

// The shares of n blocks; the blocks behind them have none.
struct PagedShare {
  int64_t total, each, more;  // block c: `each` units, one more for c < more
  int32_t n;
  CPATTN_HD PagedShare(int64_t t, int blocks) : total(t), n(blocks > 0 ? blocks : 1) {
    each = paged_div(t, n);
    more = t - each * n;
  }
  CPATTN_HD int64_t first(int c) const { return c >= n ? total : each * c + (c < more ? c : more); }
};

// Pairs of SMs that the many-row requests of a call get where it has few-row
// ones too; the other SMs run the slice launch at the same time.
CPATTN_HD int paged_pairs(const PagedArgs& a, int64_t pair_units, int64_t slice_units) {
  if (slice_units == 0) return a.pairs;
  if (pair_units == 0) return 0;
  const int64_t x = pair_units * a.pair_cost, sum = x + slice_units * a.slice_cost;
  // rounded down: a pair too few costs the many-row requests 1 in 76, one too
  // many could leave the others half of what they need
  const int k = int(float(x) / float(sum) * a.pairs);
  return k < 1 ? 1 : (k > a.pairs - 2 ? a.pairs - 2 : k);
}
// Blocks of this launch that share its units.
CPATTN_HD int paged_blocks(const PagedArgs& a, bool pair, int64_t mine, int64_t others) {
  if (a.other_R == 0) return a.grid;
  const int k = paged_pairs(a, pair ? mine : others, pair ? others : mine);
  return pair ? k : a.blocks - 2 * k;
}
// The other launch's view of the requests.
template <class A>
CPATTN_HD A paged_other(const A& a) {
  A o = a;
  o.R = a.other_R;
  o.r_inv = a.other_r_inv;
  o.row_min = a.other_min;
  o.row_max = a.other_max;
  return o;
}

// Where a unit lies: its tile and the units of the tile before it.
struct PagedStart {
  int32_t r, h, t, off;
};

// One piece of a tile as the block that runs it sees it.
struct PagedPiece {
  PagedReq q;
  PagedTile tile;
  int32_t r, h;
  int32_t ua, ub;   // units [ua, ub) of the tile's n, counted from b0
  int32_t slot;     // -1: the whole tile, written to the outputs; else its partial state
};

// Walks the pieces of one block's share.
template <int U, int E>
struct PagedWalk {
  PagedStart at;
  PagedReq q;
  int32_t nt;
  int64_t left;
  int32_t slot0;
  bool first;

  template <class A>
  CPATTN_HD void start(const A& a, const PagedStart& s, int64_t units, int block) {
    at = s;
    left = units;
    slot0 = 2 * block;
    first = true;
    if (left > 0) {
      q = paged_req(a, at.r);
      nt = paged_tiles(a, q);
    }
  }

  template <class A>
  CPATTN_HD bool next(const A& a, PagedPiece& p) {
    if (left <= 0) return false;
    while (at.t >= nt) {  // the next kv-head, or the next request that has a row
      at.t = 0;
      if (nt > 0 && at.h + 1 < a.Hkv) {
        ++at.h;
        continue;
      }
      at.h = 0;
      if (++at.r >= a.n_reqs) {
        left = 0;
        return false;
      }
      q = paged_req(a, at.r);
      nt = paged_tiles(a, q);
    }
    p.q = q;
    p.r = at.r;
    p.h = at.h;
    p.tile = paged_tile<U>(a, q, at.t);
    const int32_t cost = p.tile.n + E;
    const int32_t rest = cost - at.off;
    const int32_t take = rest < left ? rest : int32_t(left);
    p.ua = at.off < p.tile.n ? at.off : p.tile.n;
    p.ub = at.off + take < p.tile.n ? at.off + take : p.tile.n;
    p.slot = at.off == 0 && take == cost ? -1 : slot0 + (first ? 0 : 1);
    first = false;
    left -= take;
    if (take == rest) {
      at.off = 0;
      ++at.t;
    } else {
      at.off += take;
    }
    return true;
  }
};

// Keys of a unit of each kernel, and what a tile's ends cost in them (16
// prompts of about 400 tokens: pair extra 2 161 us, 4 136, 6 129; 200 single
// tokens over about 200 keys: slice extra 1 62 us, 2 55, 3 53, but one token over 777 keys
// 12.2, 12.5 and 14.2).  kv-head groups wider than kPairRows never reach the pair kernel.
constexpr int kSliceUnit = 64, kSliceExtra = 2;
constexpr int kPairUnit = 128, kPairExtra = 6, kPairRows = 128;

// Units, extra and so on of the launch that is not this one.
template <int U>
struct PagedOther {
  static constexpr int kUnit = U == kPairUnit ? kSliceUnit : kPairUnit;
  static constexpr int kExtra = U == kPairUnit ? kSliceExtra : kPairExtra;
};

enum PagedKernel { kPagedSlice4, kPagedSlice16, kPagedSlice32, kPagedPair };
inline int paged_rows(PagedKernel k, int G) {
  switch (k) {
    case kPagedSlice4: return 4;
    case kPagedSlice16: return 16;
    case kPagedSlice32: return 32;
    case kPagedPair: return 2 * (kPairRows / G) * G;
  }
  return 16;
}

// after_pair: behind a pair launch on the same stream, whose blocks' last
// moments it may overlap (and which is complete when it is).
cp_status launch_paged_slice(const PagedArgs& a, PagedKernel k, bool after_pair, cudaStream_t s);
// Joins the cut tiles of a pair launch, a slice launch or both (grid 0: none).
cp_status launch_paged_merge(const PagedArgs& pair, const PagedArgs& slice, cudaStream_t s);
int paged_slice_grid();
cp_status launch_paged_pair(const PagedArgs& a, cudaStream_t s);
// Pairs of SMs that can run at once (sets the kernel up on the first call).
cp_status paged_pair_grid(int32_t d, int32_t* pairs);

// Rotation of the pairs of a head (cp_rope): turns per position of every
// pair as 64-bit binary fractions, and the pair's axis.
struct RopeTurns {
  uint64_t turn[64];
  uint8_t axis[64];
  int32_t pairs;  // 0: no rotation
  int32_t adjacent, inverse;
};

// Rows of up to three groups of heads: q and k are rotated (when turns.pairs
// > 0), v is copied.  With slots, k and v go to the slots of the cache and
// rows whose slot is outside it are left out (q's too).
struct HeadRows {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;  // elements between rows
  void* q_out;                           // [rows][heads_q][d]
  void* k_out;                           // [rows][heads_k][d], or the cache
  void* v_out;
  int32_t heads_q, heads_k, heads_v, d;
  int64_t rows;
  const int32_t* pos;    // [axes][rows]
  const int32_t* slots;  // [rows] or null
  int32_t page_shift, n_pages;
  int64_t page_stride, token_stride, head_stride;
  RopeTurns turns;
};
cp_status launch_head_rows(const HeadRows& a, cp_dtype dtype, cudaStream_t s);

struct KvTables {
  int32_t n_reqs, max_blocks, page_size, pool;
  int64_t max_rows;
  const int32_t* lens;
  const int32_t* add;  // extend: tokens to add; release: which requests end
  int32_t* free_pages;
  const int32_t* n_free;
  int32_t* table;
  int32_t* lens_out;
  int32_t* cu;
  int32_t* slots;
  int32_t* pos;
  int32_t* n_free_out;
};
constexpr int kMaxTableReqs = 16384;
cp_status launch_kv_extend(const KvTables& a, cudaStream_t s);
cp_status launch_kv_release(const KvTables& a, cudaStream_t s);

}  // namespace cpattn
