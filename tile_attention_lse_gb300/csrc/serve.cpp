// extern "C" boundary of the serving operators: request tables of a paged K/V
// cache, multi-axis rotary positions, cache append, paged attention.  Argument
// validation and launches on the caller's stream; nothing here allocates.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "internal.h"
#include "paged.h"

using namespace cpattn;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int64_t elem(cp_dtype t) { return t == CP_BF16 ? 2 : 4; }
bool row_aligned(int64_t stride, cp_dtype t) { return stride * elem(t) % 16 == 0; }

int log2_of(int32_t x) {
  int n = 0;
  while ((int64_t(1) << n) < x) ++n;
  return n;
}

cp_status check_cache(const cp_kv_cache* c) {
  if (!c || c->n_pages < 1 || c->heads_kv < 1) return CP_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return CP_ERR_UNSUPPORTED;
  if (c->dtype != CP_F32 && c->dtype != CP_BF16) return CP_ERR_UNSUPPORTED;
  if (c->page_size < 8 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return CP_ERR_UNSUPPORTED;
  if (int64_t(c->n_pages) * c->page_size >= (int64_t(1) << 31)) return CP_ERR_UNSUPPORTED;
  if (!c->k || !c->v) return CP_ERR_INVALID_ARG;
  if (c->page_stride < 0 || c->token_stride < c->head_dim || c->head_stride < c->head_dim) return CP_ERR_INVALID_ARG;
  if (c->n_pages > 1 && c->page_stride < c->head_dim) return CP_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !row_aligned(c->page_stride, c->dtype) ||
      !row_aligned(c->token_stride, c->dtype) || !row_aligned(c->head_stride, c->dtype))
    return CP_ERR_ALIGNMENT;
  return CP_OK;
}

// Axis and exponent of every pair, and its turns per position as a 64-bit
// binary fraction (whole turns fall away: positions are whole numbers).
// The table of the last rotation is kept (by its contents): 64 powers cost
// as much host time as the launch.
cp_status make_turns(const cp_rope* r, int32_t head_dim, RopeTurns* t);

cp_status fill_turns(const cp_rope* r, int32_t head_dim, RopeTurns* t) {
  static thread_local cp_rope last = {};
  static thread_local int32_t last_dim = 0;
  static thread_local RopeTurns kept;
  *t = RopeTurns{};
  if (!r) return CP_OK;
  const bool same = last_dim == head_dim && last.n_axes == r->n_axes && last.base == r->base &&
                    last.interleaved == r->interleaved && last.restart == r->restart &&
                    last.adjacent == r->adjacent && std::memcmp(last.section, r->section, sizeof(r->section)) == 0;
  if (!same) {
    last_dim = 0;
    const cp_status st = make_turns(r, head_dim, &kept);
    if (st != CP_OK) return st;
    last = *r;
    last_dim = head_dim;
  }
  *t = kept;
  return CP_OK;
}

cp_status make_turns(const cp_rope* r, int32_t head_dim, RopeTurns* t) {
  *t = RopeTurns{};
  if (r->n_axes < 1 || r->n_axes > 4 || !(r->base > 0.f) || !std::isfinite(r->base)) return CP_ERR_INVALID_ARG;
  int32_t pairs = 0, left[4] = {}, seen[4] = {};
  for (int i = 0; i < r->n_axes; ++i) {
    if (r->section[i] < 0 || r->section[i] > head_dim / 2) return CP_ERR_INVALID_ARG;
    left[i] = r->section[i];
    pairs += r->section[i];
  }
  if (pairs < 1 || pairs > head_dim / 2) return CP_ERR_INVALID_ARG;
  if (pairs % 8 != 0) return CP_ERR_UNSUPPORTED;
  t->pairs = pairs;
  t->adjacent = r->adjacent != 0;
  int axis = 0;
  for (int i = 0; i < pairs; ++i) {
    while (left[axis] == 0) axis = (axis + 1) % r->n_axes;
    --left[axis];
    t->axis[i] = uint8_t(axis);
    const double e = r->restart ? double(seen[axis]++) / r->section[axis] : double(i) / pairs;
    const double turn = std::pow(double(r->base), -e) * 0.15915494309189535;  // / 2 pi
    const double frac = turn - std::floor(turn);
    // frac * 2^64 in two exact halves: a double holds 53 bits
    const double hi = std::floor(frac * 4294967296.0);
    const double lo = (frac * 4294967296.0 - hi) * 4294967296.0;
    t->turn[i] = (uint64_t(hi) << 32) + uint64_t(lo);
    if (r->interleaved) axis = (axis + 1) % r->n_axes;
  }
  return CP_OK;
}

// The launches of a call, by its types and by the packed rows of a request
// (max_new * G at most).  bf16: requests of up to 16 rows run on the slice kernel
// (bound by their keys' bytes), and so do up to 32 where none has more
// (32 requests of 8 tokens over 4000 keys, 4 heads a group: 101 us, 131 on
// the pair kernel); those of more on the pair kernel (bound by the products and the
// softmax).  Where both may come, both are launched, each for its own
// requests and on its own share of the SMs, at the same time (20 single tokens and 4
// chunks of up to 509 over 6000 cached tokens: 251 us with all of them on the
// pair kernel, 177 one after the other, 164 together, 161 by now).  A single request of
// unknown length runs on the pair kernel whatever it brings.
struct PagedPlan {
  PagedKernel slice = kPagedSlice16;
  bool use_slice = true, use_pair = false;
};
PagedPlan pick_kernels(const cp_paged_desc& d, int32_t n_reqs) {
  const int64_t G = d.heads_q / d.kv.heads_kv;
  const int64_t rows = d.max_new > 0 ? G * d.max_new : INT64_MAX;
  PagedPlan p;
  if (d.kv.dtype == CP_F32) {
    p.slice = rows <= 4 ? kPagedSlice4 : kPagedSlice16;
  } else if (rows > 32 && G <= kPairRows) {
    p.use_pair = true;
    p.use_slice = n_reqs > 1 && G <= 16;
  } else if (rows > 16) {
    p.slice = kPagedSlice32;
  }
  return p;
}

cp_status check_paged(const cp_paged_desc* d) {
  if (!d) return CP_ERR_INVALID_ARG;
  const cp_status st = check_cache(&d->kv);
  if (st != CP_OK) return st;
  if (d->heads_q < 1 || d->max_new < 0 || d->window < 0 || d->window >= (1 << 30)) return CP_ERR_INVALID_ARG;
  if (!(d->softmax_scale >= 0.f) || !std::isfinite(d->softmax_scale)) return CP_ERR_INVALID_ARG;
  if (d->heads_q % d->kv.heads_kv != 0) return CP_ERR_UNSUPPORTED;
  return CP_OK;
}

// Sizes of a call on a checked descriptor: packed rows (less a tile) and keys are 32-bit numbers.
cp_status check_paged_sizes(const cp_paged_desc& d, int64_t rows, int32_t max_blocks) {
  if (rows >= (int64_t(1) << 31) || rows * (d.heads_q / d.kv.heads_kv) >= (int64_t(1) << 31) - 1024 ||
      int64_t(max_blocks) * d.kv.page_size > (int64_t(1) << 30))
    return CP_ERR_UNSUPPORTED;
  return CP_OK;
}

// Walks every block's share on the host.
template <int U, int E, typename F>
void walk_all(const PagedArgs& a, F f) {
  int64_t total = 0, others = 0;
  for (int r = 0; r < a.n_reqs; ++r) total += paged_req_units<U, E>(a, paged_req(a, r)) * a.Hkv;
  if (a.other_R > 0) {
    const PagedArgs o = paged_other(a);
    for (int r = 0; r < a.n_reqs; ++r)
      others += paged_req_units<PagedOther<U>::kUnit, PagedOther<U>::kExtra>(o, paged_req(o, r)) * a.Hkv;
  }
  const PagedShare share(total, paged_blocks(a, U == kPairUnit, total, others));
  PagedStart at{0, 0, 0, 0};
  for (int c = 0; c < a.grid; ++c) {
    const int64_t u0 = share.first(c), u1 = share.first(c + 1);
    if (u1 <= u0) continue;
    // where u0 lies: the walk of the block before ended there; step over what
    // has no tile
    PagedReq q = paged_req(a, at.r);
    while (at.t >= paged_tiles(a, q)) {
      at.t = 0;
      if (paged_tiles(a, q) > 0 && at.h + 1 < a.Hkv) {
        ++at.h;
      } else {
        at.h = 0;
        ++at.r;
        q = paged_req(a, at.r);
      }
    }
    PagedWalk<U, E> w;
    w.start(a, at, u1 - u0, c);
    PagedPiece p;
    while (w.next(a, p)) {
      const int32_t k0 = (p.tile.b0 + p.ua) * U, k1 = (p.tile.b0 + p.ub) * U;
      const int32_t lo = clamp_i32(k0, p.tile.lo, p.tile.hi), hi = clamp_i32(k1, p.tile.lo, p.tile.hi);
      f(c, p, lo, hi);
    }
    at = w.at;
  }
}

// Partial states: two per block, the pair launch's in front of the slice launch's.
int pair_blocks(const PagedPlan& p) { return p.use_pair ? paged_slice_grid() / 2 : 0; }
int64_t pair_states(const cp_paged_desc& d, const PagedPlan& p) {
  return int64_t(2) * pair_blocks(p) * paged_rows(kPagedPair, d.heads_q / d.kv.heads_kv);
}
int64_t slice_states(const cp_paged_desc& d, const PagedPlan& p) {
  return p.use_slice ? int64_t(2) * paged_slice_grid() * paged_rows(p.slice, d.heads_q / d.kv.heads_kv) : 0;
}

// What both launches of a call share.
PagedArgs paged_args(const cp_paged_desc& d, int32_t n_reqs, int64_t rows, int32_t max_blocks, const int32_t* cu,
                     const int32_t* lens) {
  PagedArgs a{};
  a.cu = cu;
  a.lens = lens;
  a.n_reqs = n_reqs;
  a.rows = rows;
  a.max_blocks = max_blocks;
  a.max_keys = max_blocks * d.kv.page_size;
  a.H = d.heads_q;
  a.Hkv = d.kv.heads_kv;
  a.G = a.H / a.Hkv;
  a.g_inv = paged_inverse(uint32_t(a.G));
  a.d = d.kv.head_dim;
  a.dtype = d.kv.dtype;
  a.causal = d.causal != 0;
  a.window = d.window;
  a.page_shift = log2_of(d.kv.page_size);
  a.row_max = INT32_MAX;
  return a;
}
void split_args(const PagedPlan& p, const PagedArgs& a, PagedArgs* pair, PagedArgs* slice) {
  *pair = *slice = a;
  pair->R = paged_rows(kPagedPair, p.use_pair ? a.G : 1);
  slice->R = paged_rows(p.slice, a.G);
  pair->r_inv = slice->other_r_inv = paged_inverse(uint32_t(pair->R));
  slice->r_inv = pair->other_r_inv = paged_inverse(uint32_t(slice->R));
  pair->grid = pair_blocks(p);
  slice->grid = p.use_slice ? paged_slice_grid() : 0;
  if (p.use_pair && p.use_slice) {
    pair->row_min = slice->other_min = 17;
    slice->row_max = pair->other_max = 16;
    slice->other_max = INT32_MAX;
    pair->other_R = slice->R;
    slice->other_R = pair->R;
    pair->pairs = slice->pairs = pair->grid;
    pair->blocks = slice->blocks = slice->grid;
    // What gave the shortest times on batches of both, by page size: a slice
    // unit's time on one SM (64 keys of K and V, at head_dim 128 32 KB: 480 ns are
    // 68 GB/s) and twice a pair unit's on its two, for both head_dims alike as the softmax
    // bounds it (alone, 1024 tokens over 8192 to 40960: 1.54 us at head_dim 64 and
    // 1.71 at 128 in pages of 64, 2.11 and 2.10 in pages of 8, whose boxes bound it).
    const bool wide = a.d == 128;
    const int page = 1 << a.page_shift;
    pair->pair_cost = slice->pair_cost = page == 8 ? 2400 : 1800;
    pair->slice_cost = slice->slice_cost =
        page >= 64 ? (wide ? 480 : 290) : page == 32 ? (wide ? 500 : 290) : page == 16 ? (wide ? 640 : 340) : (wide ? 950 : 520);
  }
}

}  // namespace

extern "C" {

cp_status cp_kv_extend(int32_t n_reqs, int32_t max_blocks, int32_t page_size, int64_t max_rows, int32_t n_pool,
                       const int32_t* lens, const int32_t* add, const int32_t* free_pages, const int32_t* n_free,
                       int32_t* block_table, int32_t* lens_out, int32_t* cu_new, int32_t* slots, int32_t* pos,
                       int32_t* n_free_out, void* stream) {
  if (n_reqs < 0 || max_blocks < 1 || page_size < 1 || max_rows < 0 || n_pool < 0) return CP_ERR_INVALID_ARG;
  if (n_reqs > kMaxTableReqs || max_rows >= (int64_t(1) << 31) ||
      int64_t(max_blocks) * page_size > (int64_t(1) << 30))
    return CP_ERR_UNSUPPORTED;
  if (!n_free || !cu_new || !n_free_out || n_free == n_free_out) return CP_ERR_INVALID_ARG;
  if (n_reqs > 0 && (!lens || !add || !block_table || !lens_out || lens == lens_out)) return CP_ERR_INVALID_ARG;
  if (n_pool > 0 && !free_pages) return CP_ERR_INVALID_ARG;
  if (max_rows > 0 && (!slots || !pos)) return CP_ERR_INVALID_ARG;
  KvTables a{};
  a.n_reqs = n_reqs;
  a.max_blocks = max_blocks;
  a.page_size = page_size;
  a.pool = n_pool;
  a.max_rows = max_rows;
  a.lens = lens;
  a.add = add;
  a.free_pages = const_cast<int32_t*>(free_pages);
  a.n_free = n_free;
  a.table = block_table;
  a.lens_out = lens_out;
  a.cu = cu_new;
  a.slots = slots;
  a.pos = pos;
  a.n_free_out = n_free_out;
  ProfScope ps(CP_K_KV_TABLES, static_cast<cudaStream_t>(stream));
  return launch_kv_extend(a, static_cast<cudaStream_t>(stream));
}

cp_status cp_kv_release(int32_t n_reqs, int32_t max_blocks, int32_t page_size, int32_t n_pool, const int32_t* lens,
                        const int32_t* done, int32_t* free_pages, const int32_t* n_free, int32_t* block_table,
                        int32_t* lens_out, int32_t* n_free_out, void* stream) {
  if (n_reqs < 0 || max_blocks < 1 || page_size < 1 || n_pool < 0) return CP_ERR_INVALID_ARG;
  if (n_reqs > kMaxTableReqs || int64_t(max_blocks) * page_size > (int64_t(1) << 30)) return CP_ERR_UNSUPPORTED;
  if (!n_free || !n_free_out || n_free == n_free_out) return CP_ERR_INVALID_ARG;
  if (n_reqs > 0 && (!lens || !done || !block_table || !lens_out || lens == lens_out)) return CP_ERR_INVALID_ARG;
  if (n_pool > 0 && !free_pages) return CP_ERR_INVALID_ARG;
  KvTables a{};
  a.n_reqs = n_reqs;
  a.max_blocks = max_blocks;
  a.page_size = page_size;
  a.pool = n_pool;
  a.lens = lens;
  a.add = done;
  a.free_pages = free_pages;
  a.n_free = n_free;
  a.table = block_table;
  a.lens_out = lens_out;
  a.n_free_out = n_free_out;
  ProfScope ps(CP_K_KV_TABLES, static_cast<cudaStream_t>(stream));
  return launch_kv_release(a, static_cast<cudaStream_t>(stream));
}

cp_status cp_rope_axes(const cp_rope* rope, const int32_t* pos, int64_t rows, int32_t head_dim, cp_dtype dtype,
                       int32_t heads_q, const void* q, int64_t q_stride, void* q_out, int32_t heads_k, const void* k,
                       int64_t k_stride, void* k_out, int32_t inverse, void* stream) {
  if (!rope || rows < 0 || heads_q < 1 || heads_k < 0) return CP_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return CP_ERR_UNSUPPORTED;
  if (dtype != CP_F32 && dtype != CP_BF16) return CP_ERR_UNSUPPORTED;
  if (rows >= (int64_t(1) << 31)) return CP_ERR_UNSUPPORTED;
  HeadRows a{};
  const cp_status st = fill_turns(rope, head_dim, &a.turns);
  if (st != CP_OK) return st;
  if (rows == 0) return CP_OK;
  if (!pos || !q || !q_out || (heads_k > 0 && (!k || !k_out))) return CP_ERR_INVALID_ARG;
  const int64_t qw = int64_t(heads_q) * head_dim, kw = int64_t(heads_k) * head_dim;
  if (q_stride < qw || (heads_k > 0 && k_stride < kw)) return CP_ERR_INVALID_ARG;
  // in place only where every element stays where it is
  if ((q == q_out && q_stride != qw && rows > 1) || (heads_k > 0 && k == k_out && k_stride != kw && rows > 1))
    return CP_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(q_out, 16) || !row_aligned(q_stride, dtype)) return CP_ERR_ALIGNMENT;
  if (heads_k > 0 && (!aligned(k, 16) || !aligned(k_out, 16) || !row_aligned(k_stride, dtype)))
    return CP_ERR_ALIGNMENT;
  a.turns.inverse = inverse != 0;
  a.q = q;
  a.k = k;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.q_out = q_out;
  a.k_out = k_out;
  a.heads_q = heads_q;
  a.heads_k = heads_k;
  a.d = head_dim;
  a.rows = rows;
  a.pos = pos;
  ProfScope ps(CP_K_HEAD_ROWS, static_cast<cudaStream_t>(stream));
  return launch_head_rows(a, dtype, static_cast<cudaStream_t>(stream));
}

cp_status cp_kv_append(const cp_kv_cache* cache, const int32_t* slots, int64_t rows, const void* k, int64_t k_stride,
                       const void* v, int64_t v_stride, const cp_rope* rope, const int32_t* pos, int32_t heads_q,
                       const void* q, int64_t q_stride, void* q_out, void* stream) {
  cp_status st = check_cache(cache);
  if (st != CP_OK) return st;
  if (rows < 0 || heads_q < 0 || (heads_q > 0 && !rope)) return CP_ERR_INVALID_ARG;
  if (rows >= (int64_t(1) << 31)) return CP_ERR_UNSUPPORTED;
  HeadRows a{};
  st = fill_turns(rope, cache->head_dim, &a.turns);
  if (st != CP_OK) return st;
  if (rows == 0) return CP_OK;
  if (!slots || !k || !v || (rope && !pos) || (heads_q > 0 && (!q || !q_out))) return CP_ERR_INVALID_ARG;
  const int64_t kw = int64_t(cache->heads_kv) * cache->head_dim, qw = int64_t(heads_q) * cache->head_dim;
  if (k_stride < kw || v_stride < kw || (heads_q > 0 && q_stride < qw)) return CP_ERR_INVALID_ARG;
  if (heads_q > 0 && q == q_out && q_stride != qw && rows > 1) return CP_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !row_aligned(k_stride, cache->dtype) ||
      !row_aligned(v_stride, cache->dtype))
    return CP_ERR_ALIGNMENT;
  if (heads_q > 0 && (!aligned(q, 16) || !aligned(q_out, 16) || !row_aligned(q_stride, cache->dtype)))
    return CP_ERR_ALIGNMENT;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out = q_out;
  a.k_out = cache->k;
  a.v_out = cache->v;
  a.heads_q = heads_q;
  a.heads_k = a.heads_v = cache->heads_kv;
  a.d = cache->head_dim;
  a.rows = rows;
  a.pos = pos;
  a.slots = slots;
  a.page_shift = log2_of(cache->page_size);
  a.n_pages = cache->n_pages;
  a.page_stride = cache->page_stride;
  a.token_stride = cache->token_stride;
  a.head_stride = cache->head_stride;
  ProfScope ps(CP_K_HEAD_ROWS, static_cast<cudaStream_t>(stream));
  return launch_head_rows(a, cache->dtype, static_cast<cudaStream_t>(stream));
}

cp_status cp_validate_paged_desc(const cp_paged_desc* desc) { return check_paged(desc); }

size_t cp_paged_attn_workspace_bytes(const cp_paged_desc* desc) {
  if (check_paged(desc) != CP_OK) return 0;
  const PagedPlan p = pick_kernels(*desc, 2);  // the most that any number of requests takes
  return size_t(pair_states(*desc, p) + slice_states(*desc, p)) * (size_t(desc->kv.head_dim) + 1) * 4;
}

cp_status cp_paged_schedule(const cp_paged_desc* desc, int32_t n_reqs, int64_t rows, int32_t max_blocks,
                            const int32_t* cu_new, const int32_t* kv_lens, int32_t* grid, int64_t* n,
                            int32_t* pieces) {
  cp_status st = check_paged(desc);
  if (st != CP_OK) return st;
  if (n_reqs < 1 || rows < 0 || max_blocks < 1 || !cu_new || !kv_lens) return CP_ERR_INVALID_ARG;
  st = check_paged_sizes(*desc, rows, max_blocks);
  if (st != CP_OK) return st;
  const PagedPlan plan = pick_kernels(*desc, n_reqs);
  PagedArgs pair, slice;
  split_args(plan, paged_args(*desc, n_reqs, rows, max_blocks, cu_new, kv_lens), &pair, &slice);
  int32_t pairs = 0;
  if (plan.use_pair && paged_pair_grid(desc->kv.head_dim, &pairs) == CP_OK)
    pair.pairs = slice.pairs = pair.grid = pairs;  // what the launch takes on this device
  else
    cudaGetLastError();  // no device: half of the SMs
  if (grid) *grid = pair.grid + slice.grid;
  int64_t count = 0;
  int first = 0;
  auto f = [&](int c, const PagedPiece& p, int32_t k0, int32_t k1) {
    if (pieces) {
      const int32_t row[8] = {first + c, p.r,  p.h, p.tile.row0, p.tile.nrows,
                              k0,        k1, p.slot < 0 ? -1 : 2 * first + p.slot};
      for (int i = 0; i < 8; ++i) pieces[8 * count + i] = row[i];
    }
    ++count;
  };
  if (plan.use_pair) walk_all<kPairUnit, kPairExtra>(pair, f);
  first = pair.grid;
  if (plan.use_slice) walk_all<kSliceUnit, kSliceExtra>(slice, f);
  if (n) *n = count;
  return CP_OK;
}

cp_status cp_paged_attn_fwd(const cp_paged_desc* desc, int32_t n_reqs, int64_t rows, int32_t max_blocks,
                            const void* q, int64_t q_stride, const int32_t* block_table, const int32_t* cu_new,
                            const int32_t* kv_lens, void* o, float* lse, void* ws, size_t ws_bytes, void* stream) {
  cp_status st = check_paged(desc);
  if (st != CP_OK) return st;
  if (n_reqs < 0 || rows < 0 || max_blocks < 1) return CP_ERR_INVALID_ARG;
  const cp_kv_cache& c = desc->kv;
  st = check_paged_sizes(*desc, rows, max_blocks);
  if (st != CP_OK) return st;
  if (n_reqs == 0 || rows == 0) return CP_OK;
  if (!q || !block_table || !cu_new || !kv_lens || !o || !lse || !ws || !aligned(ws, 256)) return CP_ERR_INVALID_ARG;
  if (q_stride < int64_t(desc->heads_q) * c.head_dim) return CP_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !row_aligned(q_stride, c.dtype)) return CP_ERR_ALIGNMENT;
  if (ws_bytes < cp_paged_attn_workspace_bytes(desc)) return CP_ERR_WORKSPACE;
  if (!tc_available()) return CP_ERR_UNSUPPORTED;
  const PagedPlan plan = pick_kernels(*desc, n_reqs);
  PagedArgs a = paged_args(*desc, n_reqs, rows, max_blocks, cu_new, kv_lens);
  a.q = q;
  a.q_stride = q_stride;
  a.k = c.k;
  a.v = c.v;
  a.page_stride = c.page_stride;
  a.token_stride = c.token_stride;
  a.head_stride = c.head_stride;
  a.table = block_table;
  a.o = o;
  a.lse = lse;
  a.n_pages = c.n_pages;
  const float scale = desc->softmax_scale > 0.f ? desc->softmax_scale : 1.f / std::sqrt(float(c.head_dim));
  a.scale_log2 = scale * 1.4426950408889634f;
  a.err = device_error_ptr();
  PagedArgs pair, slice;
  split_args(plan, a, &pair, &slice);
  const int64_t states = pair_states(*desc, plan) + slice_states(*desc, plan);
  pair.part_o = static_cast<float*>(ws);
  pair.part_l = pair.part_o + states * c.head_dim;
  slice.part_o = pair.part_o + pair_states(*desc, plan) * c.head_dim;
  slice.part_l = pair.part_l + pair_states(*desc, plan);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cp_status r = CP_OK;
  if (plan.use_pair) {
    r = paged_pair_grid(c.head_dim, &pair.grid);
    if (r != CP_OK) return r;
    pair.pairs = slice.pairs = pair.grid;
    ProfScope ps(CP_K_PAGED, s);
    r = launch_paged_pair(pair, s);
    if (r != CP_OK) return r;
  }
  if (plan.use_slice) {
    ProfScope ps(CP_K_PAGED, s);
    r = launch_paged_slice(slice, plan.slice, plan.use_pair, s);
    if (r != CP_OK) return r;
  }
  ProfScope ps(CP_K_PAGED_MERGE, s);
  return launch_paged_merge(pair, slice, s);
}

}  // extern "C"
