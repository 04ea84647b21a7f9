// extern "C" boundary of cross attention: attention of packed query sequences
// over packed key sequences of other lengths, with a bias of the relative
// position and dropout.  Argument validation, the layout of the workspace and
// launches on the caller's stream; nothing here allocates.
#include "cross.h"

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "internal.h"

using namespace cpattn;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int64_t elem(cp_dtype t) { return t == CP_BF16 ? 2 : 4; }
bool row_ok(const void* p, int64_t stride, cp_dtype t) { return aligned(p, 16) && stride * elem(t) % 16 == 0; }
size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// Pieces of 15 bits below this one drop their probability: p 2^15 to the nearest, halves to even.
uint32_t drop_min(const cp_cross_desc& d) {
  const double x = double(d.dropout) * 32768.0, low = std::floor(x), over = x - low;
  return uint32_t(low) + (over > 0.5 || (over == 0.5 && (int64_t(low) & 1)) ? 1 : 0);
}

cp_status check(const cp_cross_desc* d) {
  if (!d || d->heads_q < 1 || d->heads_kv < 1 || d->max_q < 0) return CP_ERR_INVALID_ARG;
  if (d->head_dim != 64 && d->head_dim != 128) return CP_ERR_UNSUPPORTED;
  if (d->dtype != CP_F32 && d->dtype != CP_BF16) return CP_ERR_UNSUPPORTED;
  if (d->heads_q % d->heads_kv != 0) return CP_ERR_UNSUPPORTED;
  if (!(d->softmax_scale >= 0.f) || !std::isfinite(d->softmax_scale)) return CP_ERR_INVALID_ARG;
  if (!(d->dropout >= 0.f) || !(d->dropout < 1.f) || drop_min(*d) > 32767) return CP_ERR_INVALID_ARG;
  if (d->rel_buckets != 0) {
    if (d->rel_buckets < 0 || (d->rel_both && d->rel_buckets % 2)) return CP_ERR_INVALID_ARG;
    const int32_t per = d->rel_both ? d->rel_buckets / 2 : d->rel_buckets;
    if (per < 2 || d->rel_max_distance < per / 2) return CP_ERR_INVALID_ARG;
    if (d->rel_buckets > kMaxBuckets || d->rel_max_distance > 65536) return CP_ERR_UNSUPPORTED;
  }
  // a head is a row of the spread's grid
  if (d->rel_buckets != 0 && d->heads_q > 65535) return CP_ERR_UNSUPPORTED;
  // dropout in bf16 is the pair kernel's, which packs a group's heads into a tile
  if (d->dtype == CP_BF16 && d->dropout > 0.f && d->heads_q / d->heads_kv > kPairRows) return CP_ERR_UNSUPPORTED;
  return CP_OK;
}

cp_status check_sizes(const cp_cross_desc& d, int32_t n_seqs, int64_t rows_q, int64_t rows_k) {
  if (n_seqs < 0 || rows_q < 0 || rows_k < 0) return CP_ERR_INVALID_ARG;
  // packed rows (less a tile), sequences times heads and keys are 32-bit numbers
  const int64_t most = int64_t(1) << 31;
  if (rows_q >= most || rows_q * (d.heads_q / d.heads_kv) >= most - 1024 || rows_k > (int64_t(1) << 30) ||
      int64_t(n_seqs) * d.heads_q >= most || int64_t(n_seqs) + rows_k / 64 >= most || int64_t(n_seqs) + rows_q / 64 >= most)
    return CP_ERR_UNSUPPORTED;
  return CP_OK;
}

// The distances that the buckets of a direction start at: 0, 1, .. for the first
// half, then e (max / e)^(t / (per - e)), e = per / 2, t = 0, 1, ..
// (Those of the last call are kept, by what they come from: the powers cost as much host time as a launch.)
RelStarts rel_starts(const cp_cross_desc& d) {
  static thread_local RelStarts kept = {};
  static thread_local int32_t buckets = 0, distance = 0, both = 0;
  if (buckets == d.rel_buckets && distance == d.rel_max_distance && both == d.rel_both) return kept;
  RelStarts s{};
  s.both = d.rel_both != 0;
  s.per = s.both ? d.rel_buckets / 2 : d.rel_buckets;
  const int32_t e = s.per / 2;
  for (int32_t b = 0; b < s.per; ++b) {
    if (b < e) {
      s.start[b] = b;
    } else {
      const double x = e * std::pow(double(d.rel_max_distance) / e, double(b - e) / (s.per - e));
      s.start[b] = int32_t(std::ceil(x * (1.0 - 1e-12)));
    }
  }
  kept = s;
  buckets = d.rel_buckets;
  distance = d.rel_max_distance;
  both = d.rel_both;
  return s;
}
struct RelLayout {
  int32_t reach, zero, stride;
};
RelLayout rel_layout(const cp_cross_desc& d) {
  if (!d.rel_buckets) return RelLayout{0, 0, 0};
  const RelStarts s = rel_starts(d);
  const int32_t reach = s.start[s.per - 1];
  return RelLayout{reach, reach + kRelPad, (2 * (reach + kRelPad) + 4) & ~3};
}

// The forward's kernel, by types and by the packed rows of a sequence (max_q * G).
// bf16: up to 16 and up to 32 rows are bound by the bytes of their keys and run on the slice
// kernel, more on the pair kernel, as in the paged attention (serve.cpp has both sides
// measured), and so does all dropout.  Groups wider than the pair kernel's tile stay on slices.
// With rest under a bias P goes into its product in two parts, which is the pair kernel's
// (64 sequences of 2 queries over 2000 keys, 16 heads of 64, with a bias: 95 us on slices, 352 so).
// float32 is all the slice kernel's.
PagedKernel pick(const cp_cross_desc& d, bool rest) {
  const int64_t G = d.heads_q / d.heads_kv, rows = d.max_q > 0 ? G * d.max_q : INT64_MAX;
  if (d.dtype == CP_F32) return rows <= 4 ? kPagedSlice4 : kPagedSlice16;
  if (d.dropout > 0.f || (rest && d.rel_buckets)) return kPagedPair;
  if (rows <= 16 || G > kPairRows) return kPagedSlice16;
  return rows <= 32 ? kPagedSlice32 : kPagedPair;
}

int64_t fwd_states(const cp_cross_desc& d, PagedKernel k) {
  const int64_t blocks = k == kPagedPair ? paged_slice_grid() / 2 : paged_slice_grid();
  return 2 * blocks * paged_rows(k, d.heads_q / d.heads_kv);
}

// The workspace: the spread biases, then the forward's partial states or what
// the backward keeps, from the same place on.
struct Layout {
  size_t states = 0, total = 0;
  // backward
  size_t k_list = 0, q_list = 0, counts = 0, delta = 0, lse2 = 0, part = 0, dq_acc = 0;
  int32_t k_most = 0, q_most = 0, size = 0, parts = 0, stride = 0;
};
Layout layout(const cp_cross_desc& d, int64_t rows_q, int64_t rows_k, int32_t n_seqs, bool backward) {
  Layout l;
  l.states = up256(size_t(d.heads_q) * rel_layout(d).stride * 4);
  const bool fine = d.dtype == CP_BF16 && d.heads_q / d.heads_kv <= kPairRows;  // a rest may be asked for
  const int64_t states = std::max(fwd_states(d, pick(d, false)), fwd_states(d, pick(d, fine)));
  l.total = l.states + size_t(states) * (size_t(d.head_dim) + 1) * 4;
  if (!backward) return l;
  const bool bf16 = d.dtype == CP_BF16;
  l.size = bf16 ? 128 : 64;
  // every sequence has at most one tile that is not full
  l.k_most = int32_t(rows_k / l.size + n_seqs);
  l.q_most = bf16 ? 0 : int32_t(rows_q / l.size + n_seqs);
  l.parts = bf16 ? 8 : 1;
  l.stride = d.rel_buckets <= 32 ? 32 : 64;
  size_t at = l.states;
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at += up256(bytes);
    return x;
  };
  const size_t rh = size_t(rows_q) * d.heads_q;
  l.counts = take(2 * 4);
  l.k_list = take(size_t(l.k_most) * sizeof(CrossTile));
  l.q_list = take(size_t(l.q_most) * sizeof(CrossTile));
  l.delta = take(rh * 4);
  l.lse2 = take(rh * 4);
  l.part = take(d.rel_buckets ? size_t(l.k_most) * d.heads_q * l.parts * l.stride * 4 : 0);
  l.dq_acc = take(bf16 ? rh * d.head_dim * 4 : 0);
  l.total = std::max(l.total, at);
  return l;
}

CrossArgs cross_args(const cp_cross_desc& d, int32_t n_seqs, int64_t rows_q, int64_t rows_k, const void* q,
                     int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                     const int32_t* cu_q, const int32_t* cu_k, const int32_t* len_q, const int32_t* len_k,
                     const uint64_t* rng, char* ws) {
  CrossArgs a{};
  // without rows: a map of one row that nothing reads
  a.q = q ? q : k;
  a.k = k ? k : q;
  a.v = v ? v : a.k;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.cu = cu_q;
  a.cu_k = cu_k;
  a.len_q = len_q;
  a.len_k = len_k;
  a.n_reqs = n_seqs;
  a.rows = rows_q;
  a.rows_k = rows_k;
  a.max_keys = int32_t(rows_k);
  a.H = d.heads_q;
  a.Hkv = d.heads_kv;
  a.G = a.H / a.Hkv;
  a.g_inv = paged_inverse(uint32_t(a.G));
  a.d = d.head_dim;
  a.dtype = d.dtype;
  a.causal = d.causal != 0;
  a.row_max = INT32_MAX;
  a.n_pages = 1;  // the slice kernel's view: one page of all rows
  a.page_shift = 30;
  a.token_stride = a.k_stride;
  a.head_stride = a.d;
  const float scale = d.softmax_scale > 0.f ? d.softmax_scale : 1.f / std::sqrt(float(d.head_dim));
  a.scale_log2 = scale * 1.4426950408889634f;
  a.err = device_error_ptr();
  if (d.rel_buckets) {
    const RelLayout r = rel_layout(d);
    a.rel = reinterpret_cast<float*>(ws);
    a.rel_stride = r.stride;
    a.rel_zero = r.zero;
    a.reach = r.reach;
  }
  a.drop_scale = 1.f;
  if (d.dropout > 0.f) {
    a.rng = rng;
    a.drop_min = drop_min(d);
    a.drop_scale = 1.f / (1.f - float(a.drop_min) / 32768.f);
  }
  return a;
}

cp_status spread(const cp_cross_desc& d, const CrossArgs& a, const void* bias, cudaStream_t s) {
  RelSpread r;
  r.table = bias;
  r.rel = const_cast<float*>(a.rel);
  r.heads = a.H;
  r.rel_stride = a.rel_stride;
  r.rel_zero = a.rel_zero;
  r.starts = rel_starts(d);
  ProfScope ps(CP_K_CROSS_PREP, s);
  return launch_rel_spread(r, d.dtype, s);
}

// The checks that both directions share.
cp_status check_call(const cp_cross_desc* desc, int64_t rows_q, int64_t rows_k, const void* q, int64_t q_stride,
                     const void* k, int64_t k_stride, const void* v, int64_t v_stride, const int32_t* cu_q,
                     const int32_t* cu_k, const void* bias, const uint64_t* rng) {
  if (!cu_q || !cu_k || (rows_q > 0 && !q) || (rows_k > 0 && (!k || !v))) return CP_ERR_INVALID_ARG;
  if ((desc->rel_buckets != 0) != (bias != nullptr)) return CP_ERR_INVALID_ARG;
  if (desc->dropout > 0.f && (!rng || !aligned(rng, 8))) return CP_ERR_INVALID_ARG;
  const int64_t qw = int64_t(desc->heads_q) * desc->head_dim, kw = int64_t(desc->heads_kv) * desc->head_dim;
  if ((rows_q > 0 && q_stride < qw) || (rows_k > 0 && (k_stride < kw || v_stride < kw))) return CP_ERR_INVALID_ARG;
  // strides of a tensor map are below 2^40 bytes
  const int64_t most = (int64_t(1) << 40) / 4;
  if (q_stride >= most || k_stride >= most || v_stride >= most) return CP_ERR_UNSUPPORTED;
  if (rows_q > 0 && !row_ok(q, q_stride, desc->dtype)) return CP_ERR_ALIGNMENT;
  if (rows_k > 0 && (!row_ok(k, k_stride, desc->dtype) || !row_ok(v, v_stride, desc->dtype))) return CP_ERR_ALIGNMENT;
  return CP_OK;
}

}  // namespace

extern "C" {

cp_status cp_validate_cross_desc(const cp_cross_desc* desc) { return check(desc); }

size_t cp_cross_attn_workspace_bytes(const cp_cross_desc* desc, int32_t n_seqs, int64_t rows_q, int64_t rows_k,
                                     int32_t backward) {
  if (check(desc) != CP_OK || check_sizes(*desc, n_seqs, rows_q, rows_k) != CP_OK) return 0;
  return layout(*desc, rows_q, rows_k, n_seqs, backward != 0).total;
}

cp_status cp_cross_attn_fwd(const cp_cross_desc* desc, int32_t n_seqs, int64_t rows_q, int64_t rows_k, const void* q,
                            int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                            const int32_t* cu_q, const int32_t* cu_k, const int32_t* len_q, const int32_t* len_k,
                            const void* bias, const uint64_t* rng, void* o, void* rest, float* lse, void* ws,
                            size_t ws_bytes, void* stream) {
  cp_status st = check(desc);
  if (st != CP_OK) return st;
  st = check_sizes(*desc, n_seqs, rows_q, rows_k);
  if (st != CP_OK) return st;
  if (n_seqs == 0 || rows_q == 0) return CP_OK;
  st = check_call(desc, rows_q, rows_k, q, q_stride, k, k_stride, v, v_stride, cu_q, cu_k, bias, rng);
  if (st != CP_OK) return st;
  if (!o || !lse || !ws || !aligned(ws, 256)) return CP_ERR_INVALID_ARG;
  if (rest && desc->dtype != CP_BF16) return CP_ERR_INVALID_ARG;
  if (rest && bias && desc->heads_q / desc->heads_kv > kPairRows) return CP_ERR_UNSUPPORTED;
  if (!aligned(o, 16) || !aligned(rest, 16)) return CP_ERR_ALIGNMENT;
  const Layout l = layout(*desc, rows_q, rows_k, n_seqs, false);
  if (ws_bytes < l.total) return CP_ERR_WORKSPACE;
  if (!tc_available()) return CP_ERR_UNSUPPORTED;
  char* w = static_cast<char*>(ws);
  if (rows_k == 0) {  // a map of one row: q's strides fit
    k_stride = v_stride = q_stride;
    k = v = q;
  }
  CrossArgs a = cross_args(*desc, n_seqs, rows_q, rows_k, q, q_stride, k, k_stride, v, v_stride, cu_q, cu_k, len_q,
                           len_k, rng, w);
  a.o = o;
  a.lse = lse;
  a.rest = rest;
  const PagedKernel kern = pick(*desc, rest != nullptr);
  a.R = paged_rows(kern, a.G);
  a.r_inv = paged_inverse(uint32_t(a.R));
  a.part_o = reinterpret_cast<float*>(w + l.states);
  a.part_l = a.part_o + fwd_states(*desc, kern) * a.d;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (kern == kPagedPair) {
    st = cross_pair_grid(a, &a.grid);
    if (st != CP_OK) return st;
  } else {
    a.grid = paged_slice_grid();
  }
  if (a.rel) {
    st = spread(*desc, a, bias, s);
    if (st != CP_OK) return st;
  }
  {
    ProfScope ps(CP_K_CROSS, s);
    st = kern == kPagedPair ? launch_cross_pair(a, a.rel != nullptr, s)
                            : launch_cross_few(a, kern, a.rel != nullptr, s);
    if (st != CP_OK) return st;
  }
  ProfScope ps(CP_K_CROSS_MERGE, s);
  return launch_cross_merge(a, kern == kPagedPair, s);
}

cp_status cp_cross_attn_bwd(const cp_cross_desc* desc, int32_t n_seqs, int64_t rows_q, int64_t rows_k, const void* q,
                            int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                            const void* o, const void* rest, const float* lse, const void* dout, int64_t dout_stride,
                            const int32_t* cu_q, const int32_t* cu_k, const int32_t* len_q, const int32_t* len_k,
                            const void* bias, const uint64_t* rng, void* dq, void* dk, void* dv, void* dbias, void* ws,
                            size_t ws_bytes, void* stream) {
  cp_status st = check(desc);
  if (st != CP_OK) return st;
  st = check_sizes(*desc, n_seqs, rows_q, rows_k);
  if (st != CP_OK) return st;
  st = check_call(desc, rows_q, rows_k, q, q_stride, k, k_stride, v, v_stride, cu_q, cu_k, bias, rng);
  if (st != CP_OK) return st;
  if ((rows_q > 0 && (!o || !lse || !dout || !dq)) || (rows_k > 0 && (!dk || !dv)) || (bias && !dbias) || !ws ||
      !aligned(ws, 256))
    return CP_ERR_INVALID_ARG;
  if (rest && desc->dtype != CP_BF16) return CP_ERR_INVALID_ARG;
  // no forward leaves the rest that the table's gradient needs
  if (bias && desc->dtype == CP_BF16 && desc->heads_q / desc->heads_kv > kPairRows) return CP_ERR_UNSUPPORTED;
  if (rows_q > 0 && dout_stride < int64_t(desc->heads_q) * desc->head_dim) return CP_ERR_INVALID_ARG;
  if (dout_stride >= (int64_t(1) << 40) / 4) return CP_ERR_UNSUPPORTED;
  if (!aligned(o, 16) || !aligned(rest, 16) || (rows_q > 0 && !row_ok(dout, dout_stride, desc->dtype)) ||
      !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16))
    return CP_ERR_ALIGNMENT;
  const Layout l = layout(*desc, rows_q, rows_k, n_seqs, true);
  if (ws_bytes < l.total) return CP_ERR_WORKSPACE;
  if (!tc_available()) return CP_ERR_UNSUPPORTED;
  char* w = static_cast<char*>(ws);
  const bool empty = rows_q == 0 || rows_k == 0;  // as without sequences: zeros
  if (empty) n_seqs = 0;
  CrossBwd a{};
  static_cast<CrossArgs&>(a) = cross_args(*desc, n_seqs, rows_q, rows_k, q, q_stride, k, k_stride, v, v_stride, cu_q,
                                          cu_k, len_q, len_k, rng, w);
  a.o = const_cast<void*>(o);
  a.rest = const_cast<void*>(rest);
  a.lse = const_cast<float*>(lse);
  a.dout = dout;
  a.do_stride = dout_stride;
  a.delta = reinterpret_cast<float*>(w + l.delta);
  a.lse2 = reinterpret_cast<float*>(w + l.lse2);
  a.dq_acc = desc->dtype == CP_BF16 ? reinterpret_cast<float*>(w + l.dq_acc) : nullptr;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.dtable = dbias;
  a.part = reinterpret_cast<float*>(w + l.part);
  a.parts = l.parts;
  a.buckets = desc->rel_buckets;
  a.bucket_stride = l.stride;
  int32_t* counts = reinterpret_cast<int32_t*>(w + l.counts);
  a.k_tiles = CrossTiles{reinterpret_cast<CrossTile*>(w + l.k_list), counts, l.k_most, l.size};
  a.q_tiles = CrossTiles{reinterpret_cast<CrossTile*>(w + l.q_list), counts + 1, l.q_most, l.size};
  if (desc->rel_buckets) a.starts = rel_starts(*desc);
  a.scale = a.scale_log2 * 0.69314718055994531f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.rel) {
    st = spread(*desc, a, bias, s);
    if (st != CP_OK) return st;
  }
  {
    ProfScope ps(CP_K_CROSS_PREP, s);
    st = launch_cross_bwd_prep(a, s);
    if (st != CP_OK) return st;
  }
  if (!empty && n_seqs > 0) {
    ProfScope ps(CP_K_CROSS_BWD, s);
    st = desc->dtype == CP_BF16 ? launch_cross_bwd(a, s) : launch_cross_bwd_f32(a, s);
    if (st != CP_OK) return st;
  }
  ProfScope ps(CP_K_CROSS_POST, s);
  return launch_cross_bwd_post(a, s);
}

}  // extern "C"
