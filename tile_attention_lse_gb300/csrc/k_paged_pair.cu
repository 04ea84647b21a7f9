// Paged attention of many rows (bf16) on pairs of SMs
// (cta_group::2, sm_103a): chunks of prompts over their pages.
//
// The mathematics is the slice kernel's (k_paged.cu): one pass over the visible
// keys with a running maximum and sum per row.  With hundreds of rows per key the
// two products are the bound, 4 * 128 flops per (row, key) on the tensor
// cores, and the division of a tile's work over two SMs is that of the ring
// forward (k_fwd_pair.cu): CTA r of a cluster holds 128 packed rows, half of every
// key tile (64 keys) and half of every value tile (64 columns); the even CTA issues
//   S_b = Q K^T (M 256, N 128, K 128) and O += P_b V (P in TMEM),
// two softmax warpgroups take the 128-key tiles in turn, O stays in TMEM.  What differs:
//  - Rows are packed (token * G + head of the group), so the G heads of a kv-head
//    share every load of K and V; a CTA's tile is 128 / G whole tokens.
//  - Pages: the producer warp's lanes issue one box per page and 64 columns
//    (at most 64 keys of a page); lane l looks up the page of the l-th 8 keys of
//    a tile ahead of its use.  A page
//    that no row sees is given the page number n_pages: outside the map, read
//    as zeros without touching memory.
//  - The tile that holds a request's last key inside a page (or a window's
//    first): P is 0 there, but 0 times whatever the page holds may be NaN.
//    V of such a tile is copied by its producer's lanes with plain
//    asynchronous copies that zero-fill the keys outside, a tile or two per
//    piece; all others come by TMA.  V has a producer of its own: its plain copies
//    hold up no K, and a box costs its issuer about 55 ns (pages of 16: 16 boxes a tile).
//  - head_dim 64: K has half the steps.  The second product keeps N = 128: the
//    even CTA's half of V is all 64 columns, the odd one's is never written and
//    its columns of O never read (the pair is bound by its softmax by then, and
//    a half of 32 columns would need another swizzle).
//  - Work is the common axis of paged.h: a pair runs an equal share of
//    all key tiles, and a tile that is cut leaves float32 partial states.
#include <cuda_bf16.h>

#include <atomic>
#include <mutex>

#include "internal.h"
#include "pair_util.cuh"
#include "paged_dev.cuh"
#include "paged_tmap.h"
#include "tc_util.cuh"
#include "tmap.h"

namespace cpattn {

namespace {

using Walk = PagedWalk<kPairUnit, kPairExtra>;
// A softmax warp's walk and its piece, in shared memory: its first lane goes on,
// all read the piece.  In registers they made the tiles' loop spill 268 bytes
// (2048 tokens over 30720 cached: 721 us, 693 from shared memory; 16 prompts of
// 400: 80.3, 77.5).
struct WalkBox {
  Walk w;
  PagedPiece pc;
  int32_t more;
};

constexpr int kThreads = 384;
constexpr int kLaunchRegs = 168;  // per thread at launch (65536 / 384, rounded down to 8)
constexpr int kSmallRegs = 72, kSoftmaxRegs = 216;
static_assert(128 * kSmallRegs + 256 * kSoftmaxRegs == kThreads * kLaunchRegs,
              "register split must add up to the launch total");
constexpr uint32_t kQBytes = 128 * 128 * 2, kQHalf = kQBytes / 2;  // this CTA's Q tile, one 64-column box of it
constexpr uint32_t kKBytes = 64 * 128 * 2;                         // its half of a key tile (64 keys), head_dim 128
constexpr uint32_t kVBytes = 128 * 64 * 2;                         // its half of a value tile (64 columns)
constexpr int kQBufs = 2, kKStages = 4, kVStages = 4, kSBufs = 2;
constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + kQBufs * kQBytes;
constexpr int kOffV = kOffK + kKStages * kKBytes;
constexpr int kOffBar = kOffV + kVStages * kVBytes;
constexpr int kOffX = kOffBar + 512;  // running max [2 tile parities][128], row-sum base and sum [2 piece parities][2 warps][2][128]
constexpr int kOffScan = kOffX + (2 * 128 + 2 * 2 * 2 * 128) * 4;
constexpr int kOffWalk = kOffScan + 64 * 8 + int(sizeof(PagedStart));
constexpr int kSmemBytes = kOffWalk + 8 * int(sizeof(WalkBox));
static_assert(kOffWalk % 8 == 0, "alignment of the walks");
static_assert(kSmemBytes <= 232448, "shared memory budget of one CTA");

// Barrier slots, the same layout in both CTAs.  "even": only the even CTA's
// copy is used; "both": the MMA commits arrive on both copies.
enum {
  B_QFULL0 = 0,                     // even, + buffer: both CTAs' Q bytes landed
  B_QEMPTY0 = B_QFULL0 + kQBufs,    // both, + buffer: the piece's last S has read Q
  B_KFULL0 = B_QEMPTY0 + kQBufs,    // even, + stage
  B_KEMPTY0 = B_KFULL0 + kKStages,  // both, + stage
  B_VFULL0 = B_KEMPTY0 + kKStages,  // even, + stage
  B_VEMPTY0 = B_VFULL0 + kVStages,  // both, + stage
  B_VODD0 = B_VEMPTY0 + kVStages,   // even, + stage: the odd CTA has copied its half of a cut value tile
  B_SFULL0 = B_VODD0 + kVStages,    // both, + S buffer: S_b written
  B_SEMPTY0 = B_SFULL0 + kSBufs,    // even, + S buffer: both CTAs have read S_b (8 warp arrivals)
  B_PFULL0 = B_SEMPTY0 + kSBufs,    // even, + P buffer: P written in both CTAs (8 warp arrivals)
  B_PVDONE0 = B_PFULL0 + kSBufs,    // both, + P buffer: the PV that read it is complete
  B_ODONE = B_PVDONE0 + kSBufs,     // both: the piece's O is final
  B_OEMPTY,                         // even: both CTAs' epilogues have read O (16 warp arrivals)
  B_DRAIN,                          // both: every MMA of both issuers complete (2 arrivals)
  B_MREADY0,                        // + 2 quarter + parity: the running max after a tile of that parity
  B_JOIN0 = B_MREADY0 + 8,          // + quarter: its two warps' row sums of a piece are in shared memory (2 arrivals)
  B_COUNT = B_JOIN0 + 4
};
static_assert(8 * B_COUNT + 8 <= 512, "barrier area");

constexpr uint32_t kIdescS = tc::idesc_bf16(256, 128, /*b_mn_major=*/0);
constexpr uint32_t kIdescPV = tc::idesc_bf16(256, 128, /*b_mn_major=*/1);
// TMEM columns: S_0, S_1 (128 each), P_0, P_1 (64 each), O (128): 512.
constexpr uint32_t kColP = kSBufs * 128;
constexpr uint32_t kColO = kColP + kSBufs * 64;
static_assert(kColO + 128 == 512, "TMEM columns");
constexpr uint16_t kBothCtas = 0x3;

struct Params {
  CUtensorMap tmq;       // [rows][heads][128], box {64, G, 128 / G tokens}
  CUtensorMap tmk, tmv;  // [pages][page][heads][128] (token and head dimensions in the order of their strides)
  PagedArgs a;
  int32_t box_shift;   // log2 keys of a box
  int32_t head_inner;  // the head dimension comes before the token dimension
  long long wait_limit;
};

__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                                 int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
// Arrival on the other CTA's barrier that publishes this CTA's shared memory.
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// kShortWaits: the copy launched while cp_debug_set_wait_limit has set a
// short wait budget; the default copy never reads the limit.
template <int D, bool kShortWaits>
__global__ void __launch_bounds__(kThreads, 1) paged_pair_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = tc::smem_u32(smem);
  if (sbase & 1023) {  // the swizzled layouts need a 1 KB aligned base (the same in both CTAs)
    if (threadIdx.x == 0 && p.a.err) atomicCAS(p.a.err, 0, 2);
    return;
  }
  const uint32_t rank = tc::cluster_ctarank();  // 0: issues the pair's MMAs
  const bool even = rank == 0;
  const uint32_t sQ = sbase + kOffQ, sK = sbase + kOffK, sV = sbase + kOffV;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  auto bar = [&](int i) { return tc::smem_u32(bars + i); };
  auto bar_even = [&](int i) { return tc::map_to_rank(bar(i), 0); };  // the even CTA's copy
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffBar + 8 * B_COUNT);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + 8 * B_COUNT + 4);
  const uint32_t peer_abort = tc::map_to_rank(tc::smem_u32(const_cast<int*>(abort_flag)), rank ^ 1u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedArgs& a = p.a;

  // A wait that gives up stops the peer too (its abort flag, written remotely).
  auto wt = [&](int b, uint32_t parity) -> bool {
    const bool r = tc::wait_bounded<kShortWaits>(bar(b), parity, abort_flag, a.err, p.wait_limit);
    if (!r) tc::st_remote_u32(peer_abort, 1u);
    return r;
  };

  grid_launch_dependents();
  // this pair's share of the units
  const int pair = int(tc::cluster_id_x());
  int64_t* s_scan = reinterpret_cast<int64_t*>(smem + kOffScan);
  PagedStart* s_start = reinterpret_cast<PagedStart*>(smem + kOffScan + 64 * 8);
  const PagedShare share = paged_locate<kPairUnit, kPairExtra, kThreads>(a, s_scan, s_start, pair);
  const int64_t units = share.first(pair + 1) - share.first(pair);
  if (pair >= share.n) return;  // these SMs are the slice launch's

  static_assert(B_COUNT <= kThreads, "a thread a barrier");
  if (const int i = threadIdx.x; i < B_COUNT) {
    uint32_t cnt = 1;
    if ((i >= B_PFULL0 && i < B_PFULL0 + kSBufs) || (i >= B_SEMPTY0 && i < B_SEMPTY0 + kSBufs))
      cnt = 8;  // a tile's 4 softmax warps x 2 CTAs
    if (i == B_OEMPTY) cnt = 16;  // all 8 softmax warps x 2 CTAs
    if (i == B_DRAIN) cnt = 2;    // both issuers
    if (i >= B_JOIN0) cnt = 2;
    tc::mbar_init(bar(i), cnt);
    tc::fence_mbar_init();
  }
  if (threadIdx.x == 0) *abort_flag = 0;
  if (warp == 1) {
    tc::tmem_alloc_pair(tc::smem_u32(tmem_slot), 512);
    tc::tmem_relinquish_pair();
  }
  tc::fence_before_sync();
  tc::cluster_sync();  // both CTAs' barriers exist before any remote arrival, copy or commit
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  Walk w;
  w.start(a, units > 0 ? *s_start : PagedStart{0, 0, 0, 0}, units, pair);
  const int half_rows = a.R >> 1;  // packed rows of a CTA

  if (warp < 4) {
    tc::setmaxnreg_dec<kSmallRegs>();
  }
  if (warp == 0 || warp == 3) {
    // ------------------------------------ producers: Q and K, and V --
    const bool of_k = warp == 0;
    if (lane == 0) {
      if (of_k) tc::prefetch_tmap(&p.tmq);
      tc::prefetch_tmap(of_k ? &p.tmk : &p.tmv);
    }
    uint32_t qi = 0, kg = 0, vg = 0, odd_parity = 0;
    bool ok = true;
    PagedPiece pc{};
    const int bs = p.box_shift, box = 1 << bs;  // keys of a box
    const int in_page = (1 << a.page_shift) - 1;
    // first key of the box that holds key 8 lane of tile t, and whether some row sees one of its keys
    auto box_key = [&](int t) { return t * kPairUnit + ((8 * lane) >> bs << bs); };
    auto seen = [&](int key) { return lane < 16 && key < pc.tile.hi && key + box > pc.tile.lo; };
    // its page, looked up ahead of its use, and checked there: n_pages for what is not read
    auto pages = [&](int t) -> int32_t {
      const int key = box_key(t);
      return seen(key) ? a.table[int64_t(pc.r) * a.max_blocks + (key >> a.page_shift)] : a.n_pages;
    };
    auto checked = [&](int t, int32_t pg) -> int32_t {
      if (uint32_t(pg) < uint32_t(a.n_pages)) return pg;
      if (seen(box_key(t)) && a.err) atomicCAS(a.err, 0, kErrBadPage);
      return a.n_pages;
    };
    auto load_box = [&](uint32_t dst, const CUtensorMap* map, uint32_t fb, int col, int key, int32_t pg) {
      const int token = key & in_page;
      if (p.head_inner)
        tma_load_4d_pair(dst, map, fb, col, pc.h, token, pg);
      else
        tma_load_4d_pair(dst, map, fb, col, token, pc.h, pg);
    };
    auto load_k = [&](int t, int32_t pg) -> bool {
      const uint32_t st = kg % kKStages;
      if (!__all_sync(0xffffffffu, wt(B_KEMPTY0 + st, ((kg / kKStages) & 1) ^ 1))) return false;
      if (even && lane == 0) tc::mbar_arrive_expect_tx(bar(B_KFULL0 + st), 2 * (64 * D * 2));
      // this lane's box: of this CTA's 64 keys those from sub * box on, columns 64 col ..
      const int sub = lane / (D / 64), col = lane % (D / 64);
      const int key = 64 * int(rank) + (sub << bs);
      const int32_t mine = __shfl_sync(0xffffffffu, pg, (key >> 3) & 31);
      if (sub < (64 >> bs))
        load_box(sK + st * kKBytes + col * (kKBytes / 2) + ((sub << bs) * 128), &p.tmk, bar_even(B_KFULL0 + st),
                 64 * col, t * kPairUnit + key, mine);
      ++kg;
      return true;
    };
    auto load_v = [&](int t, int32_t pg) -> bool {
      const uint32_t st = vg % kVStages;
      if (!__all_sync(0xffffffffu, wt(B_VEMPTY0 + st, ((vg / kVStages) & 1) ^ 1))) return false;
      const int k0 = t * kPairUnit, lo = pc.tile.lo, hi = pc.tile.hi;
      // a box that begins before lo, or ends behind the last key of the request
      const bool cut = (lo > k0 && (lo & (box - 1))) ||
                       (hi < k0 + kPairUnit && (hi & (box - 1)) && ((hi | (box - 1)) + 1) > pc.q.kv);
      if (!cut) {
        if (even && lane == 0) tc::mbar_arrive_expect_tx(bar(B_VFULL0 + st), D == 128 ? 2 * kVBytes : kVBytes);
        const int key = lane << bs;
        const int32_t mine = __shfl_sync(0xffffffffu, pg, (key >> 3) & 31);
        if (lane < (128 >> bs))
          load_box(sV + st * kVBytes + key * 128, &p.tmv, bar_even(B_VFULL0 + st), 64 * int(rank), k0 + key, mine);
      } else {
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.v) + pc.h * a.head_stride + 64 * rank;
#pragma unroll 4
        for (int i = 0; i < 32; ++i) {
          const int e = lane + 32 * i, key = e >> 3, c = e & 7;
          const int32_t pgk = __shfl_sync(0xffffffffu, pg, key >> 3);
          const int j = k0 + key;
          const bool in = j >= lo && j < hi && uint32_t(pgk) < uint32_t(a.n_pages);
          const int64_t off = in ? pgk * a.page_stride + int64_t(j & in_page) * a.token_stride + c * 8 : 0;
          cp_async16(sV + st * kVBytes + key * 128 + ((c ^ (key & 7)) << 4), src + off, in);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (D == 64) {
          if (lane == 0) tc::mbar_arrive(bar(B_VFULL0 + st));
        } else if (!even) {
          if (lane == 0) arrive_cluster(bar_even(B_VODD0 + st));
        } else {
          bool r = tc::wait_bounded<kShortWaits, true>(bar(B_VODD0 + st), (odd_parity >> st) & 1, abort_flag, a.err,
                                                       p.wait_limit);
          if (!r) tc::st_remote_u32(peer_abort, 1u);
          if (!__all_sync(0xffffffffu, r)) return false;
          odd_parity ^= 1u << st;
          if (lane == 0) tc::mbar_arrive(bar(B_VFULL0 + st));
        }
      }
      ++vg;
      return true;
    };
    if (D == 64 && !even && !of_k) ok = false;  // no half of V of its own
    while (ok && w.next(a, pc)) {
      const int n = pc.ub - pc.ua, t0 = pc.tile.b0 + pc.ua;
      if (n == 0) continue;
      int32_t pg = pages(t0);
      if (of_k) {
        const uint32_t qb = qi % kQBufs;
        ok = __all_sync(0xffffffffu, wt(B_QEMPTY0 + qb, ((qi / kQBufs) & 1) ^ 1));
        if (!ok) break;
        if (lane == 0) {
          if (even) tc::mbar_arrive_expect_tx(bar(B_QFULL0 + qb), (D / 32) * 128u * uint32_t(half_rows));
          const int tok = pc.q.q0 + paged_token(a, pc.tile.row0 + int(rank) * half_rows), h = pc.h * a.G;
          tc::tma_load_3d_pair(sQ + qb * kQBytes, &p.tmq, bar_even(B_QFULL0 + qb), 0, h, tok);
          if (D == 128) tc::tma_load_3d_pair(sQ + qb * kQBytes + kQHalf, &p.tmq, bar_even(B_QFULL0 + qb), 64, h, tok);
        }
        ++qi;
      }
      for (int t = 0; t < n && ok; ++t) {
        const int32_t now = checked(t0 + t, pg);
        if (t + 1 < n) pg = pages(t0 + t + 1);  // a tile ahead of its use
        ok = of_k ? load_k(t0 + t, now) : load_v(t0 + t, now);
      }
    }
    // Drain: every copy this CTA started has landed before the block exits
    // (the even CTA waits for the phases it armed, which count the odd CTA's
    // bytes too; the odd CTA until each slot it filled was released, or for
    // the default budget where the even CTA stopped consuming).
    if (lane == 0) {
      volatile int never = 0;
      const int first_bar[3] = {even ? B_QFULL0 : B_QEMPTY0, even ? B_KFULL0 : B_KEMPTY0,
                                even ? B_VFULL0 : B_VEMPTY0};
      for (int s = 0; s < kQBufs; ++s) {
        const uint32_t used = (qi + kQBufs - 1 - s) / kQBufs;
        if (used) tc::mbar_wait(bar(first_bar[0] + s), (used - 1) & 1, &never, nullptr);
      }
      for (int s = 0; s < kKStages; ++s) {
        const uint32_t used = (kg + kKStages - 1 - s) / kKStages;
        if (used) tc::mbar_wait(bar(first_bar[1] + s), (used - 1) & 1, &never, nullptr);
      }
      for (int s = 0; s < kVStages; ++s) {
        const uint32_t used = (vg + kVStages - 1 - s) / kVStages;
        if (used) tc::mbar_wait(bar(first_bar[2] + s), (used - 1) & 1, &never, nullptr);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // --------------------------------- S = Q K^T issuer (even CTA only) --
    if (even && lane == 0) {
      uint32_t qi = 0, kg = 0, g = 0;
      bool ok = true;
      PagedPiece pc;
      while (ok && w.next(a, pc)) {
        const int n = pc.ub - pc.ua;
        if (n == 0) continue;
        const uint32_t qb = qi % kQBufs;
        ok = wt(B_QFULL0 + qb, (qi / kQBufs) & 1);
        ++qi;
        if (!ok) break;
        tc::fence_after_sync();
        const uint64_t qd = tc::kmajor_desc(sQ + qb * kQBytes);
        for (int t = 0; t < n && ok; ++t, ++g, ++kg) {
          const uint32_t sb = g % kSBufs;
          // S buffer sb was last read by the softmax of tile g - 2
          if (g >= uint32_t(kSBufs)) {
            ok = wt(B_SEMPTY0 + sb, ((g / kSBufs) - 1) & 1);
            if (!ok) break;
          }
          const uint32_t st = kg % kKStages;
          ok = wt(B_KFULL0 + st, (kg / kKStages) & 1);
          if (!ok) break;
          tc::fence_after_sync();
          const uint64_t kd = tc::kmajor_desc(sK + st * kKBytes);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc::mma_pair_ss(tmem + sb * 128, tc::kmajor_step(qd, kk), khalf_step(kd, kk), kIdescS, kk > 0 ? 1u : 0u);
          tc::mma_commit_pair(bar(B_SFULL0 + sb), kBothCtas);
          tc::mma_commit_pair(bar(B_KEMPTY0 + st), kBothCtas);
          if (t == n - 1) tc::mma_commit_pair(bar(B_QEMPTY0 + qb), kBothCtas);
        }
      }
      tc::mma_commit_pair(bar(B_DRAIN), kBothCtas);
    }
  } else if (warp == 2) {
    // -------------------------------- O += P V issuer (even CTA only) --
    if (even && lane == 0) {
      uint32_t vg = 0, g = 0, items = 0;
      bool ok = true;
      PagedPiece pc;
      while (ok && w.next(a, pc)) {
        const int n = pc.ub - pc.ua;
        if (n == 0) continue;
        // the first PV of a piece overwrites O: both epilogues of the previous one have read it
        if (items > 0) {
          ok = wt(B_OEMPTY, (items - 1) & 1);
          if (!ok) break;
        }
        ++items;
        for (int t = 0; t < n && ok; ++t, ++g, ++vg) {
          const uint32_t sb = g % kSBufs;
          ok = wt(B_PFULL0 + sb, (g / kSBufs) & 1);
          if (!ok) break;
          const uint32_t vs = vg % kVStages;
          ok = wt(B_VFULL0 + vs, (vg / kVStages) & 1);
          if (!ok) break;
          tc::fence_after_sync();
          const uint64_t vd = tc::mnmajor_desc(sV + vs * kVBytes);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // P (bf16 pairs in TMEM) x V (MN-major smem)
            tc::mma_pair_ts(tmem + kColO, tmem + kColP + sb * 64 + kk * 8, tc::mnmajor_step(vd, kk), kIdescPV,
                            (t > 0 || kk > 0) ? 1u : 0u);
          tc::mma_commit_pair(bar(B_PVDONE0 + sb), kBothCtas);
          tc::mma_commit_pair(bar(B_VEMPTY0 + vs), kBothCtas);
          if (t == n - 1) tc::mma_commit_pair(bar(B_ODONE), kBothCtas);
        }
      }
      tc::mma_commit_pair(bar(B_DRAIN), kBothCtas);
    }
  } else if (warp >= 4) {
    tc::setmaxnreg_inc<kSoftmaxRegs>();
    // ----------------------------------------------------- softmax warps --
    // As in the ring forward: warps 4..7 the even tiles of the pair's stream,
    // warps 8..11 the odd ones; warp w reads TMEM lanes 32 (w % 4) .. +31 and
    // its thread `row` owns packed row rank * half_rows + row of the tile.  The running max passes
    // from tile to tile through shared memory (B_MREADY); a tile moves it only
    // when it lifts it by more than 2^8.  Each warp keeps the row sum of its own
    // tiles; the two warps of a quarter join theirs at the end of a piece and
    // write 64 columns each.  A warp without a row keeps the barriers' pace only.
    const int half = (warp - 4) >> 2;  // this warp takes the tiles g with g % 2 == half
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_off = uint32_t(quarter * 32) << 16;
    const uint32_t tO = tmem + lane_off + kColO;
    float* mrow = reinterpret_cast<float*>(smem + kOffX);  // [tile parity][row]
    float* xjoin = mrow + 2 * 128;                          // [piece parity][warp half][base m, sum][row]
    const float sl2 = a.scale_log2;
    const uint64_t sl2x2 = tc::f32x2(sl2, sl2);
    uint32_t g = 0, items = 0, pieces = 0;
    bool ok = true;
    WalkBox& box = reinterpret_cast<WalkBox*>(smem + kOffWalk)[warp - 4];
    const PagedPiece& pc = box.pc;
    if (lane == 0) box.w.start(a, units > 0 ? *s_start : PagedStart{0, 0, 0, 0}, units, pair);
    // One call of next() serves the first piece and, between a piece's tiles
    // and its O, the one behind it: the last PV is still running then.
    bool have = false;
    for (;;) {
      int n = 0, rows_here = 0, slot = -1, trow = 0;
      bool row_ok = false, idle = true;
      int64_t at = 0;
      float inv = 0.f;
      if (have) {
        n = pc.ub - pc.ua;
        const int t0 = pc.tile.b0 + pc.ua;
        rows_here = min(max(pc.tile.nrows - int(rank) * half_rows, 0), half_rows);
        row_ok = row < rows_here;
        idle = quarter * 32 >= rows_here;  // no row of this warp
        // rows behind the last are masked like it (their sums go nowhere)
        const int prow = pc.tile.row0 + int(rank) * half_rows + min(row, max(rows_here - 1, 0));
        const int qpos = pc.q.kv - pc.q.nq + prow / a.G;
        const int vis_hi = a.causal ? min(pc.q.kv, qpos + 1) : pc.q.kv;
        const int vis_lo = a.window > 0 ? max(qpos - a.window + 1, 0) : 0;
        float m_own = -INFINITY, l = 0.f;  // this warp's row sum and the max it is taken against
        for (int t = 0; t < n && ok; ++t, ++g) {
          if (int(g & 1) != half) continue;  // the other warp's tile
          const uint32_t sb = g % kSBufs;
          ok = __all_sync(0xffffffffu, wt(B_SFULL0 + sb, (g / kSBufs) & 1));
          if (!ok) break;
          tc::fence_after_sync();
          // visible keys of this row in this tile: lo <= j < limit
          const int kpos0 = (t0 + t) * kPairUnit;
          const int limit = min(vis_hi - kpos0, kTile);
          const int lo0 = max(vis_lo - kpos0, 0);
          const bool full = __all_sync(0xffffffffu, limit >= kTile && lo0 == 0);
          const uint32_t span = uint32_t(max(limit - lo0, 0));
          const uint32_t tS = tmem + lane_off + sb * 128;
          uint32_t sr[128];
          float mx = -INFINITY;
          if (full && !idle) {
            tc::tmem_ld32(tS, sr);
            tc::tmem_ld32(tS + 32, sr + 32);
            tc::tmem_ld32(tS + 64, sr + 64);
            tc::tmem_ld32(tS + 96, sr + 96);
            tc::tmem_wait_ld();
          }
          if (full || idle) {  // the scores are in registers: S_sb may take the next tile's scores
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_remote(bar_even(B_SEMPTY0 + sb));
            if (!idle) mx = row_max<false>(sr, 0, kTile) * sl2;
          } else {
            // A tile that the mask cuts is read 32 scores at a time, now and
            // again for P, in loops: unrolled like the others its code
            // came from memory once a launch, 4 to 11 us.
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t s32[32];
              tc::tmem_ld32(tS + 32 * c, s32);
              tc::tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j)
                mx = fmaxf(mx, uint32_t(32 * c + j - lo0) < span ? __uint_as_float(s32[j]) : -INFINITY);
            }
            mx *= sl2;
          }
          // the running max after tile g - 1 (every tile but the stream's first
          // waits, so each barrier is waited once per phase; a piece's first tile
          // starts from -inf)
          float m_in = -INFINITY;
          if (g > 0) {
            const uint32_t pq = (g - 1) & 1;
            ok = __all_sync(0xffffffffu, wt(B_MREADY0 + 2 * quarter + int(pq), ((g - 1) >> 1) & 1));
            if (!ok) break;
            if (t > 0) m_in = mrow[pq * 128 + row];
          }
          const float m_up = fmaxf(m_in, mx);
          const bool grow = m_up > m_in + 8.0f;  // also true when m_in is -inf and m_up finite
          const float m = grow ? m_up : m_in;
          mrow[(g & 1) * 128 + row] = m;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(bar(B_MREADY0 + 2 * quarter + int(g & 1)));
          if (m != m_own) {  // this warp's sum, against the new max
            l *= tc::ex2(m_own - m);  // from -inf: 0, or NaN where a score was
            m_own = m;
          }
          const float mu = (m == -INFINITY) ? 0.f : m;
          // P buffer sb was last read by the PV of tile g - 2 (this warp waits
          // for every such phase, in order)
          if (g >= uint32_t(kSBufs)) {
            ok = __all_sync(0xffffffffu, wt(B_PVDONE0 + sb, ((g / kSBufs) - 1) & 1));
            if (!ok) break;
            tc::fence_after_sync();
          }
          if (!idle) {
            const uint32_t tP = tmem + lane_off + kColP + sb * 64;
            if (full) {
              l += p_pass<false>(sr, 0, kTile, mu, sl2x2, tP);
            } else {
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                uint32_t s32[32], pk[16];
                tc::tmem_ld32(tS + 32 * c, s32);
                tc::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                  const int k = 32 * c + j - lo0;
                  const float p0 = uint32_t(k) < span ? tc::ex2(fmaf(__uint_as_float(s32[j]), sl2, -mu)) : 0.f;
                  const float p1 = uint32_t(k + 1) < span ? tc::ex2(fmaf(__uint_as_float(s32[j + 1]), sl2, -mu)) : 0.f;
                  l += p0 + p1;
                  pk[j / 2] = tc::pack_bf16x2(p0, p1);
                }
                tc::tmem_st16(tP + 16 * c, pk);
              }
              tc::fence_before_sync();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive_remote(bar_even(B_SEMPTY0 + sb));
            }
            if (t > 0 && __any_sync(0xffffffffu, grow)) {
              // O holds the sum up to tile g - 1 against m_in once the PV that
              // read P of tile g - 1 is complete (the next PV waits for this P).
              // That phase is the latest one of its barrier: PV(g - 3) is
              // complete (PV(g - 2) is, see above) and PV(g + 1) waits for PV(g).
              const float corr = (m_in == -INFINITY) ? 0.f : tc::ex2(m_in - m);
              const uint32_t pb = (g - 1) % kSBufs;
              ok = __all_sync(0xffffffffu, wt(B_PVDONE0 + pb, ((g - 1) / kSBufs) & 1));
              if (!ok) break;
              tc::fence_after_sync();
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t orr[32];
                tc::tmem_ld32(tO + c * 32, orr);
                tc::tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j) orr[j] = __float_as_uint(__uint_as_float(orr[j]) * corr);
                tc::tmem_st32(tO + c * 32, orr);
              }
            }
            tc::tmem_wait_st();
          }
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive_remote(bar_even(B_PFULL0 + sb));
        }
        if (!ok) break;
        // ------------------------------------------------------ epilogue --
        // What does not need O comes first: the last PV is still running.  The
        // row's sum over both warps' tiles is taken against the final max (the
        // larger of the two bases: the max never decreases along the stream).
        float* xend = xjoin + (pieces & 1) * 512;
        xend[half * 256 + row] = m_own;
        xend[half * 256 + 128 + row] = l;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(B_JOIN0 + quarter));
        ok = __all_sync(0xffffffffu, wt(B_JOIN0 + quarter, pieces & 1));
        if (!ok) break;
        ++pieces;
        const float m_o = xend[(half ^ 1) * 256 + row], l_o = xend[(half ^ 1) * 256 + 128 + row];
        const float m_fin = fmaxf(m_own, m_o);
        const float l_all = m_fin == -INFINITY ? l + l_o : l * tc::ex2(m_own - m_fin) + l_o * tc::ex2(m_o - m_fin);
        inv = l_all == 0.f ? 0.f : 1.f / l_all;
        // A whole tile writes the final O (bf16, round to nearest even) and LSE;
        // a piece of one its partial state (O in float32, LSE in log2 units).
        slot = pc.slot;
        const bool direct = slot < 0;
        trow = int(rank) * half_rows + row;
        const int packed = pc.tile.row0 + trow;
        const int tok = paged_token(a, packed);
        at = direct ? int64_t(pc.q.q0 + tok) * a.H + pc.h * a.G + (packed - tok * a.G)
                    : int64_t(slot) * a.R + trow;
        if (row_ok && half == 0) {
          const float l2 = l_all == 0.f ? -INFINITY : m_fin + tc::lg2(l_all);
          if (direct)
            a.lse[at] = l2 * 0.69314718055994531f;
          else
            a.part_l[at] = l2;
        }
      }
      __syncwarp();  // every lane has read the piece
      if (lane == 0) box.more = box.w.next(a, box.pc);
      __syncwarp();
      const bool more = box.more;
      if (!have) {
        if (!more) break;
        have = true;
        continue;
      }
      const bool direct = slot < 0;
      const int c0 = D / 2 * half;  // each warp writes half of the columns
      if (n > 0) {
        ok = __all_sync(0xffffffffu, wt(B_ODONE, items & 1));
        if (!ok) break;
        tc::fence_after_sync();
        ++items;
      }
#pragma unroll
      for (int cc = 0; cc < D / 64; ++cc) {
        uint32_t orr[32];
        if (n > 0 && !idle) {
          tc::tmem_ld32(tO + c0 + cc * 32, orr);
          tc::tmem_wait_ld();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) orr[j] = 0u;
        }
        if (n > 0 && cc == D / 64 - 1) {  // O is in registers: the next piece's first PV may overwrite it
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive_remote(bar_even(B_OEMPTY));
        }
        if (idle) continue;
        if (direct) {
          uint4 v[4];  // 16-byte chunk j of this lane's row
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t* e = orr + 8 * j;
            v[j] = make_uint4(tc::pack_bf16x2(__uint_as_float(e[0]) * inv, __uint_as_float(e[1]) * inv),
                              tc::pack_bf16x2(__uint_as_float(e[2]) * inv, __uint_as_float(e[3]) * inv),
                              tc::pack_bf16x2(__uint_as_float(e[4]) * inv, __uint_as_float(e[5]) * inv),
                              tc::pack_bf16x2(__uint_as_float(e[6]) * inv, __uint_as_float(e[7]) * inv));
          }
          // four lanes turn their rows' chunks about: chunk (lane & 3) of row j
          // of the four, so that a store writes 64 bytes of a row
#pragma unroll
          for (int s = 1; s < 4; s <<= 1) {
            const bool up = lane & s;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (j & s) continue;
              const uint4 send = up ? v[j] : v[j | s];
              uint4 got;
              got.x = __shfl_xor_sync(0xffffffffu, send.x, s);
              got.y = __shfl_xor_sync(0xffffffffu, send.y, s);
              got.z = __shfl_xor_sync(0xffffffffu, send.z, s);
              got.w = __shfl_xor_sync(0xffffffffu, send.w, s);
              if (up)
                v[j] = got;
              else
                v[j | s] = got;
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t at_j = __shfl_sync(0xffffffffu, at, (lane & ~3) + j);
            if (quarter * 32 + (lane & ~3) + j < rows_here)
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + at_j * D + c0 + cc * 32 + 8 * (lane & 3)) =
                  v[j];
          }
        } else if (row_ok) {
          // partial O: [slot][4 columns][row] float4, the rows of a warp side by side
          float4* dst = reinterpret_cast<float4*>(a.part_o) +
                        (int64_t(slot) * (D / 4) + (c0 + cc * 32) / 4) * a.R + trow;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            dst[int64_t(j) * a.R] =
                make_float4(__uint_as_float(orr[4 * j]) * inv, __uint_as_float(orr[4 * j + 1]) * inv,
                            __uint_as_float(orr[4 * j + 2]) * inv, __uint_as_float(orr[4 * j + 3]) * inv);
        }
      }
      if (!more) break;
    }
  }

  // Teardown: every MMA of the pair is complete (both CTAs) and both CTAs are
  // done with TMEM before the pair frees it.
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) {
      volatile int never = 0;
      tc::mbar_wait(bar(B_DRAIN), 0, &never, nullptr);
    }
    __syncwarp();
  }
  tc::fence_before_sync();
  tc::cluster_sync();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc_pair(tmem, 512);
}

// Map of q: box of 64 columns, the G heads of a kv-head and `tokens` rows.
bool make_tmap_packed(CUtensorMap* map, const PagedArgs& a, int tokens) {
  auto enc = tmap_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {cuuint64_t(a.d), cuuint64_t(a.H), cuuint64_t(a.rows)};
  const cuuint64_t strides[2] = {cuuint64_t(a.d) * 2, cuuint64_t(a.q_stride) * 2};
  const cuuint32_t b[3] = {64, cuuint32_t(a.G), cuuint32_t(tokens)};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, b, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaLaunchConfig_t pair_config(cudaLaunchAttribute* attr, int pairs, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(2 * unsigned(pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

using Kernel = void (*)(Params);
Kernel pair_kernel(int d, bool short_waits) {
  if (d == 128) return short_waits ? paged_pair_kernel<128, true> : paged_pair_kernel<128, false>;
  return short_waits ? paged_pair_kernel<64, true> : paged_pair_kernel<64, false>;
}

}  // namespace

cp_status paged_pair_grid(int32_t d, int32_t* pairs) {
  const bool short_waits = wait_limit_cycles() < tc::kWaitCycles;
  const Kernel kern = pair_kernel(d, short_waits);
  // per copy and device, set up by the first launch (under a lock: host threads may race on it)
  static std::atomic<int> max_pairs[4][64] = {};
  const int copy = (d == 128 ? 2 : 0) + short_waits;
  static std::mutex setup_mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CP_ERR_CUDA;
  int n = max_pairs[copy][dev].load(std::memory_order_acquire);
  if (n == 0) {
    std::lock_guard<std::mutex> lock(setup_mu);
    // The register hand-over inside the kernel assumes the launch count.
    cudaFuncAttributes fa{};
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return CP_ERR_CUDA;
    if (fa.numRegs != kLaunchRegs) return CP_ERR_UNSUPPORTED;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess)
      return CP_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pair_config(attr, num_sms() / 2, nullptr);
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) return CP_ERR_UNSUPPORTED;
    if (n > num_sms() / 2) n = num_sms() / 2;
    max_pairs[copy][dev].store(n, std::memory_order_release);
  }
  *pairs = n;
  return CP_OK;
}

cp_status launch_paged_pair(const PagedArgs& a, cudaStream_t s) {
  if (a.dtype != CP_BF16 || a.G > kPairRows) return CP_ERR_UNSUPPORTED;
  Params p;
  const int page = 1 << a.page_shift, box = page < 64 ? page : 64;
  if (!make_tmap_packed(&p.tmq, a, kPairRows / a.G) || !make_tmap_pages(&p.tmk, a.k, a, box) ||
      !make_tmap_pages(&p.tmv, a.v, a, box))
    return CP_ERR_CUDA;
  p.a = a;
  p.box_shift = 0;
  while ((1 << p.box_shift) < box) ++p.box_shift;
  p.head_inner = a.head_stride <= a.token_stride;
  p.wait_limit = wait_limit_cycles();
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pair_config(attr, a.grid, s);
  const Kernel kern = pair_kernel(a.d, p.wait_limit < tc::kWaitCycles);
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return CP_ERR_CUDA;
  return cuda_status(cudaGetLastError());
}

}  // namespace cpattn
