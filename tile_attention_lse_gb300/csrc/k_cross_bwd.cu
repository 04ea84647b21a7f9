// Backward of cross attention in bf16 on the tensor cores (tcgen05, sm_103a): one
// persistent kernel over tiles of keys, with the gradients of a bias of the relative
// position and under dropout.
//
// The formulas stand in cross.h.  One item is a tile of 128 keys of a sequence and one
// kv-head, with the query tiles (128 rows) of every q-head of the group, so that dK and dV
// are summed in TMEM and written once.  Per query tile:
//     S^T  = K Q^T   -> TMEM [0,128)    keep P^T (bf16) is written over it
//     dP^T = V dO^T  -> TMEM [128,256)
//     dV  += P^T dO  (A = P^T from TMEM, dO read MN-major) -> TMEM [256, 256 + D)
//     dK  += dS^T Q  (A = dS^T from shared memory, Q MN-major) -> TMEM [384, 384 + D)
//     dQ_t = dS K    (A = the same dS^T tile read MN-major, K MN-major)
//                    -> TMEM [128, 128 + D) once dS^T has been taken from dP^T
// The division into roles, the issue order and the read-out of dQ by TMA reductions
// into float32 are those of the ring backward (k_bwd_tc.cu), and so is the bound: five products on
// one SM's tensor core, whose issue waits for the key-row math in between.  (The order of the
// reductions is not fixed, so dQ may differ in the last bits between calls.)
//   Warps: 0 TMA, 1 MMA (+TMEM owner), 2 stages L2 and D of the query tile, 3 clears the
//   rows of cut tiles, 4..11 key-row math (two warps per TMEM lane quarter, each on 64 query
//   columns), 12..15 dQ read-out and reductions.
// What is this kernel's own:
//  - Where a sequence ends inside a tile of Q, dO or K and other rows follow, the copy
//    counts on a barrier of its own and warp 3 clears the rows behind the end before the
//    products may read them: 0 times what follows need not be 0.
//  - Dropout: a lane draws for 8 keys and every eighth query of its 64; the 8 lanes of
//    those keys exchange byte masks, 16 registers for P and dP.
//  - Bias: dS of a tile stays in float32 registers for the table's gradient (the sum
//    over a far bucket nearly cancels: rounded to bf16 it would be off by 2^-9 sqrt(n / w)
//    for n keys of which w lie near).  A tile beyond `reach` adds its sum to one number.  Another one sums its
//    diagonals by passing sums from lane to lane while the columns go by (down for those that
//    start at the first column, up for the others), then one sum over the lanes of a bucket's run gives
//    its share; lane b keeps bucket b.  Sums of a head and key tile go to a place of their own
//    and are added in a fixed order behind the kernel.
// Measured, 8 sequences of 2048 queries and keys, 32 heads over 8 of 128 (16 over 16 of 64): 1221 us, 1126 TFLOP/s
// (532 us, 646); with a bias 1650 (680); with dropout 1841 (804); with both 2304 (1050).  Issue slots are 40 %
// taken: the bound is the chain S -> P -> dS -> dQ, dK of one tile at a time, which a bias (loads, one more add a
// score, sums) and dropout (the generator, masks) lengthen; head_dim 64 has the same chain for half the products.
// Tried for head_dim 64 and not kept: dP of the next tile in front of dQ and dK, with dQ's own columns and two
// places each for dO and dS (532 -> 595 us: dQ and dK come later, and with them the read-out that the next tile waits for).
#include <cuda_bf16.h>

#include <atomic>

#include "cross.h"
#include "device_util.cuh"
#include "philox.cuh"
#include "tc_util.cuh"
#include "tmap.h"

namespace cpattn {

namespace {

constexpr uint32_t kHalfBytes = 128 * 128;  // 64 columns of 128 rows

struct Params {
  CUtensorMap tmq, tmk, tmv, tmdo, tmdq;
  CrossBwd a;
};

__device__ __forceinline__ void store_row_bf16(__nv_bfloat16* dst, const uint32_t* r, float mul) {
#pragma unroll
  for (int q4 = 0; q4 < 4; ++q4) {
    uint4 v;
    v.x = tc::pack_bf16x2(__uint_as_float(r[8 * q4 + 0]) * mul, __uint_as_float(r[8 * q4 + 1]) * mul);
    v.y = tc::pack_bf16x2(__uint_as_float(r[8 * q4 + 2]) * mul, __uint_as_float(r[8 * q4 + 3]) * mul);
    v.z = tc::pack_bf16x2(__uint_as_float(r[8 * q4 + 4]) * mul, __uint_as_float(r[8 * q4 + 5]) * mul);
    v.w = tc::pack_bf16x2(__uint_as_float(r[8 * q4 + 6]) * mul, __uint_as_float(r[8 * q4 + 7]) * mul);
    *reinterpret_cast<uint4*>(dst + q4 * 8) = v;
  }
}

// A value the compiler has to take as computed here (descriptors of a product's steps by one add each).
__device__ __forceinline__ uint64_t opaque(uint64_t x) {
  asm volatile("" : "+l"(x));
  return x;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// Of 8 lanes every one has drawn for one query and 8 keys, and wants the bytes (0 or 255) of its own key and all 8
// queries: an 8 x 8 transpose of bytes in three exchanges.  (Bits gathered in a byte, fetched
// lane by lane and spread again took twice the instructions.)
struct KeepTurn {
  uint32_t send2, low2, high2, send1, low1, high1;  // byte selectors of the second and third exchange
  bool upper;
  __device__ __forceinline__ explicit KeepTurn(int lane) {
    upper = lane & 4;
    const bool b = lane & 2, c = lane & 1;
    send2 = b ? 0x5410u : 0x7632u;
    low2 = b ? 0x3254u : 0x5410u;
    high2 = b ? 0x3276u : 0x7610u;
    send1 = c ? 0x6420u : 0x7531u;
    low1 = c ? 0x3514u : 0x5240u;
    high1 = c ? 0x3716u : 0x7260u;
  }
  // out: queries 0 .. 3 and 4 .. 7
  __device__ __forceinline__ void go(const Draw& d, uint32_t add, uint32_t* out) const {
    const uint32_t k0 = prmt(keep_halves(d.w[0], add), keep_halves(d.w[1], add), 0xFDB9u);  // keys 0 .. 3 of this query
    const uint32_t k4 = prmt(keep_halves(d.w[2], add), keep_halves(d.w[3], add), 0xFDB9u);
    uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? k0 : k4, 4);
    const uint32_t x = upper ? got : k0, y = upper ? k4 : got;  // queries (lane & 3) and 4 further, this half's 4 keys
    got = __shfl_xor_sync(0xffffffffu, prmt(x, y, send2), 2);
    const uint32_t x2 = prmt(x, got, low2), y2 = prmt(y, got, high2);
    got = __shfl_xor_sync(0xffffffffu, prmt(x2, y2, send1), 1);
    out[0] = prmt(x2, got, low1);
    out[1] = prmt(y2, got, high1);
  }
};

constexpr int kThreads = 512;
constexpr int kLaunchRegs = 128;  // per thread at launch (65536 / 512)
constexpr int kSmallRegs = 72;    // warpgroup 0
// warpgroups 1, 2 (key-row math) and 3 (dQ read-out, D columns a thread)
template <int D>
constexpr int kMathRegs = D == 128 ? 144 : 152;
template <int D>
constexpr int kDqRegs = D == 128 ? 152 : 136;
static_assert(128 * (kSmallRegs + kDqRegs<128>) + 256 * kMathRegs<128> == kThreads * kLaunchRegs &&
                  128 * (kSmallRegs + kDqRegs<64>) + 256 * kMathRegs<64> == kThreads * kLaunchRegs,
              "setmaxnreg shares must add up to the launch allocation");

template <int D>
struct Smem {
  static constexpr int kTile = 128 * D * 2;         // a tile of 128 rows
  static constexpr int kDqChunk = 128 * 32 * 4;     // float32, 32 columns x 128 rows
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kOffK + kTile;
  static constexpr int kOffQ = kOffV + kTile;       // 2 stages
  static constexpr int kOffDO = kOffQ + 2 * kTile;  // 1 stage
  static constexpr int kOffDQ = kOffDO + kTile;     // 2 dQ staging chunks
  static constexpr int kOffDS = kOffDQ + 2 * kDqChunk;
  static constexpr int kOffL = kOffDS + 128 * 128 * 2;  // 2 stages x 128 floats
  static constexpr int kOffD = kOffL + 2 * 512;
  static constexpr int kOffBar = kOffD + 2 * 512;
  static constexpr int kBytes = kOffBar + 256;
  static_assert(kBytes <= 232448, "shared memory budget of one CTA");
};

enum {
  B_KVFULL = 0, B_KVEMPTY, B_QFULL0, B_QFULL1, B_QEMPTY0, B_QEMPTY1, B_DOFULL, B_DOEMPTY, B_SFULL, B_DPFULL, B_PFULL,
  B_PCONS, B_DSFULL, B_DKDV, B_LDFULL0, B_LDFULL1, B_LDEMPTY0, B_LDEMPTY1, B_DQFULL, B_DQCONS, B_DRAIN,
  B_KCUT, B_QCUT0, B_QCUT1, B_DOCUT,  // the bytes of a tile that warp 3 has to clear the end of
  B_COUNT
};
static_assert(8 * B_COUNT + 8 <= 256, "barrier area");

struct Item {
  int32_t seq, first, id, g;
  int32_t krow, len;          // first key row, keys
  int32_t off;                // position of query 0
  int32_t q0, nq, qlo, nqt;   // first query row, queries, first query that sees a key, query tiles of a head
  int32_t n_tiles;
  int32_t k_cut;              // rows of other owners follow inside the key tile
};

__device__ __forceinline__ Item load_item(const CrossBwd& a, int64_t w) {
  Item it;
  const int64_t e = w / a.Hkv;
  it.g = int(w - e * a.Hkv);
  const CrossTile t = a.k_tiles.list[e];
  it.seq = t.seq;
  it.first = t.first;
  it.id = t.id;
  const PagedReq q = paged_req(a, t.seq);
  it.krow = paged_key_row(a, t.seq) + t.first;
  it.len = min(kTile, q.kv - t.first);
  it.off = q.kv - q.nq;
  it.q0 = q.q0;
  it.nq = q.nq;
  it.qlo = cross_first_query(a, q, t.first);
  it.nqt = (q.nq - it.qlo + kTile - 1) / kTile;
  it.n_tiles = it.nqt * a.G;
  it.k_cut = it.len < kTile && it.krow + it.len < a.rows_k;
  return it;
}

// The query tiles of an item in order: q-head of the group, 128 rows.
struct QTile {
  int32_t h, i0, len, row, cut;  // head, first query, queries, first row; rows of other owners follow inside the tile
};
struct Walk {
  int32_t hj, u;
  __device__ __forceinline__ Walk() : hj(0), u(0) {}
  __device__ __forceinline__ void next(const Item& it) {
    if (++u == it.nqt) {
      u = 0;
      ++hj;
    }
  }
  __device__ __forceinline__ QTile tile(const CrossBwd& a, const Item& it) const {
    QTile t;
    t.h = it.g * a.G + hj;
    t.i0 = it.qlo + u * kTile;
    t.len = min(kTile, it.nq - t.i0);
    t.row = it.q0 + t.i0;
    t.cut = t.len < kTile && t.row + t.len < a.rows;
    return t;
  }
};

// Items of this block: rounds over the list in turns from either end, so that the
// costly ones of a round fall to those that had the cheap ones before.  (A round's items lie side by side, so a block
// that has none in a round has none in the next.)
struct Share {
  int64_t n, k;
  __device__ __forceinline__ explicit Share(const CrossBwd& a) : n(int64_t(*a.k_tiles.count) * a.Hkv), k(0) {}
  __device__ __forceinline__ bool next(int64_t* w) {
    const int64_t c = (k & 1) ? int64_t(gridDim.x) - 1 - blockIdx.x : blockIdx.x;
    *w = k * gridDim.x + c;
    ++k;
    return *w < n;
  }
};

// Adds the sums of 32 relative positions from d0 on (one a lane) to the buckets (lane b: b and b + 32).
// The lanes sum within their bucket's run only: a difference of sums over all would
// leave its rounding in buckets that hold nothing.
__device__ __forceinline__ void add_window(const CrossBwd& a, float x, int d0, int lane, float* acc) {
  int n1[kMaxBuckets / 32];  // behind the last lane of the bucket; 0: none of them
  uint32_t begins = 0;       // lanes where a bucket begins
#pragma unroll
  for (int k = 0; k < kMaxBuckets / 32; ++k) {
    n1[k] = 0;
    if (lane + 32 * k < a.buckets) {
      int lo, hi;
      rel_range(a.starts, lane + 32 * k, &lo, &hi);
      const int n0 = max(lo - d0, 0), n = min(hi - d0, 31) + 1;
      if (n > n0) {
        n1[k] = n;
        begins |= 1u << n0;
      }
    }
  }
  begins = __reduce_or_sync(0xffffffffu, begins);
  const int begin = 31 - __clz(begins & (0xffffffffu >> (31 - lane)));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane - o >= begin) x += y;
  }
#pragma unroll
  for (int k = 0; k < kMaxBuckets / 32; ++k) {
    if (32 * k >= a.buckets) break;
    const float sum = __shfl_sync(0xffffffffu, x, max(n1[k] - 1, 0));
    if (n1[k] > 0) acc[k] += sum;
  }
}

template <int D, bool kBias, bool kDrop>
__global__ void __launch_bounds__(kThreads, 1) cross_bwd_kernel(const __grid_constant__ Params p) {
  using M = Smem<D>;
  constexpr uint32_t kIdescKK = tc::idesc_bf16(128, 128, 0, 0);  // A, B K-major
  constexpr uint32_t kIdescKM = tc::idesc_bf16(128, D, 1, 0);    // B MN-major
  constexpr uint32_t kIdescMM = tc::idesc_bf16(128, D, 1, 1);    // A and B MN-major
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = tc::smem_u32(smem);
  const CrossBwd& a = p.a;
  if (sbase & 1023) {  // swizzled operand layouts need a 1 KB aligned base
    if (threadIdx.x == 0 && a.err) atomicCAS(a.err, 0, 2);
    return;
  }
  const uint32_t sK = sbase + M::kOffK, sV = sbase + M::kOffV, sQ = sbase + M::kOffQ, sDO = sbase + M::kOffDO,
                 sDQ = sbase + M::kOffDQ, sDS = sbase + M::kOffDS;
  float* sL = reinterpret_cast<float*>(smem + M::kOffL);
  float* sD = reinterpret_cast<float*>(smem + M::kOffD);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + M::kOffBar);
  auto bar = [&](int i) { return tc::smem_u32(bars + i); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + M::kOffBar + 8 * B_COUNT);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + M::kOffBar + 8 * B_COUNT + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto wt = [&](int b, uint32_t parity) -> bool { return tc::mbar_wait(bar(b), parity, abort_flag, a.err); };
  auto wt_all = [&](int b, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wt(b, parity)); };

  if (const int i = threadIdx.x; i < B_COUNT) {
    uint32_t cnt = 1;
    if (i == B_PFULL || i == B_DSFULL || i == B_LDEMPTY0 || i == B_LDEMPTY1) cnt = 256;
    if (i == B_DQCONS) cnt = 128;
    if (i == B_LDFULL0 || i == B_LDFULL1) cnt = 32;
    tc::mbar_init(bar(i), cnt);
    tc::fence_mbar_init();
  }
  if (threadIdx.x == 0) *abort_flag = 0;
  if (warp == 1) {
    tc::tmem_alloc(tc::smem_u32(tmem_slot), 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS = tmem, tDP = tmem + 128, tDV = tmem + 256, tDK = tmem + 384;
  Share share(a);
  int64_t w;

  if (warp < 4) {
    tc::setmaxnreg_dec<kSmallRegs>();
  }
  if (warp == 0) {
    // ------------------------------------------------------ TMA producer --
    if (lane == 0) {
      tc::prefetch_tmap(&p.tmq);
      tc::prefetch_tmap(&p.tmk);
      tc::prefetch_tmap(&p.tmv);
      tc::prefetch_tmap(&p.tmdo);
      uint32_t gt = 0, ni = 0;
      bool ok = true;
      auto load_tile = [&](uint32_t dst, const CUtensorMap* map, int b, int head, int row) {
        tc::tma_load_3d(dst, map, bar(b), 0, head, row);
        if (D == 128) tc::tma_load_3d(dst + kHalfBytes, map, bar(b), 64, head, row);
      };
      // phases that were armed, for the drain
      uint32_t used_k = 0, used_kc = 0, used_q0 = 0, used_q1 = 0, used_qc0 = 0, used_qc1 = 0, used_do = 0, used_doc = 0;
      while (ok && share.next(&w)) {
        const Item it = load_item(a, w);
        if (it.n_tiles == 0) continue;
        ok = wt(B_KVEMPTY, (ni & 1) ^ 1);
        ++ni;
        if (!ok) break;
        // V's rows behind the end reach rows of dP^T that are masked only
        const int kb = it.k_cut ? B_KCUT : B_KVFULL;
        tc::mbar_arrive_expect_tx(bar(kb), 2 * M::kTile);
        load_tile(sK, &p.tmk, kb, it.g, it.krow);
        load_tile(sV, &p.tmv, kb, it.g, it.krow);
        ++used_k;
        if (it.k_cut) ++used_kc;
        Walk wk;
        for (int t = 0; t < it.n_tiles && ok; ++t, ++gt, wk.next(it)) {
          const QTile qt = wk.tile(a, it);
          const uint32_t st = gt & 1, ph = (gt >> 1) & 1;
          ok = wt(B_QEMPTY0 + int(st), ph ^ 1);
          if (!ok) break;
          const int qb = (qt.cut ? B_QCUT0 : B_QFULL0) + int(st);
          tc::mbar_arrive_expect_tx(bar(qb), M::kTile);
          load_tile(sQ + st * M::kTile, &p.tmq, qb, qt.h, qt.row);
          if (st) {
            ++used_q1;
            if (qt.cut) ++used_qc1;
          } else {
            ++used_q0;
            if (qt.cut) ++used_qc0;
          }
          // one dO stage: dO(t) once dV(t-1) and dP(t-1) have read dO(t-1)
          ok = wt(B_DOEMPTY, (gt & 1) ^ 1);
          if (!ok) break;
          const int db = qt.cut ? B_DOCUT : B_DOFULL;
          tc::mbar_arrive_expect_tx(bar(db), M::kTile);
          load_tile(sDO, &p.tmdo, db, qt.h, qt.row);
          ++used_do;
          if (qt.cut) ++used_doc;
        }
      }
      // Drain: every copy has landed before the block exits.  (A cut tile's FULL phase is completed
      // by warp 3; where that gave up, its CUT phase is what counts, and the default budget passes.)
      volatile int never = 0;
      auto drain = [&](int b, uint32_t used) {
        if (used) tc::mbar_wait(bar(b), (used - 1) & 1, &never, nullptr);
      };
      drain(B_DOCUT, used_doc);
      drain(B_QCUT1, used_qc1);
      drain(B_QCUT0, used_qc0);
      drain(B_KCUT, used_kc);
      drain(B_DOFULL, used_do);
      drain(B_QFULL1, used_q1);
      drain(B_QFULL0, used_q0);
      drain(B_KVFULL, used_k);
    }
  } else if (warp == 1) {
    // -------------------------------------------------------- MMA issuer --
    if (lane == 0) {
      uint32_t gt = 0, ni = 0;
      bool ok = true;
      auto issue_s = [&](uint32_t g) {  // S^T = K Q^T
        const uint64_t a0 = opaque(tc::kmajor_desc(sK)), b0 = opaque(tc::kmajor_desc(sQ + (g & 1) * M::kTile));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc::mma_ss(tS, tc::kmajor_step(a0, kk), tc::kmajor_step(b0, kk), kIdescKK, kk > 0);
        tc::mma_commit(bar(B_SFULL));
      };
      auto issue_dp = [&]() {  // dP^T = V dO^T
        const uint64_t a0 = opaque(tc::kmajor_desc(sV)), b0 = opaque(tc::kmajor_desc(sDO));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc::mma_ss(tDP, tc::kmajor_step(a0, kk), tc::kmajor_step(b0, kk), kIdescKK, kk > 0);
        tc::mma_commit(bar(B_DPFULL));
      };
      while (ok && share.next(&w)) {
        const Item it = load_item(a, w);
        if (it.n_tiles == 0) continue;
        ok = wt(B_KVFULL, ni & 1);
        ++ni;
        // S of the item's first tile once dV of the previous tile has read P^T
        if (ok) ok = wt(B_QFULL0 + int(gt & 1), (gt >> 1) & 1);
        if (ok && gt > 0) ok = wt(B_PCONS, (gt - 1) & 1);
        if (!ok) break;
        tc::fence_after_sync();
        issue_s(gt);
        for (int t = 0; t < it.n_tiles && ok; ++t, ++gt) {
          const uint32_t st = gt & 1;
          const bool has_next = t + 1 < it.n_tiles;
          // dP^T into the columns of the previous tile's dQ once it is read
          // out: it needs no P, so it runs while the math warps build P^T
          ok = wt(B_DOFULL, gt & 1);
          if (ok && gt > 0) ok = wt(B_DQCONS, (gt - 1) & 1);
          if (!ok) break;
          tc::fence_after_sync();
          issue_dp();
          ok = wt(B_PFULL, gt & 1);
          if (!ok) break;
          tc::fence_after_sync();
          const uint64_t bv = opaque(tc::mnmajor_desc(sDO));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // dV += P^T dO, P^T from TMEM
            tc::mma_ts(tDV, tS + (kk >> 2) * 64 + (kk & 3) * 8, tc::mnmajor_step(bv, kk), kIdescKM,
                       (t > 0 || kk > 0) ? 1u : 0u);
          tc::mma_commit(bar(B_PCONS));
          tc::mma_commit(bar(B_DOEMPTY));  // dP and dV have read dO
          if (has_next) {  // S of the next tile once dV has read P^T
            ok = wt(B_QFULL0 + int(st ^ 1), ((gt + 1) >> 1) & 1) && wt(B_PCONS, gt & 1);
            if (!ok) break;
            tc::fence_after_sync();
            issue_s(gt + 1);
          }
          ok = wt(B_DSFULL, gt & 1);
          if (!ok) break;
          tc::fence_after_sync();
          // dQ first: its read-out (which frees the dP^T columns for the next
          // tile's dP) overlaps dK on the tensor core
          const uint64_t aq = opaque(tc::mnmajor_desc(sDS)), bq = opaque(tc::mnmajor_desc(sK));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // dQ_t = dS K over the dP^T columns (read out by the dQ warps)
            tc::mma_ss(tDP, tc::mnmajor_step(aq, kk), tc::mnmajor_step(bq, kk), kIdescMM, kk > 0 ? 1u : 0u);
          tc::mma_commit(bar(B_DQFULL));
          const uint64_t ak = opaque(tc::kmajor_desc(sDS)), bk = opaque(tc::mnmajor_desc(sQ + st * M::kTile));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // dK += dS^T Q
            tc::mma_ss(tDK, tc::kmajor_step(ak, kk), tc::mnmajor_step(bk, kk), kIdescKM, (t > 0 || kk > 0) ? 1u : 0u);
          tc::mma_commit(bar(B_QEMPTY0 + int(st)));
          if (!has_next) {
            tc::mma_commit(bar(B_KVEMPTY));
            tc::mma_commit(bar(B_DKDV));
          }
        }
      }
      volatile int never = 0;
      tc::mma_commit(bar(B_DRAIN));
      tc::mbar_wait(bar(B_DRAIN), 0, &never, nullptr);
    }
  } else if (warp == 2) {
    // ---------------------------------------------- L and D staging warp --
    uint32_t gt = 0;
    bool ok = true;
    while (ok && share.next(&w)) {
      const Item it = load_item(a, w);
      Walk wk;
      for (int t = 0; t < it.n_tiles && ok; ++t, ++gt, wk.next(it)) {
        const QTile qt = wk.tile(a, it);
        const uint32_t st = gt & 1;
        const int64_t base = int64_t(qt.h) * a.rows + qt.row;
        float l4[4], d4[4];
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
          const int q = lane + 32 * k4;
          const bool v = q < qt.len;
          l4[k4] = v ? -a.lse2[base + q] : -INFINITY;  // -L2: exp2(S sl2 - L2) = 0 past the tile
          d4[k4] = v ? -a.delta[base + q] : 0.f;
        }
        ok = wt_all(B_LDEMPTY0 + int(st), ((gt >> 1) & 1) ^ 1);
        if (!ok) break;
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
          sL[st * 128 + lane + 32 * k4] = l4[k4];
          sD[st * 128 + lane + 32 * k4] = d4[k4];
        }
        tc::mbar_arrive(bar(B_LDFULL0 + int(st)));
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------ ends of the cut tiles --
    uint32_t gt = 0, nk = 0, nq0 = 0, nq1 = 0, ndo = 0;
    bool ok = true;
    auto clear = [&](uint32_t tile, int len) {  // rows len .. 127 of a tile, the whole warp
      for (int e = lane; e < (kTile - len) * (D / 8); e += 32) {
        const int row = len + e / (D / 8), c = e % (D / 8);
        *reinterpret_cast<uint4*>(smem + (tile - sbase) + (c >> 3) * kHalfBytes + row * 128 + ((c & 7) << 4)) =
            make_uint4(0, 0, 0, 0);
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
    };
    while (ok && share.next(&w)) {
      const Item it = load_item(a, w);
      if (it.n_tiles == 0) continue;
      if (it.k_cut) {
        ok = wt_all(B_KCUT, nk & 1);
        ++nk;
        if (!ok) break;
        clear(sK, it.len);
        if (lane == 0) tc::mbar_arrive(bar(B_KVFULL));
      }
      Walk wk;
      for (int t = 0; t < it.n_tiles && ok; ++t, ++gt, wk.next(it)) {
        const QTile qt = wk.tile(a, it);
        if (!qt.cut) continue;
        const uint32_t st = gt & 1;
        ok = wt_all(B_QCUT0 + int(st), (st ? nq1 : nq0) & 1);
        if (!ok) break;
        if (st)
          ++nq1;
        else
          ++nq0;
        clear(sQ + st * M::kTile, qt.len);
        if (lane == 0) tc::mbar_arrive(bar(B_QFULL0 + int(st)));
        ok = wt_all(B_DOCUT, ndo & 1);
        ++ndo;
        if (!ok) break;
        clear(sDO, qt.len);
        if (lane == 0) tc::mbar_arrive(bar(B_DOFULL));
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------- key-row math warps --
    // Eight warps, two per TMEM lane quarter: warp w serves key rows
    // 32 (w % 4) .. +31 and query columns 64 h .. 64 h + 63, h = (w - 4) / 4.
    tc::setmaxnreg_inc<kMathRegs<D>>();
    const int quarter = warp & 3;
    const int half = (warp - 4) >> 2;
    const int j = quarter * 32 + lane;  // key row of the tile = TMEM lane
    const uint32_t lane_off = uint32_t(quarter * 32) << 16;
    const uint64_t sl2x2 = tc::f32x2(a.scale_log2, a.scale_log2);
    DropKeys dkey{};
    if (kDrop) dkey = drop_keys(drop_key(a.rng, a.drop_min));
    const KeepTurn turn(lane);
    uint32_t gt = 0, ni = 0;
    bool ok = true;
    while (ok && share.next(&w)) {
      const Item it = load_item(a, w);
      const bool kvalid = j < it.len;
      const int kpos = it.first + j;
      float acc[kMaxBuckets / 32] = {}, back = 0.f, fore = 0.f;  // the table's gradient of a head
      Walk wk;
      for (int t = 0; t < it.n_tiles && ok; ++t, ++gt, wk.next(it)) {
        const QTile qt = wk.tile(a, it);
        const uint32_t st = gt & 1;
        const int qpos0 = qt.i0 + it.off;
        // byte masks of the 64 queries: keep[i / 8][i % 8 / 4], byte i % 4
        uint32_t keep[8][2] = {};
        if constexpr (kDrop) {
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const Draw dr = draw(dkey, uint32_t(kpos) >> 3, uint32_t(qt.i0 + 64 * half + 8 * u + (lane & 7)),
                                 uint32_t(it.seq) * uint32_t(a.H) + uint32_t(qt.h));
            turn.go(dr, dkey.add, keep[u]);
          }
        }
        // the mask of queries i, i + 1 of this warp's 64 as two 16-bit halves, and of one query as a word
        auto keep_pair = [&](int i) {
          const uint32_t r = keep[i >> 3][(i >> 2) & 1], u = uint32_t(i) & 3u;
          return prmt(r, r, u * 0x11u + (u + 1) * 0x1100u);
        };
        auto keep_word = [&](int i) {
          const uint32_t r = keep[i >> 3][(i >> 2) & 1];
          return prmt(r, r, (uint32_t(i) & 3u) * 0x1111u);
        };
        // the bias: query i of the 64 lies at relative position x0 - i; `top` is the largest of
        // the warp, the smallest is 94 below
        const int x0 = kpos - qpos0 - 64 * half;
        const int top = it.first + quarter * 32 + 31 - qpos0 - 64 * half;
        bool near = false;
        float add = 0.f;
        const float* rel = nullptr;
        if (kBias) {
          rel = a.rel + int64_t(qt.h) * a.rel_stride + a.rel_zero;
          near = top > -a.reach && top - 94 < a.reach;
          if (!near) add = rel[top <= -a.reach ? -a.reach : a.reach];
        }
        ok = wt_all(B_LDFULL0 + int(st), (gt >> 1) & 1) && wt_all(B_SFULL, gt & 1);
        if (!ok) break;
        tc::fence_after_sync();
        // visible queries: i_lo <= i < i_hi
        int i_lo = a.causal ? max(0, kpos - qpos0) : 0;
        if (!kvalid) i_lo = kTile;
        const int i_hi = qt.len;
        const bool open = __all_sync(0xffffffffu, i_lo <= half * 64 && i_hi >= half * 64 + 64);  // no masking
        const uint32_t i_span = uint32_t(max(i_hi - i_lo, 0));
        auto seen = [&](int i) { return uint32_t(half * 64 + i - i_lo) < i_span; };
        const float4* L4 = reinterpret_cast<const float4*>(sL + st * 128 + half * 64);  // -L2
        const float4* D4 = reinterpret_cast<const float4*>(sD + st * 128 + half * 64);  // -D / r
        // scores, then P in float32 (dQ and dK are off by 0.0030 of their norm with a rounded P in dS, by 0.0024
        // so), then, with a bias, dS; and bf16 pairs of 32 of P, then of dS
        uint32_t sr[64], pk[32];
        tc::tmem_ld32(tS + lane_off + half * 64, sr);
        tc::tmem_ld32(tS + lane_off + half * 64 + 32, sr + 32);
        tc::tmem_wait_ld();
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {  // P^T = exp2(S^T sl2 - L2); P^T kept in its own half
          if (kBias && near) {
            const float* e = rel + x0 - 32 * cc;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              sr[32 * cc + i] = __float_as_uint(fmaf(__uint_as_float(sr[32 * cc + i]), a.scale_log2, e[-i]));
          }
          const uint64_t mul2 = kBias && near ? tc::f32x2(1.f, 1.f) : sl2x2;
#pragma unroll
          for (int e4 = 0; e4 < 8; ++e4) {
            const float4 l4 = L4[cc * 8 + e4];
            const float lv[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {
              const int i = cc * 32 + e4 * 4 + e2 * 2;
              uint64_t l2 = tc::f32x2(lv[2 * e2], lv[2 * e2 + 1]);
              if (kBias) l2 = tc::fadd2(l2, tc::f32x2(add, add));
              float y0, y1;
              tc::f32x2_split(tc::ffma2(tc::f32x2(__uint_as_float(sr[i]), __uint_as_float(sr[i + 1])), mul2, l2), y0, y1);
              y0 = tc::ex2(y0);
              y1 = tc::ex2(y1);
              if (!open) {  // (an overflowed exponential becomes 0 too)
                y0 = seen(i) ? y0 : 0.f;
                y1 = seen(i + 1) ? y1 : 0.f;
              }
              sr[i] = __float_as_uint(y0);
              sr[i + 1] = __float_as_uint(y1);
              pk[e4 * 2 + e2] = tc::pack_bf16x2(y0, y1);
              if constexpr (kDrop) pk[e4 * 2 + e2] &= keep_pair(i);
            }
          }
          tc::tmem_st16(tS + lane_off + half * 64 + cc * 16, pk);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        tc::mbar_arrive(bar(B_PFULL));
        ok = wt_all(B_DPFULL, gt & 1);
        if (!ok) break;
        tc::fence_after_sync();
        uint64_t sum2 = 0;
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {  // dS^T / r = P^T (keep dP^T - D / r)
          uint32_t dr[32];
          tc::tmem_ld32(tDP + lane_off + half * 64 + cc * 32, dr);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e4 = 0; e4 < 8; ++e4) {
            const float4 d4 = D4[cc * 8 + e4];
            const float dv4[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {
              const int e = e4 * 4 + e2 * 2, i = cc * 32 + e;
              if constexpr (kDrop) {
                dr[e] &= keep_word(i);
                dr[e + 1] &= keep_word(i + 1);
              }
              const uint64_t dd = tc::fadd2(tc::f32x2(__uint_as_float(dr[e]), __uint_as_float(dr[e + 1])),
                                            tc::f32x2(dv4[2 * e2], dv4[2 * e2 + 1]));
              float d0, d1;
              tc::f32x2_split(tc::fmul2(tc::f32x2(__uint_as_float(sr[i]), __uint_as_float(sr[i + 1])), dd), d0, d1);
              if (!open) {  // 0 times what a row behind the end holds
                d0 = seen(i) ? d0 : 0.f;
                d1 = seen(i + 1) ? d1 : 0.f;
              }
              if (kBias) {
                sr[i] = __float_as_uint(d0);
                sr[i + 1] = __float_as_uint(d1);
                sum2 = tc::fadd2(sum2, tc::f32x2(d0, d1));
              }
              pk[i / 2] = tc::pack_bf16x2(d0, d1);
            }
          }
        }
        tc::fence_before_sync();
        tc::mbar_arrive(bar(B_LDEMPTY0 + int(st)));
        // dK and dQ of the previous tile (issued before this dP) have read the old dS^T;
        // this warp writes its 64 query columns = one 128-byte swizzle region
        uint8_t* drow = smem + M::kOffDS + half * kHalfBytes + j * 128;
#pragma unroll
        for (int kc = 0; kc < 8; ++kc)
          *reinterpret_cast<uint4*>(drow + ((kc ^ (j & 7)) << 4)) =
              make_uint4(pk[4 * kc], pk[4 * kc + 1], pk[4 * kc + 2], pk[4 * kc + 3]);
        tc::fence_proxy_async_smem();
        tc::fence_before_sync();
        tc::mbar_arrive(bar(B_DSFULL));
        if constexpr (kBias) {
          // the table's gradient, while the products of this tile run
          if (!near) {
            float s0, s1;
            tc::f32x2_split(sum2, s0, s1);
            if (top <= -a.reach)
              back += s0 + s1;
            else
              fore += s0 + s1;
          } else {
            const float up_on = lane == 0 ? 0.f : 1.f, down_on = lane == 31 ? 0.f : 1.f;
            float dn[2] = {}, up[2] = {};
#pragma unroll
            for (int i = 0; i < 32; ++i) {
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                dn[c] = fmaf(__shfl_down_sync(0xffffffffu, dn[c], 1), down_on, __uint_as_float(sr[32 * c + 31 - i]));
                up[c] = fmaf(__shfl_up_sync(0xffffffffu, up[c], 1), up_on, __uint_as_float(sr[32 * c + i]));
              }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) up[c] = __shfl_up_sync(0xffffffffu, up[c], 1) * up_on;
            const int d0 = it.first + quarter * 32 - qpos0 - 64 * half;  // of lane 0 and the first column
            add_window(a, dn[0], d0, lane, acc);
            add_window(a, up[0] + dn[1], d0 - 32, lane, acc);
            add_window(a, up[1], d0 - 64, lane, acc);
          }
          if (wk.u == it.nqt - 1) {  // the head's last query tile
            back = warp_sum(back);
            fore = warp_sum(fore);
            const int last = a.starts.per - 1, ahead = a.starts.both ? 2 * a.starts.per - 1 : 0;
            float* to = a.part + ((int64_t(it.id) * a.H + qt.h) * 8 + (warp - 4)) * a.bucket_stride;
#pragma unroll
            for (int k = 0; k < kMaxBuckets / 32; ++k) {
              const int b = lane + 32 * k;
              if (b < a.bucket_stride) to[b] = acc[k] + (b == last ? back : 0.f) + (b == ahead ? fore : 0.f);
              acc[k] = 0.f;
            }
            back = fore = 0.f;
          }
        }
      }
      if (!ok) break;
      if (it.n_tiles > 0) {
        ok = wt_all(B_DKDV, ni & 1);
        ++ni;
        if (!ok) break;
        tc::fence_after_sync();
      } else if (kBias) {
        for (int hj = 0; hj < a.G; ++hj)
          for (int b = lane; b < a.bucket_stride; b += 32)
            a.part[((int64_t(it.id) * a.H + it.g * a.G + hj) * 8 + (warp - 4)) * a.bucket_stride + b] = 0.f;
      }
      // item epilogue: half 0 writes r dV, half 1 writes scale r dK of this key row
      const uint32_t tsrc = half == 0 ? tDV : tDK;
      const float mul = half == 0 ? a.drop_scale : a.scale * a.drop_scale;
      __nv_bfloat16* dst =
          static_cast<__nv_bfloat16*>(half == 0 ? a.dv : a.dk) + (int64_t(it.krow + j) * a.Hkv + it.g) * D;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t r[32];
        if (it.n_tiles > 0) {
          tc::tmem_ld32(tsrc + lane_off + c * 32, r);
          tc::tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) r[e] = 0u;
        }
        if (kvalid) store_row_bf16(dst + c * 32, r, mul);
      }
      tc::fence_before_sync();
    }
  } else {
    // --------------------------------------------- dQ read-out warps --
    // Warp w reads TMEM lane quarter w % 4 = query rows 32 (w % 4) .. +31 of
    // the tile, all D dQ columns, and hands the columns back for the next
    // dP^T.  The four warps then stage the tile in 32-column chunks (two
    // staging buffers) and one thread adds each chunk into the accumulator
    // with a TMA reduction.  Rows behind the sequence's end add zeros.
    tc::setmaxnreg_inc<kDqRegs<D>>();
    const int quarter = warp & 3;
    const int i = quarter * 32 + lane;  // query row of the tile = TMEM lane
    const uint32_t lane_off = uint32_t(quarter * 32) << 16;
    const bool leader = warp == 12 && lane == 0;
    if (leader) tc::prefetch_tmap(&p.tmdq);
    uint32_t gt = 0, nchunk = 0;
    bool ok = true;
    while (ok && share.next(&w)) {
      const Item it = load_item(a, w);
      Walk wk;
      for (int t = 0; t < it.n_tiles && ok; ++t, ++gt, wk.next(it)) {
        const QTile qt = wk.tile(a, it);
        ok = wt_all(B_DQFULL, gt & 1);
        ok = tc::named_bar_all(1, 128, ok);
        if (!ok) break;
        tc::fence_after_sync();
        uint32_t r[D];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) tc::tmem_ld32(tDP + lane_off + c * 32, r + c * 32);
        tc::tmem_wait_ld();
        tc::fence_before_sync();
        tc::mbar_arrive(bar(B_DQCONS));
        if (i >= qt.len) {
#pragma unroll
          for (int e = 0; e < D; ++e) r[e] = 0u;
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c, ++nchunk) {
          const uint32_t buf = sDQ + (nchunk & 1) * M::kDqChunk;
          if (leader && nchunk >= 2) tc::bulk_wait_group_read<1>();  // the reduction that last used buf has read it
          tc::named_bar(1, 128);
          // row i: 32 floats = 8 x 16 bytes, 128-byte swizzle (unit k at k ^ (i % 8))
          uint8_t* row = smem + (buf - sbase) + i * 128;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(row + ((k ^ (i & 7)) << 4)) =
                make_uint4(r[32 * c + 4 * k], r[32 * c + 4 * k + 1], r[32 * c + 4 * k + 2], r[32 * c + 4 * k + 3]);
          tc::fence_proxy_async_smem();
          tc::named_bar(1, 128);
          if (leader) {
            tc::tma_reduce_add_3d(&p.tmdq, buf, c * 32, qt.row, qt.h);
            tc::bulk_commit_group();
          }
        }
      }
    }
    if (leader) tc::bulk_wait_group<0>();  // every reduction complete before the block exits
  }

  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) {
    __syncwarp();
    tc::tmem_dealloc(tmem, 512);
  }
}

// [rows][heads][d] of row stride `stride`: a box of 64 columns of 128 rows of one head.
bool make_tmap_tile(CUtensorMap* map, const void* base, int64_t rows, int64_t stride, int heads, int d) {
  auto enc = tmap_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(heads), cuuint64_t(rows)};
  const cuuint64_t strides[2] = {cuuint64_t(d) * 2, cuuint64_t(stride) * 2};
  const cuuint32_t box[3] = {64, 1, 128}, es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [heads][rows][d] of float32: a box of 32 columns of 128 rows, 128-byte swizzle.
bool make_tmap_sums(CUtensorMap* map, void* base, int heads, int64_t rows, int d) {
  auto enc = tmap_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(rows), cuuint64_t(heads)};
  const cuuint64_t strides[2] = {cuuint64_t(d) * 4, cuuint64_t(rows) * cuuint64_t(d) * 4};
  const cuuint32_t box[3] = {32, 128, 1}, es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kBias, bool kDrop>
cp_status run(const CrossBwd& a, cudaStream_t s) {
  auto* kern = cross_bwd_kernel<D, kBias, kDrop>;
  static std::atomic<bool> ready[64] = {};  // per device (an idempotent first set-up)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CP_ERR_CUDA;
  if (!ready[dev].load(std::memory_order_acquire)) {
    // The register hand-over inside the kernel assumes the launch count.
    cudaFuncAttributes fa{};
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return CP_ERR_CUDA;
    if (fa.numRegs != kLaunchRegs) return CP_ERR_UNSUPPORTED;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes) != cudaSuccess)
      return CP_ERR_CUDA;
    ready[dev].store(true, std::memory_order_release);
  }
  Params p;
  if (!make_tmap_tile(&p.tmq, a.q, a.rows, a.q_stride, a.H, D) ||
      !make_tmap_tile(&p.tmk, a.k, a.rows_k, a.k_stride, a.Hkv, D) ||
      !make_tmap_tile(&p.tmv, a.v, a.rows_k, a.v_stride, a.Hkv, D) ||
      !make_tmap_tile(&p.tmdo, a.dout, a.rows, a.do_stride, a.H, D) ||
      !make_tmap_sums(&p.tmdq, a.dq_acc, a.H, a.rows, D))
    return CP_ERR_CUDA;
  p.a = a;
  const int64_t most = int64_t(a.k_tiles.most) * a.Hkv;
  const int64_t grid = most < num_sms() ? most : num_sms();
  kern<<<unsigned(grid), kThreads, Smem<D>::kBytes, s>>>(p);
  return cuda_status(cudaGetLastError());
}

template <int D>
cp_status run_d(const CrossBwd& a, cudaStream_t s) {
  if (a.rel) return a.rng ? run<D, true, true>(a, s) : run<D, true, false>(a, s);
  return a.rng ? run<D, false, true>(a, s) : run<D, false, false>(a, s);
}

}  // namespace

cp_status launch_cross_bwd(const CrossBwd& a, cudaStream_t s) {
  if (a.dtype != CP_BF16) return CP_ERR_UNSUPPORTED;
  return a.d == 128 ? run_d<128>(a, s) : run_d<64>(a, s);
}

}  // namespace cpattn
