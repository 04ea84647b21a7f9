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
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "device_util.cuh"
#include "paged_dev.cuh"
#include "paged_tmap.h"
#include "tc_util.cuh"
#include "tmap.h"

namespace cpattn {

namespace {

template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr int kJoiners = 2;  // with the producers they make the 12 warps that 168 registers allow

// What the rows of a tile need to know of a piece, in shared memory.
struct PieceInfo {
  int32_t valid;
  int32_t q0, row0, nrows, h;  // first row of the request in q, tile rows, kv-head
  int32_t pos0;                // position of the request's first new token
  int32_t kv;
  int32_t key0, n;             // first stage's first key, stages
  int32_t lo, hi;              // keys that some row sees, up to the piece's end
  int32_t full_lo, full_hi;    // keys that every row sees
  int32_t slot;
};

template <int kStageKeys>
__device__ __forceinline__ PieceInfo piece_info(const PagedArgs& a, const PagedPiece& p) {
  PieceInfo i;
  i.valid = 1;
  i.q0 = p.q.q0;
  i.row0 = p.tile.row0;
  i.nrows = p.tile.nrows;
  i.h = p.h;
  i.pos0 = p.q.kv - p.q.nq;
  i.kv = p.q.kv;
  i.key0 = (p.tile.b0 + p.ua) * kSliceUnit;
  const int end = min((p.tile.b0 + p.ub) * kSliceUnit, p.tile.hi);
  i.n = end > i.key0 ? (end - i.key0 + kStageKeys - 1) / kStageKeys : 0;
  i.lo = p.tile.lo;
  i.hi = end;  // the last stage may reach into the next piece's keys
  const int first = i.pos0 + paged_token(a, i.row0), last = i.pos0 + paged_token(a, i.row0 + i.nrows - 1);
  i.full_hi = a.causal ? min(i.kv, first + 1) : i.kv;
  i.full_lo = a.window > 0 ? max(0, last - a.window + 1) : 0;
  i.slot = p.slot;
  return i;
}

// Where a row of a tile goes: the outputs, or its partial state.
template <typename T, int D, int R>
struct SliceOut {
  T* o;         // final O, or
  float* part;  // partial O
  float* lse;
  bool in, whole;
  __device__ __forceinline__ SliceOut(const PagedArgs& a, const PieceInfo& p, int r) {
    in = r < p.nrows;
    whole = p.slot < 0;
    const int x = p.row0 + r;
    const int t = paged_token(a, x);
    const int64_t row = int64_t(p.q0 + t) * a.H + p.h * a.G + (x - t * a.G), prow = int64_t(p.slot) * R + r;
    o = static_cast<T*>(a.o) + row * D;
    part = a.part_o + prow * D;
    lse = whole ? a.lse + row : a.part_l + prow;
  }
  template <int N>
  __device__ __forceinline__ void put(int c, const float* x) const {
    if (!in) return;
    if (whole)
      store_vec<T, N>(o + c, x);
    else
      store_vec<float, N>(part + c, x);
  }
  __device__ __forceinline__ void put_lse(float log2_sum) const {
    if (in) *lse = whole ? log2_sum * 0.69314718055994531f : log2_sum;
  }
};

// ------------------------------------------------- bf16: mma.sync tiles ---
template <int D, int R>
struct SliceBf16 {
  using T = __nv_bfloat16;
  // 32 rows of 128 columns: the states of four workers are what shared memory holds
  static constexpr int kWarps = D * R > 64 * 32 && R > 16 ? 4 : 8;
  // kPerStage: workers of a stage.  Stages of 32 KB: a stage costs a producer as much
  // as several boxes (head_dim 64, pages of 16, contexts of 60000: 105 us with 16 KB, 88)
  static constexpr int kPerStage = D == 128 ? 4 : 8, kKeys = 16, kStages = 4;
  static constexpr int kStageKeys = kPerStage * kKeys;
  static __device__ __forceinline__ int first_key(int warp) { return (warp % kPerStage) * kKeys; }  // a worker's slice of a stage
  static constexpr int MT = R / 16, NT = D / 8;
  static constexpr int kAcc = MT * NT * 4, kRows = MT * 2;  // accumulators and rows of a thread
  static constexpr int kQBytes = R * D * 2;
  static constexpr int kScratch = 0;
  static constexpr int kState = (kAcc / 4 + kRows / 2) * 32;  // float4s of a worker's state
  static constexpr int kPieces = kWarps == 4 ? 3 : 4;  // pieces that the producers are ahead
  static constexpr bool kKeepQ = MT == 1;
  float acc[kAcc];
  float m[kRows], l[kRows];
  uint32_t qf[kKeepQ ? D / 16 : 1][4];
  int32_t lo[kRows], hi[kRows];

  // 16-byte chunk c of row r: of Q, and of a stage (128-byte columns of all its keys, swizzled by TMA)
  static __device__ __forceinline__ uint32_t q_at(int r, int c) { return uint32_t(r * D * 2 + ((c ^ (r & 7)) << 4)); }
  static __device__ __forceinline__ uint32_t at(int r, int c) {
    return uint32_t((c >> 3) * (kStageKeys * 128) + r * 128 + (((c ^ r) & 7) << 4));
  }

  __device__ __forceinline__ void begin(const PagedArgs& a, const PieceInfo& p, uint32_t sq, int, int lane) {
#pragma unroll
    for (int i = 0; i < kAcc; ++i) acc[i] = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      const int pos = p.pos0 + paged_token(a, p.row0 + (lane >> 2) + 8 * i);
      hi[i] = a.causal ? min(p.kv, pos + 1) : p.kv;
      lo[i] = a.window > 0 ? pos - a.window + 1 : 0;
    }
    if constexpr (kKeepQ) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) ldm4(sq + q_at(lane & 15, 2 * k + (lane >> 4)), qf[k]);
    }
  }

  // One slice: the keys from `key` on, in rows `srow` .. of the stage at sk and sv; klo, khi: the tile's keys.
  __device__ __forceinline__ void slice(const PagedArgs& a, uint32_t sq, uint32_t sk, uint32_t sv, int srow, float*,
                                        int key, bool full, int klo, int khi, int lane) {
    float s[MT][2][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][n][e] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t b[4];
      ldm4(sk + at(srow + (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)), b);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        uint32_t f[4];
        if constexpr (kKeepQ) {
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = qf[k][e];
        } else {
          ldm4(sq + q_at(16 * i + (lane & 15), 2 * k + (lane >> 4)), f);
        }
        mma16816(s[i][0], f, b[0], b[1]);
        mma16816(s[i][1], f, b[2], b[3]);
      }
    }
    const int j0 = key + 2 * (lane & 3);
    if (!full) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = j0 + 8 * n + (e & 1), r = 2 * i + (e >> 1);
            s[i][n][e] = j >= lo[r] && j < hi[r] ? s[i][n][e] : -INFINITY;
          }
    }
    float up[kRows];
    bool grow = false;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float* x = s[r >> 1][0] + 2 * (r & 1);
      const float* y = s[r >> 1][1] + 2 * (r & 1);
      float v = fmaxf(fmaxf(x[0], x[1]), fmaxf(y[0], y[1]));
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
      v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
      up[r] = v * a.scale_log2;
      // the maximum moves only when a slice lifts it by more than 2^8: sums
      // stay within float32 and the state is rescaled rarely
      grow |= up[r] > m[r] + 8.f;
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float t = fmaxf(m[r], up[r]);
        const float c = m[r] == -INFINITY ? 0.f : tc::ex2(m[r] - t);
        m[r] = t;
        l[r] *= c;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[((r >> 1) * NT + n) * 4 + 2 * (r & 1)] *= c;
          acc[((r >> 1) * NT + n) * 4 + 2 * (r & 1) + 1] *= c;
        }
      }
    }
    uint32_t p[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 2 * i + h;
        const float base = m[r] == -INFINITY ? 0.f : m[r];
        float e[4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int w = 0; w < 2; ++w) e[2 * n + w] = tc::ex2(fmaf(s[i][n][2 * h + w], a.scale_log2, -base));
        l[r] += (e[0] + e[1]) + (e[2] + e[3]);
        p[i][h] = tc::pack_bf16x2(e[0], e[1]);
        p[i][2 + h] = tc::pack_bf16x2(e[2], e[3]);
      }
    }
    uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;  // this lane's keys of V: j0, j0 + 1 and 8 further
    if (!full) {
      auto in = [&](int j) { return j >= klo && j < khi; };
      keep0 = (in(j0) ? 0xffffu : 0u) | (in(j0 + 1) ? 0xffff0000u : 0u);
      keep1 = (in(j0 + 8) ? 0xffffu : 0u) | (in(j0 + 9) ? 0xffff0000u : 0u);
    }
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
      uint32_t b[4];
      ldm4t(sv + at(srow + (lane & 15), 2 * n + (lane >> 4)), b);
      b[0] &= keep0;
      b[1] &= keep1;
      b[2] &= keep0;
      b[3] &= keep1;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        mma16816(acc + (i * NT + 2 * n) * 4, p[i], b[0], b[1]);
        mma16816(acc + (i * NT + 2 * n + 1) * 4, p[i], b[2], b[3]);
      }
    }
  }

  // The lanes of a row bring their sums together before warps join.
  __device__ __forceinline__ void end() {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
  }

  // A worker's state: float4s [MT][NT / 2][row half][lane] of O (its row lane / 4, or
  // 8 further, in two n-tiles), then m and l of both rows [MT][lane].  Lanes and halves
  // without a row of the tile are left out on both sides: with 4 heads a group three
  // quarters of what would cross shared memory.
  static __device__ __forceinline__ bool any_row(const PieceInfo& p, int i, int lane) {
    return (lane >> 2) + 16 * i < p.nrows;
  }
  static __device__ __forceinline__ bool upper(const PieceInfo& p, int i) { return p.nrows > 16 * i + 8; }

  // Joins the workers' states and writes them out.  Loops stay loops: one warp runs this once per
  // piece, and unrolled it waited for its own instructions (4 to 9 us a piece, 1 us so).
  static __device__ __forceinline__ void join(const PagedArgs& a, const PieceInfo& p, const float4* st, int part,
                                              int lane) {
#pragma unroll 1
    for (int i = 0; i < MT; ++i) {  // this lane's rows 8 * 2 i + lane / 4 and 8 further
      if (!any_row(p, i, lane)) break;
      const SliceOut<T, D, R> out0(a, p, (lane >> 2) + 16 * i), out1(a, p, (lane >> 2) + 16 * i + 8);
      float c0[kWarps], c1[kWarps], t0 = -INFINITY, t1 = -INFINITY, l0 = 0.f, l1 = 0.f;
      float4 x[kWarps];  // m and l of the two rows
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        x[w] = st[w * kState + (kAcc / 4 + i) * 32 + lane];
        t0 = fmaxf(t0, x[w].x);
        t1 = fmaxf(t1, x[w].y);
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        c0[w] = x[w].x == -INFINITY ? 0.f : tc::ex2(x[w].x - t0);
        c1[w] = x[w].y == -INFINITY ? 0.f : tc::ex2(x[w].y - t1);
        l0 = fmaf(x[w].z, c0[w], l0);
        l1 = fmaf(x[w].w, c1[w], l1);
      }
      if (part == 0 && (lane & 3) == 0) {
        out0.put_lse(l0 == 0.f ? -INFINITY : t0 + tc::lg2(l0));
        out1.put_lse(l1 == 0.f ? -INFINITY : t1 + tc::lg2(l1));
      }
      const float v0 = l0 == 0.f ? 0.f : 1.f / l0, v1 = l1 == 0.f ? 0.f : 1.f / l1;
      auto half = [&](const SliceOut<T, D, R>& out, const float* c, float v, int n, const float4* at) {
        float o[4] = {};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 y = at[w * kState];
          o[0] = fmaf(y.x, c[w], o[0]);
          o[1] = fmaf(y.y, c[w], o[1]);
          o[2] = fmaf(y.z, c[w], o[2]);
          o[3] = fmaf(y.w, c[w], o[3]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= v;
        out.template put<2>(16 * n + 2 * (lane & 3), o);
        out.template put<2>(16 * n + 8 + 2 * (lane & 3), o + 2);
      };
#pragma unroll 2
      for (int n = part; n < NT / 2; n += kJoiners) {
        const float4* at = st + ((i * (NT / 2) + n) * 2) * 32 + lane;
        half(out0, c0, v0, n, at);
        if (upper(p, i)) half(out1, c1, v1, n, at + 32);
      }
    }
  }
  __device__ __forceinline__ void leave(const PieceInfo& p, float4* st, int warp, int lane) const {
    float4* x = st + warp * kState + lane;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (!any_row(p, i, lane)) break;
#pragma unroll
      for (int n = 0; n < NT / 2; ++n) {
        const float* y = acc + (i * NT + 2 * n) * 4;
        x[((i * (NT / 2) + n) * 2) * 32] = make_float4(y[0], y[1], y[4], y[5]);
        if (upper(p, i)) x[((i * (NT / 2) + n) * 2 + 1) * 32] = make_float4(y[2], y[3], y[6], y[7]);
      }
      x[(kAcc / 4 + i) * 32] = make_float4(m[2 * i], m[2 * i + 1], l[2 * i], l[2 * i + 1]);
    }
  }
};

// --------------------------------------------------------- float32: FFMA ---
// A stage of 32 keys (64 at head_dim 64 and 16 rows) is one worker's, or two workers' with half of the tile's
// rows each.  First product: a lane owns a key, or two
// (four requests of 100 tokens over 3000, 8 heads over 2, head_dim 64: 112 us, 97 with two: shared memory
// gives a row's Q to twice the products; one request of 3 over 100: 12.1 us, 13.8;
// head_dim 128 has no room for such stages), and the rows of Q come by broadcast, so nothing is summed across lanes and every
// exponential is formed once; P changes hands through shared memory, and in the second product a lane
// owns 4 columns (head_dim 64: of half of the keys).
template <int D, int R>
struct SliceF32 {
  using T = float;
  static constexpr int RW = R < 8 ? R : 8;  // rows of a worker
  static constexpr int KL = D == 64 && R >= 8 ? 2 : 1;  // keys of a lane
  static constexpr int kWarps = R < 8 ? 4 : 8, kPerStage = R / RW, kKeys = 32 * KL, kStages = D == 128 || KL == 2 ? 4 : 8;
  static constexpr int kStageKeys = kKeys;
  static __device__ __forceinline__ int first_key(int) { return 0; }
  static constexpr int kAcc = 4 * RW;
  static constexpr int kQBytes = R * D * 4;
  static constexpr int kScratch = kKeys * RW * 4;  // P of a worker's slice
  static constexpr int kState = RW * 32 + RW / 2;  // float4s of a worker's state; m and l are the same in every lane
  static constexpr int kPieces = 4;                // pieces that the producer is ahead
  uint64_t acc[kAcc / 2];  // [row pair][column] of (row, row + 1): packed float32 pairs, two FMAs an instruction
  float m[RW], l[RW];
  int32_t pos0, row0, kv, first;  // first: this worker's first row of the tile

  static __device__ __forceinline__ uint32_t at(int r, int c) {
    return uint32_t((c >> 3) * (kStageKeys * 128) + r * 128 + (((c ^ r) & 7) << 4));
  }
  static __device__ __forceinline__ uint32_t q_at(int r, int c) { return uint32_t(r * D * 4 + (c << 4)); }
  // P of rows r .. r + 3 for a key, swizzled so that 8 lanes' keys fall on different banks
  static __device__ __forceinline__ float4* p_at(float* sp, int key, int r) {
    return reinterpret_cast<float4*>(sp + key * RW) + (RW == 8 ? (r / 4) ^ ((key >> 2) & 1) : r / 4);
  }
  static __device__ __forceinline__ void lds2(uint32_t addr, uint64_t& lo, uint64_t& hi) {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(lo), "=l"(hi) : "r"(addr) : "memory");
  }

  __device__ __forceinline__ void begin(const PagedArgs&, const PieceInfo& p, uint32_t, int warp, int) {
#pragma unroll
    for (int i = 0; i < kAcc / 2; ++i) acc[i] = 0;
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
    }
    pos0 = p.pos0;
    first = (warp % kPerStage) * RW;
    row0 = p.row0 + first;
    kv = p.kv;
  }

  __device__ __forceinline__ void slice(const PagedArgs& a, uint32_t sq, uint32_t sk, uint32_t sv, int srow, float* sp,
                                        int key, bool full, int klo, int khi, int lane) {
    uint64_t s2[KL][RW];               // sums over even and odd elements of the head
#pragma unroll
    for (int x = 0; x < KL; ++x)
#pragma unroll
      for (int r = 0; r < RW; ++r) s2[x][r] = 0;
#pragma unroll(KL == 2 ? 2 : 4)
    for (int c = 0; c < D / 4; ++c) {
      uint64_t k0[KL], k1[KL];
#pragma unroll
      for (int x = 0; x < KL; ++x) lds2(sk + at(srow + lane + 32 * x, c), k0[x], k1[x]);
      uint64_t q0[RW], q1[RW];
#pragma unroll
      for (int r = 0; r < RW; ++r) lds2(sq + q_at(first + r, c), q0[r], q1[r]);
#pragma unroll
      for (int x = 0; x < KL; ++x) {
#pragma unroll
        for (int r = 0; r < RW; ++r) s2[x][r] = tc::ffma2(q0[r], k0[x], s2[x][r]);
#pragma unroll
        for (int r = 0; r < RW; ++r) s2[x][r] = tc::ffma2(q1[r], k1[x], s2[x][r]);
      }
    }
    float s[KL][RW];
#pragma unroll
    for (int x = 0; x < KL; ++x)
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        float u, w;
        tc::f32x2_split(s2[x][r], u, w);
        s[x][r] = u + w;
      }
    if (!full) {
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        const int pos = pos0 + paged_token(a, row0 + r);
#pragma unroll
        for (int x = 0; x < KL; ++x) {
          const int j = key + lane + 32 * x;
          const bool see = j < kv && (!a.causal || j <= pos) && (a.window == 0 || pos - j < a.window);
          s[x][r] = see ? s[x][r] : -INFINITY;
        }
      }
    }
    float up[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) up[r] = fmaxf(s[0][r], s[KL - 1][r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int r = 0; r < RW; ++r) up[r] = fmaxf(up[r], __shfl_xor_sync(0xffffffffu, up[r], o));
    bool grow = false;
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      up[r] *= a.scale_log2;
      grow |= up[r] > m[r] + 8.f;
    }
    if (grow) {  // the same in every lane
#pragma unroll
      for (int r = 0; r < RW; r += 2) {
        float c[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const float t = fmaxf(m[r + w], up[r + w]);
          c[w] = m[r + w] == -INFINITY ? 0.f : exp2f(m[r + w] - t);
          m[r + w] = t;
          l[r + w] *= c[w];
        }
        const uint64_t c2 = tc::f32x2(c[0], c[1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[2 * r + e] = tc::fmul2(acc[2 * r + e], c2);
      }
    }
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      const float base = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
      for (int x = 0; x < KL; ++x) {
        s[x][r] = exp2f(fmaf(s[x][r], a.scale_log2, -base));
        l[r] += s[x][r];
      }
    }
#pragma unroll
    for (int x = 0; x < KL; ++x)
#pragma unroll
      for (int r = 0; r < RW; r += 4)
        *p_at(sp, lane + 32 * x, r) = make_float4(s[x][r], s[x][r + 1], s[x][r + 2], s[x][r + 3]);
    __syncwarp();
    constexpr int kn = D == 128 ? kKeys : kKeys / 2;
    const int c = D == 128 ? lane : lane & 15, x0 = D == 128 ? 0 : (lane >> 4) * kn;
#pragma unroll 4
    for (int i = 0; i < kn; ++i) {
      const int x = x0 + i;
      uint64_t v0, v1;
      lds2(sv + at(srow + x, c), v0, v1);
      if (!full && (key + x < klo || key + x >= khi)) v0 = v1 = 0;
      float v[4];
      tc::f32x2_split(v0, v[0], v[1]);
      tc::f32x2_split(v1, v[2], v[3]);
      uint64_t vv[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) vv[e] = tc::f32x2(v[e], v[e]);
#pragma unroll
      for (int r = 0; r < RW; r += 4) {
        uint64_t p0, p1;  // rows r, r + 1 and r + 2, r + 3
        lds2(tc::smem_u32(p_at(sp, x, r)), p0, p1);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[2 * r + e] = tc::ffma2(p0, vv[e], acc[2 * r + e]);
          acc[2 * r + 4 + e] = tc::ffma2(p1, vv[e], acc[2 * r + 4 + e]);
        }
      }
    }
  }

  __device__ __forceinline__ void end() {
#pragma unroll
    for (int r = 0; r < RW; ++r) l[r] = warp_sum(l[r]);
    if (D == 64) {
#pragma unroll
      for (int i = 0; i < kAcc / 2; ++i) acc[i] = tc::fadd2(acc[i], __shfl_xor_sync(0xffffffffu, acc[i], 16));
    }
  }

  static __device__ __forceinline__ void join(const PagedArgs& a, const PieceInfo& p, const float4* st, int part,
                                              int lane) {
    constexpr int kAt = D == 128 ? 1 : 2;  // rows at once: a row's columns take 32 lanes or 16
#pragma unroll 1
    for (int i = part * kAt; i < R; i += kJoiners * kAt) {
      const int r = D == 128 ? i : i + (lane >> 4), c = D == 128 ? lane : lane & 15;
      const SliceOut<T, D, R> out(a, p, r);
      constexpr int W = kWarps / kPerStage;  // workers that hold the row: every kPerStage-th
      const int rw = r % RW;
      const float4* base = st + (r / RW) * kState;
      float2 x[W];  // m and l
      float top = -INFINITY, sum = 0.f;
      const float* ml = reinterpret_cast<const float*>(base + RW * 32) + (rw >> 1) * 4 + (rw & 1);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        x[w] = make_float2(ml[w * kPerStage * kState * 4], ml[w * kPerStage * kState * 4 + 2]);
        top = fmaxf(top, x[w].x);
      }
      float o[4] = {};
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = x[w].x == -INFINITY ? 0.f : exp2f(x[w].x - top);
        sum = fmaf(x[w].y, f, sum);
        const float4 y = base[w * kPerStage * kState + rw * 32 + c];
        o[0] = fmaf(y.x, f, o[0]);
        o[1] = fmaf(y.y, f, o[1]);
        o[2] = fmaf(y.z, f, o[2]);
        o[3] = fmaf(y.w, f, o[3]);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] *= inv;
      out.template put<4>(4 * c, o);
      if (c == 0) out.put_lse(sum == 0.f ? -INFINITY : top + log2f(sum));
    }
  }
  __device__ __forceinline__ void leave(const PieceInfo&, float4* st, int warp, int lane) const {
    float4* x = st + warp * kState + lane;
#pragma unroll
    for (int r = 0; r < RW; r += 2) {
      float u[4], w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) tc::f32x2_split(acc[2 * r + e], u[e], w[e]);
      x[r * 32] = make_float4(u[0], u[1], u[2], u[3]);
      x[(r + 1) * 32] = make_float4(w[0], w[1], w[2], w[3]);
    }
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < RW / 2; ++i) x[RW * 32 + i] = make_float4(m[2 * i], m[2 * i + 1], l[2 * i], l[2 * i + 1]);
    }
  }
};

template <typename S, int D, int R>
struct SliceLayout {
  static constexpr int kStageBytes = 2 * S::kStageKeys * D * int(sizeof(typename S::T));
  static constexpr int kOffRing = 0;
  static constexpr int kOffState = kOffRing + S::kStages * kStageBytes;
  static constexpr int kStateBytes = S::kState * 16;  // one worker's
  static constexpr int kOffQ = kOffState + S::kWarps * kStateBytes;
  static constexpr int kQBytes = (S::kQBytes + 127) & ~127;
  static constexpr int kOffP = kOffQ + S::kPieces * kQBytes;
  static constexpr int kBytes = kOffP + S::kWarps * S::kScratch;
  static constexpr int kThreads = (S::kWarps + kJoiners + 2) * 32;
  static_assert(kBytes + 2048 <= 232448, "shared memory of one block");
};

struct SliceParams {
  CUtensorMap tmk, tmv;  // the cache (make_tmap_pages)
  PagedArgs a;
  int32_t box_shift;     // log2 keys of a box
  int32_t head_inner;    // the head dimension comes before the token dimension
  int32_t after_pair;
  long long wait_limit;
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

// kShortWaits: the copy launched while cp_debug_set_wait_limit has set a
// short wait budget; the default copy never reads the limit.
template <typename S, int D, int R, bool kShortWaits>
__global__ void __launch_bounds__(SliceLayout<S, D, R>::kThreads, 1)
    paged_slice_kernel(const __grid_constant__ SliceParams sp) {
  using T = typename S::T;
  using L = SliceLayout<S, D, R>;
  constexpr int W = S::kWarps, NS = S::kStages, kKeys = S::kKeys, SK = S::kStageKeys, kPieces = S::kPieces;
  constexpr int V = 16 / int(sizeof(T));           // elements of a Q copy
  constexpr int CH = D / V;                        // Q copies of a row
  constexpr int CB = D * int(sizeof(T)) / 128;     // 128-byte columns of a row
  // a slot of the ring is always the same workers', who wait for its phases in
  // order (a phase's parity tells it only from the next one)
  static_assert(NS % (W / S::kPerStage) == 0, "a worker's stages keep their slots");
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ int64_t s_scan[64];
  __shared__ PagedStart s_start;
  __shared__ PieceInfo s_piece[kPieces];
  // piece published, its Q landed, its states joined (per entry); stage landed, stage read; all workers' states left
  __shared__ uint64_t s_bar[3 * kPieces + 2 * NS + 1];
  __shared__ int s_abort;
  const PagedArgs& a = sp.a;
  const uint32_t sbase = tc::smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar_piece = [&](int k) { return tc::smem_u32(s_bar + (k % kPieces)); };
  auto bar_q = [&](int k) { return tc::smem_u32(s_bar + kPieces + (k % kPieces)); };
  auto bar_joined = [&](int k) { return tc::smem_u32(s_bar + 2 * kPieces + (k % kPieces)); };
  auto bar_full = [&](uint32_t g) { return tc::smem_u32(s_bar + 3 * kPieces + g % NS); };
  auto bar_empty = [&](uint32_t g) { return tc::smem_u32(s_bar + 3 * kPieces + NS + g % NS); };
  const uint32_t bar_state = tc::smem_u32(s_bar + 3 * kPieces + 2 * NS);
  auto phase = [](int k) { return uint32_t(k / kPieces) & 1u; };
  // whole-warp bounded wait; false: some wait of the block gave up
  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, tc::wait_bounded<kShortWaits>(bar, parity, &s_abort, a.err, sp.wait_limit));
  };
  if (sbase & 1023) {  // the swizzled layouts need a 1 KB aligned base
    if (tid == 0 && a.err) atomicCAS(a.err, 0, 2);
    return;
  }

  grid_launch_dependents();
  // a thread a barrier: one thread's loop over them took 0.4 us
  static_assert(3 * kPieces + 2 * NS + 1 <= 64, "two warps' barriers");
  if (tid < 3 * kPieces + 2 * NS + 1) {
    constexpr int full = 3 * kPieces, empty = full + NS, state = empty + NS;
    tc::mbar_init(tc::smem_u32(s_bar + tid), tid < kPieces       ? 1
                                             : tid < 2 * kPieces ? 32
                                             : tid < full        ? kJoiners
                                             : tid < empty       ? 2  // both producers
                                             : tid < state       ? S::kPerStage
                                                                 : W);
    tc::fence_mbar_init();
  }
  if (tid == 64) s_abort = 0;
  if (tid == 96) tc::prefetch_tmap(&sp.tmk);
  if (tid == 128) tc::prefetch_tmap(&sp.tmv);
  const PagedShare share = paged_locate<kSliceUnit, kSliceExtra, L::kThreads>(a, s_scan, &s_start, blockIdx.x);
  const int64_t u0 = share.first(blockIdx.x), u1 = share.first(blockIdx.x + 1);
  if (u1 <= u0) {
    if (sp.after_pair) grid_wait();
    return;
  }

  if (warp >= W + kJoiners) {
    // ---------------------------------------------------------- producer --
    PagedWalk<kSliceUnit, kSliceExtra> walk;
    walk.start(a, s_start, u1 - u0, blockIdx.x);
    const int bs = sp.box_shift, box = 1 << bs, nb = SK >> bs;  // keys of a box, boxes of a stage's keys
    const bool of_k = warp == W + kJoiners;
    const int sub = lane / CB, col = lane % CB;  // this lane's box
    const bool mine = sub < nb;
    const CUtensorMap* map = of_k ? &sp.tmk : &sp.tmv;
    struct Next {
      PieceInfo i;
      int32_t r;
    };
    auto come = [&]() {
      Next x;
      x.i.valid = 0;
      x.i.nrows = x.i.n = 0;
      x.i.lo = x.i.hi = x.i.key0 = 0;
      x.r = 0;
      PagedPiece p;
      if (walk.next(a, p)) {
        x.i = piece_info<SK>(a, p);
        x.r = p.r;
      }
      return x;
    };
    // Pages of 32 boxes from box f of a piece on, one per lane (n_pages where
    // no row sees a key of it): asked for a window, or a piece, ahead of their use.
    auto seen = [&](const PieceInfo& i, int key) { return key < i.hi && key + box > i.lo; };
    auto window = [&](const Next& x, int f) -> int32_t {
      const int key = x.i.key0 + ((f + lane) << bs);
      return seen(x.i, key) ? a.table[int64_t(x.r) * a.max_blocks + (key >> a.page_shift)] : a.n_pages;
    };
    uint32_t g = 0, q_rows = 0x01010101u * R;  // rows of the places of Q that may hold something
    bool ok = true;
    Next at = come();
    int32_t pages = window(at, 0);
    for (int k = 0; ok; ++k) {
      const PieceInfo& i = at.i;
      if (of_k) {
        ok = k < kPieces || wait(bar_joined(k), phase(k) ^ 1);
        if (!ok) break;
        if (lane == 0) {
          s_piece[k % kPieces] = i;
          tc::mbar_arrive(bar_piece(k));
        }
      }
      if (!i.valid) break;
      // Q, and zeros behind the tile's rows where the place does not hold them yet
      static_assert(kPieces <= 4 && R < 256, "rows of each place in a byte");
      const int byte = 8 * (k % kPieces), had = int(q_rows >> byte) & 255;
      q_rows = (q_rows & ~(255u << byte)) | (uint32_t(i.nrows) << byte);
      const int copies = of_k ? max(i.nrows, had) * CH : 0;
      for (int e = lane; e < copies; e += 32) {
        const int r = e / CH, c = e % CH, row = i.row0 + r;
        const bool in = r < i.nrows;
        const int tok = paged_token(a, row);
        const int64_t off = in ? int64_t(i.q0 + tok) * a.q_stride + int64_t(i.h * a.G + row - tok * a.G) * D + c * V : 0;
        cp_async16(sbase + L::kOffQ + (k % kPieces) * L::kQBytes + S::q_at(r, c), static_cast<const T*>(a.q) + off, in);
      }
      if (of_k) asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar_q(k)) : "memory");
      int32_t more = i.n * nb > 32 ? window(at, 32) : a.n_pages;
      Next ahead;
      int32_t ahead_pages = 0;
      for (int t = 0; t < i.n || t == 0; ++t) {
        if (t < i.n) {
          const int f = t * nb;
          if (f > 0 && (f & 31) == 0) {
            pages = more;
            if (i.n * nb > f + 32) more = window(at, f + 32);
          }
          ok = wait(bar_empty(g), ((g / NS) & 1) ^ 1);
          if (!ok) break;
          if (lane == 0) tc::mbar_arrive_expect_tx(bar_full(g), L::kStageBytes / 2);
          int32_t page = __shfl_sync(0xffffffffu, pages, (f + sub) & 31);
          if (mine) {
            const int key = i.key0 + t * SK + (sub << bs);
            if (uint32_t(page) >= uint32_t(a.n_pages)) {
              if (seen(i, key) && a.err) atomicCAS(a.err, 0, kErrBadPage);
              page = a.n_pages;
            }
            const int token = key & ((1 << a.page_shift) - 1);
            const uint32_t dst = sbase + L::kOffRing + (g % NS) * L::kStageBytes +
                                 (of_k ? 0 : L::kStageBytes / 2) + col * (SK * 128) + ((sub << bs) * 128);
            tma_load_4d(dst, map, bar_full(g), col * (128 / int(sizeof(T))), sp.head_inner ? i.h : token,
                        sp.head_inner ? token : i.h, page);
          }
          ++g;
        }
        if (t == 0) {  // the next piece, and its first pages, behind this one's first stage
          ahead = come();
          ahead_pages = window(ahead, 0);
        }
      }
      at = ahead;
      pages = ahead_pages;
    }
    // Every copy has landed before the block ends, whatever this warp left its
    // loop for: the workers may have given up on the last stages.  (A slot's phase
    // before its last one is complete: its stage was read.  Where the other
    // producer stopped earlier the last phases stay open; then the default
    // budget passes, which the copies do not take.)
    if (lane == 0) {
      volatile int never = 0;
      for (uint32_t s = g > uint32_t(NS) ? g - NS : 0; s < g; ++s) tc::mbar_wait(bar_full(s), (s / NS) & 1, &never, nullptr);
    }
    cp_async_wait<0>();
    if (sp.after_pair) grid_wait();  // this launch is complete only when the one before it is
    return;
  }

  float4* states = reinterpret_cast<float4*>(smem + L::kOffState);
  if (warp >= W) {
    // ------------------------------------------------------------ joiner --
    for (int k = 0;; ++k) {
      if (!wait(bar_piece(k), phase(k))) break;
      const PieceInfo& p = s_piece[k % kPieces];
      if (!p.valid) break;
      if (!wait(bar_state, uint32_t(k) & 1u)) break;
      S::join(a, p, states, warp - W, lane);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar_joined(k));
    }
    return;
  }

  // -------------------------------------------------------------- worker --
  float* scratch = reinterpret_cast<float*>(smem + L::kOffP + warp * S::kScratch);
  const int srow = S::first_key(warp);
  uint32_t g = 0;
  bool ok = true;
  S st;
  for (int k = 0; ok; ++k) {
    if (!wait(bar_piece(k), phase(k))) break;
    const PieceInfo& p = s_piece[k % kPieces];
    if (!p.valid) break;
    if (!wait(bar_q(k), phase(k))) break;
    const uint32_t sq = sbase + L::kOffQ + (k % kPieces) * L::kQBytes;
    st.begin(a, p, sq, warp, lane);
    const int n = p.n, lo = p.lo, hi = p.hi, full_lo = p.full_lo, full_hi = p.full_hi;
    int key = p.key0 + srow;
    for (int t = 0; t < n; ++t, ++g, key += SK) {
      if (int(g % (W / S::kPerStage)) != warp / S::kPerStage) continue;  // other workers' stage
      ok = wait(bar_full(g), (g / NS) & 1);
      if (!ok) break;
      const uint32_t sk = sbase + L::kOffRing + (g % NS) * L::kStageBytes;
      if (key < hi && key + kKeys > lo)
        st.slice(a, sq, sk, sk + L::kStageBytes / 2, srow, scratch, key, key >= full_lo && key + kKeys <= full_hi, lo,
                 hi, lane);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar_empty(g));
    }
    if (!ok) break;
    st.end();
    // the state's place is free once the piece before it is joined
    if (k > 0 && !wait(bar_joined(k - 1), phase(k - 1))) break;
    st.leave(p, states, warp, lane);
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar_state);
  }
}

// Launch that may start while the launch before it on the stream still runs
// (it waits for that one itself: grid_wait).
template <typename P>
cp_status launch_early(void (*kern)(P), dim3 grid, dim3 block, int smem, bool early, cudaStream_t s, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return CP_ERR_CUDA;
  return cuda_status(cudaGetLastError());
}

// ---------------------------------------------------------------- merge ---
// One tile that starts in block c and goes on behind it: its partial states
// are the blocks' from c on.  O = sum_e w_e O_e / sum_e w_e, w_e = 2^(L_e - max L),
// L in log2 units.  The first pieces' O is asked for together with their weights.  What bounds
// it is its launch and three dependent loads (2 us): it starts while the attention
// still runs and finds its tile meanwhile.
constexpr int kMergeThreads = 128, kMergeRows = 32;

template <typename T, int D, int U, int E>
__device__ __forceinline__ void merge_block(const PagedArgs& a, int c, int part, int64_t* s_scan, PagedStart& s_start) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PagedShare share = paged_locate<U, E, kMergeThreads>(a, s_scan, &s_start, c + 1);
  const int64_t u0 = share.first(c), u1 = share.first(c + 1);
  const PagedStart st = s_start;
  // cut here, and started in this block
  const bool work = u1 > u0 && u1 < share.total && st.off > 0 && u1 - st.off >= u0;
  PagedReq q{};
  PagedTile t{};
  int last = c, slot0 = 0;
  if (work) {
    q = paged_req(a, st.r);
    t = paged_tile<U>(a, q, st.t);
    const int64_t begin = u1 - st.off, end = begin + t.n + E;
    // blocks c .. last hold a piece (a block without units cannot lie between
    // two of them: the first ones have the more), c's in its first or second slot
    last = c + 1;
    while (share.first(last + 1) < end) ++last;
    slot0 = 2 * c + (begin == u0 ? 0 : 1);
  }
  grid_wait();
  if (!work) return;
  const int n = last - c + 1;
  auto slot = [&](int e) { return int64_t(e == 0 ? slot0 : 2 * (c + e)); };
  // A slice's partial O is [row][column], 16 lanes a row; a pair's is
  // [4 columns][row] (float4), and 4 lanes with every fourth of them take a row, 8
  // rows a warp side by side.
  constexpr bool kPair = U == kPairUnit;
  constexpr int kLanes = kPair ? 4 : 16, N = D / kLanes, kEager = kPair ? 1 : 2, kAtOnce = kPair ? 1 : 4;
  constexpr int kRowsAtOnce = 32 / kLanes;
  const int which = kPair ? lane & 7 : lane >> 4, sl = kPair ? lane >> 3 : lane & 15;
  const uint32_t lanes = kPair ? 0x01010101u << which : 0xffffu << (16 * which);  // a row's
  auto load = [&](int e, int r, float* x) {
#pragma unroll
    for (int v = 0; v < N; v += 4) {
      const int c4 = sl + kLanes * (v / 4);  // 4 columns
      const int64_t at = kPair ? (slot(e) * (D / 4) + c4) * a.R + r : (slot(e) * a.R + r) * (D / 4) + c4;
      load_vec<float, 4>(a.part_o + 4 * at, x + v);
    }
  };
  for (int i = kRowsAtOnce * warp + which; i < kMergeRows; i += kMergeThreads / kLanes) {
    const int r = part * kMergeRows + i;
    if (r >= t.nrows) break;
    float x[kEager][N];
#pragma unroll
    for (int j = 0; j < kEager; ++j) load(j, r, x[j]);  // n >= 2
    auto weigh = [&](int e0) { return e0 + sl < n ? a.part_l[slot(e0 + sl) * a.R + r] : -INFINITY; };
    const float first = weigh(0);  // the whole of it, up to kLanes pieces
    float top = first;
    for (int e0 = kLanes; e0 < n; e0 += kLanes) top = fmaxf(top, weigh(e0));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(lanes, top, kPair ? 8 * o : o));
    float acc[N] = {};
    float sum = 0.f;
    auto add = [&](float w, int j, const float* y) {
      const float we = __shfl_sync(lanes, w, kPair ? which + 8 * j : 16 * which + j);
      sum += we;
#pragma unroll
      for (int v = 0; v < N; ++v) acc[v] = fmaf(we, y[v], acc[v]);
    };
    for (int e0 = 0; e0 < n; e0 += kLanes) {
      const float own = e0 == 0 ? first : weigh(e0);
      const float w = own == -INFINITY ? 0.f : exp2f(own - top);  // an empty state's O is 0
      const int m = min(kLanes, n - e0);
      int j = 0;
      if (e0 == 0) {
#pragma unroll
        for (; j < kEager; ++j) add(w, j, x[j]);
      }
      for (; j < m; j += kAtOnce) {  // kAtOnce under way (behind the last one, that again)
        float y[kAtOnce][N];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) load(e0 + min(j + i, m - 1), r, y[i]);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          if (j + i < m) add(w, j + i, y[i]);
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int v = 0; v < N; ++v) acc[v] *= inv;
    const int row = t.row0 + r;
    const int tok = paged_token(a, row);
    const int64_t out = int64_t(q.q0 + tok) * a.H + st.h * a.G + (row - tok * a.G);
#pragma unroll
    for (int v = 0; v < N; v += 4)
      store_vec<T, 4>(static_cast<T*>(a.o) + out * D + 4 * (sl + kLanes * (v / 4)), acc + v);
    if (sl == 0) a.lse[out] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
  }
}

struct MergeParams {
  PagedArgs pair, slice;
  int32_t pair_parts;  // blocks of kMergeRows rows of a pair's tile
};

template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const __grid_constant__ MergeParams p) {
  __shared__ int64_t s_scan[64];
  __shared__ PagedStart s_start;
  const int n_pair = p.pair.grid * p.pair_parts;
  if constexpr (sizeof(T) == 2) {
    if (int(blockIdx.x) < n_pair)
      return merge_block<T, D, kPairUnit, kPairExtra>(p.pair, blockIdx.x / p.pair_parts, blockIdx.x % p.pair_parts,
                                                      s_scan, s_start);
  }
  merge_block<T, D, kSliceUnit, kSliceExtra>(p.slice, blockIdx.x - n_pair, 0, s_scan, s_start);
}

template <typename S, int D, int R>
cp_status run_slice(const PagedArgs& a, bool after_pair, cudaStream_t s) {
  using L = SliceLayout<S, D, R>;
  const long long limit = wait_limit_cycles();
  const bool short_waits = limit < tc::kWaitCycles;
  auto* kern = short_waits ? paged_slice_kernel<S, D, R, true> : paged_slice_kernel<S, D, R, false>;
  static std::atomic<bool> ready[2][64] = {};  // per copy and device (an idempotent first set-up)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CP_ERR_CUDA;
  if (!ready[short_waits][dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) != cudaSuccess)
      return CP_ERR_CUDA;
    ready[short_waits][dev].store(true, std::memory_order_release);
  }
  SliceParams p;
  const int page = 1 << a.page_shift, most = std::min(S::kStageKeys, kSliceUnit), box = std::min(page, most);
  p.head_inner = a.head_stride <= a.token_stride;
  if (!make_tmap_pages(&p.tmk, a.k, a, box) || !make_tmap_pages(&p.tmv, a.v, a, box)) return CP_ERR_CUDA;
  p.a = a;
  p.box_shift = 0;
  while ((1 << p.box_shift) < box) ++p.box_shift;
  p.after_pair = after_pair;
  p.wait_limit = limit;
  return launch_early(kern, dim3(unsigned(a.grid)), dim3(L::kThreads), L::kBytes, after_pair, s, p);
}

template <typename T, int D>
cp_status run_merge(const PagedArgs& pair, const PagedArgs& slice, cudaStream_t s) {
  static_assert(kMergeRows >= 32, "a slice's tile is one block's");
  const int parts = (pair.R + kMergeRows - 1) / kMergeRows;
  return launch_early(paged_merge_kernel<T, D>, dim3(unsigned(pair.grid * parts + slice.grid)), dim3(kMergeThreads), 0,
                      true, s, MergeParams{pair, slice, parts});
}

}  // namespace

int paged_slice_grid() { return num_sms(); }

cp_status launch_paged_slice(const PagedArgs& a, PagedKernel k, bool after_pair, cudaStream_t s) {
  if (a.dtype == CP_BF16) {
    if (k == kPagedSlice16)
      return a.d == 128 ? run_slice<SliceBf16<128, 16>, 128, 16>(a, after_pair, s)
                        : run_slice<SliceBf16<64, 16>, 64, 16>(a, after_pair, s);
    if (k == kPagedSlice32)
      return a.d == 128 ? run_slice<SliceBf16<128, 32>, 128, 32>(a, after_pair, s)
                        : run_slice<SliceBf16<64, 32>, 64, 32>(a, after_pair, s);
    return CP_ERR_UNSUPPORTED;
  }
  if (k == kPagedSlice4)
    return a.d == 128 ? run_slice<SliceF32<128, 4>, 128, 4>(a, after_pair, s)
                      : run_slice<SliceF32<64, 4>, 64, 4>(a, after_pair, s);
  if (k == kPagedSlice16)
    return a.d == 128 ? run_slice<SliceF32<128, 16>, 128, 16>(a, after_pair, s)
                      : run_slice<SliceF32<64, 16>, 64, 16>(a, after_pair, s);
  return CP_ERR_UNSUPPORTED;
}

cp_status launch_paged_merge(const PagedArgs& pair, const PagedArgs& slice, cudaStream_t s) {
  const PagedArgs& a = pair.grid > 0 ? pair : slice;
  if (pair.grid > 0 && a.dtype != CP_BF16) return CP_ERR_UNSUPPORTED;
  if (a.dtype == CP_BF16)
    return a.d == 128 ? run_merge<__nv_bfloat16, 128>(pair, slice, s) : run_merge<__nv_bfloat16, 64>(pair, slice, s);
  return a.d == 128 ? run_merge<float, 128>(pair, slice, s) : run_merge<float, 64>(pair, slice, s);
}

}  // namespace cpattn
