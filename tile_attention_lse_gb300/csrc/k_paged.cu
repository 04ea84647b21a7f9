// Attention of a request's new tokens over its pages: the slice kernel and the
// merge of cut tiles.
//
// For a query row at position i of a request with kv cached keys:
//   S_j = scale q . k_j over the visible keys (j < kv; causal: j <= i; window
//   W: i - j < W), L = log sum_j exp S_j, O = sum_j exp(S_j - L) v_j, and O = 0,
//   L = -inf for a row that sees none.  One pass over the keys with a running
//   maximum and sum per row.
//
// What bounds it: a single token per request reads 4 d bytes (bf16) of K and V
// per key and kv-head and does 8 d G flops on them, so HBM is the bound; the
// kernel's job is to keep enough loads in flight on every SM.  Each warp walks
// its own slices of 16 keys (slices w, w + W, ... of the block's piece) through a
// ring of its own, filled by 16-byte asynchronous copies: no block barrier
// stands between a load and its use.  The ring runs on across pieces, so the
// next tile's keys are on their way while a finished tile's warps join their
// states.  Keys behind the request's last, in front of a window or on a page
// number outside the cache are zero-filled without being read, so whatever
// the rest of a page holds cannot reach a sum.
//
// bf16: mma.sync m16n8k16, rows of the tile on M (16 or 32, G query heads of a
//   kv-head packed), so K and V are read once for all of them; P is rounded
//   to bf16 for the second product (relative 2^-8, the inputs' own
//   precision), its row sum is taken in float32 before that.  The legacy
//   tensor path is chosen here because these tiles have too few rows to be
//   bound by it.
// float32: FFMA throughout.  A lane pair owns a key (half of the head each) in
//   the first product, a lane 4 columns of the head in the second.
#include <cuda_bf16.h>

#include <atomic>
#include <mutex>

#include "device_util.cuh"
#include "paged_dev.cuh"
#include "tc_util.cuh"
#include "tmap.h"

namespace cpattn {

namespace {

constexpr int kKeys = 16;  // keys of a slice

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool read) {
  const int n = read ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
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

// What the rows of a tile need to know of a piece, in shared memory.
struct PieceInfo {
  int32_t valid;
  int32_t q0, row0, nrows, h;  // first row of the request in q, tile rows, kv-head
  int32_t pos0;                // position of the request's first new token
  int32_t kv;
  int32_t key0, n;             // first slice's first key, slices
  int32_t lo, hi;              // keys that some row sees
  int32_t full_lo, full_hi;    // keys that every row sees
  int32_t slot;
};

__device__ __forceinline__ void slices_of(const PagedPiece& p, int32_t& key0, int32_t& n) {
  const int a = (p.tile.b0 + p.ua) * kSliceUnit, b = (p.tile.b0 + p.ub) * kSliceUnit;
  key0 = max(a, p.tile.lo & ~(kKeys - 1));
  const int end = min(b, p.tile.hi);
  n = end > key0 ? (end - key0 + kKeys - 1) / kKeys : 0;
}

__device__ __forceinline__ PieceInfo piece_info(const PagedArgs& a, const PagedPiece& p) {
  PieceInfo i;
  i.valid = 1;
  i.q0 = p.q.q0;
  i.row0 = p.tile.row0;
  i.nrows = p.tile.nrows;
  i.h = p.h;
  i.pos0 = p.q.kv - p.q.nq;
  i.kv = p.q.kv;
  slices_of(p, i.key0, i.n);
  i.lo = p.tile.lo;
  i.hi = p.tile.hi;
  const int first = i.pos0 + i.row0 / a.G, last = i.pos0 + (i.row0 + i.nrows - 1) / a.G;
  i.full_hi = a.causal ? min(i.kv, first + 1) : i.kv;
  i.full_lo = a.window > 0 ? max(0, last - a.window + 1) : 0;
  i.slot = p.slot;
  return i;
}

// ------------------------------------------------- bf16: mma.sync tiles ---
template <int D, int R>
struct SliceBf16 {
  using T = __nv_bfloat16;
  static constexpr int kWarps = 8, kStages = 2;
  static constexpr int MT = R / 16, NT = D / 8;
  static constexpr int kAcc = MT * NT * 4, kRows = MT * 2;  // accumulators and rows of a thread
  static constexpr int kQBytes = R * D * 2;
  static constexpr int kScratch = 0;
  static constexpr bool kKeepQ = MT == 1;
  float acc[kAcc];
  float m[kRows], l[kRows];
  uint32_t qf[kKeepQ ? D / 16 : 1][4];
  int32_t lo[kRows], hi[kRows];

  // 16-byte chunk c of row r
  static __device__ __forceinline__ uint32_t at(int r, int c) { return uint32_t(r * D * 2 + ((c ^ (r & 7)) << 4)); }
  static __device__ __forceinline__ uint32_t q_at(int r, int c) { return at(r, c); }

  __device__ __forceinline__ void begin(const PagedArgs& a, const PieceInfo& p, uint32_t sq, int lane) {
#pragma unroll
    for (int i = 0; i < kAcc; ++i) acc[i] = 0.f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      const int pos = p.pos0 + (p.row0 + (lane >> 2) + 8 * i) / a.G;
      hi[i] = a.causal ? min(p.kv, pos + 1) : p.kv;
      lo[i] = a.window > 0 ? pos - a.window + 1 : 0;
    }
    if constexpr (kKeepQ) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) ldm4(sq + at(lane & 15, 2 * k + (lane >> 4)), qf[k]);
    }
  }

  __device__ __forceinline__ void slice(const PagedArgs& a, uint32_t sq, uint32_t sk, uint32_t sv, float*, int key,
                                        bool full, int lane) {
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
      ldm4(sk + at((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)), b);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        uint32_t f[4];
        if constexpr (kKeepQ) {
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = qf[k][e];
        } else {
          ldm4(sq + at(16 * i + (lane & 15), 2 * k + (lane >> 4)), f);
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
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
      uint32_t b[4];
      ldm4t(sv + at(lane & 15, 2 * n + (lane >> 4)), b);
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
  static __device__ __forceinline__ int row_of(int i) { return (i / (NT * 4)) * 2 + ((i >> 1) & 1); }

  // f(row, column, values of two columns), lse(row, value)
  template <typename FO, typename FL>
  __device__ __forceinline__ void write(int lane, FO f, FL g) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int row = (lane >> 2) + 8 * r;
      const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int i = ((r >> 1) * NT + n) * 4 + 2 * (r & 1);
        const float x[2] = {acc[i] * inv, acc[i + 1] * inv};
        f.template operator()<2>(row, 8 * n + 2 * (lane & 3), x);
      }
      if ((lane & 3) == 0) g(row, l[r] > 0.f ? m[r] + tc::lg2(l[r]) : -INFINITY);
    }
  }
};

// --------------------------------------------------------- float32: FFMA ---
template <int D, int R>
struct SliceF32 {
  using T = float;
  static constexpr int kWarps = 4, kStages = 2;
  static constexpr int kAcc = 4 * R, kRows = R;
  static constexpr int kQStride = (D + 4) * 4;  // the second half of a row sits 16 bytes on: other banks
  static constexpr int kQBytes = R * kQStride;
  static constexpr int kScratch = kKeys * R * 4;  // P of a warp's slice
  float acc[kAcc];
  float m[R], l[R];
  int32_t pos0, row0, kv;

  static __device__ __forceinline__ uint32_t at(int r, int c) { return uint32_t(r * D * 4 + ((c ^ (r & 7)) << 4)); }
  static __device__ __forceinline__ uint32_t q_at(int r, int c) {
    return uint32_t(r * kQStride + ((c + (c >= D / 8 ? 1 : 0)) << 4));
  }
  static __device__ __forceinline__ float4 lds4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
  }

  __device__ __forceinline__ void begin(const PagedArgs&, const PieceInfo& p, uint32_t, int) {
#pragma unroll
    for (int i = 0; i < kAcc; ++i) acc[i] = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
    }
    pos0 = p.pos0;
    row0 = p.row0;
    kv = p.kv;
  }

  __device__ __forceinline__ void slice(const PagedArgs& a, uint32_t sq, uint32_t sk, uint32_t sv, float* sp, int key,
                                        bool full, int lane) {
    const int kx = lane & 15, half = lane >> 4;
    float s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = 0.f;
#pragma unroll 4
    for (int c0 = 0; c0 < D / 8; ++c0) {
      const int c = half * (D / 8) + c0;
      const float4 k = lds4(sk + at(kx, c));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 q = lds4(sq + uint32_t(r * kQStride + ((c + half) << 4)));
        s[r] = fmaf(q.x, k.x, s[r]);
        s[r] = fmaf(q.y, k.y, s[r]);
        s[r] = fmaf(q.z, k.z, s[r]);
        s[r] = fmaf(q.w, k.w, s[r]);
      }
    }
    const int j = key + kx;
    bool grow = false;
    float up[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[r] += __shfl_xor_sync(0xffffffffu, s[r], 16);
      if (!full) {
        const int pos = pos0 + (row0 + r) / a.G;
        const bool see = j < kv && (!a.causal || j <= pos) && (a.window == 0 || pos - j < a.window);
        s[r] = see ? s[r] : -INFINITY;
      }
      float v = s[r];
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
      up[r] = v * a.scale_log2;
      grow |= up[r] > m[r] + 8.f;
    }
    if (grow) {  // the same in every lane
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float t = fmaxf(m[r], up[r]);
        const float c = m[r] == -INFINITY ? 0.f : exp2f(m[r] - t);
        m[r] = t;
        l[r] *= c;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[4 * r + e] *= c;
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float base = m[r] == -INFINITY ? 0.f : m[r];
      s[r] = exp2f(fmaf(s[r], a.scale_log2, -base));
      if (half == 0) l[r] += s[r];
    }
    if (half == 0) {
#pragma unroll
      for (int r = 0; r < R; r += 4)
        *reinterpret_cast<float4*>(sp + kx * R + r) = make_float4(s[r], s[r + 1], s[r + 2], s[r + 3]);
    }
    __syncwarp();
    // head_dim 128: 32 lanes x 4 columns; 64: 16 lanes x 4 columns, each half of the warp half of the keys
    constexpr int kn = D == 128 ? kKeys : kKeys / 2;
    const int c = D == 128 ? lane : kx;
#pragma unroll 4
    for (int i = 0; i < kn; ++i) {
      const int x = D == 128 ? i : half * kn + i;
      const float4 v = lds4(sv + at(x, c));
#pragma unroll
      for (int r = 0; r < R; r += 4) {
        const float4 p = *reinterpret_cast<const float4*>(sp + x * R + r);
        const float pr[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          float* o = acc + 4 * (r + t);
          o[0] = fmaf(pr[t], v.x, o[0]);
          o[1] = fmaf(pr[t], v.y, o[1]);
          o[2] = fmaf(pr[t], v.z, o[2]);
          o[3] = fmaf(pr[t], v.w, o[3]);
        }
      }
    }
  }

  __device__ __forceinline__ void end() {
#pragma unroll
    for (int r = 0; r < R; ++r) l[r] = warp_sum(l[r]);
    if (D == 64) {
#pragma unroll
      for (int i = 0; i < kAcc; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 16);
    }
  }
  static __device__ __forceinline__ int row_of(int i) { return i >> 2; }

  template <typename FO, typename FL>
  __device__ __forceinline__ void write(int lane, FO f, FL g) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
      const float x[4] = {acc[4 * r] * inv, acc[4 * r + 1] * inv, acc[4 * r + 2] * inv, acc[4 * r + 3] * inv};
      if (4 * lane < D) f.template operator()<4>(r, 4 * lane, x);
      if (lane == 0) g(r, l[r] > 0.f ? m[r] + log2f(l[r]) : -INFINITY);
    }
  }
};

// Where a tile's rows go: the outputs, or its partial state.
template <typename T, int D, int R>
struct SliceOut {
  const PagedArgs& a;
  int slot, nrows, G, row0, h0;
  int64_t q0;
  __device__ __forceinline__ int64_t row(int r) const {
    const int x = row0 + r;
    return (q0 + x / G) * a.H + h0 + x % G;
  }
  template <int N>
  __device__ __forceinline__ void operator()(int r, int c, const float* x) const {
    if (r >= nrows) return;
    if (slot < 0)
      store_vec<T, N>(static_cast<T*>(a.o) + row(r) * D + c, x);
    else
      store_vec<float, N>(a.part_o + (int64_t(slot) * R + r) * D + c, x);
  }
};

template <typename S, int D, int R>
struct SliceLayout {
  static constexpr int kStageBytes = 2 * kKeys * D * int(sizeof(typename S::T));
  static constexpr int kOffRing = 0;
  static constexpr int kOffJoin = kOffRing + S::kWarps * S::kStages * kStageBytes;
  static constexpr int kJoinBytes = 32 * (S::kAcc + 2 * S::kRows) * 4;  // one warp's state
  static constexpr int kOffQ = kOffJoin + (S::kWarps / 2) * kJoinBytes;
  static constexpr int kQBytes = (S::kQBytes + 127) & ~127;
  static constexpr int kOffP = kOffQ + 2 * kQBytes;
  static constexpr int kBytes = kOffP + S::kWarps * S::kScratch;
  static_assert(kBytes + 2048 <= 232448, "shared memory of one block");
};

template <typename S, int D, int R>
__global__ void __launch_bounds__(S::kWarps * 32, 1) paged_slice_kernel(const __grid_constant__ PagedArgs a) {
  using T = typename S::T;
  using L = SliceLayout<S, D, R>;
  constexpr int W = S::kWarps, NS = S::kStages, kThreads = W * 32;
  constexpr int V = 16 / int(sizeof(T));   // elements of a copy
  constexpr int CH = D / V;                // copies of a row
  constexpr int KPI = 32 / CH > 0 ? 32 / CH : 1;  // keys of one step of a warp's copies
  static_assert(CH <= 32, "a row fits a warp's copies");
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ int64_t s_scan[34];
  __shared__ PagedStart s_start[2];
  __shared__ PieceInfo s_piece[4];
  __shared__ PagedWalk<kSliceUnit, kSliceExtra> s_walk;
  const uint32_t sbase = tc::smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  grid_launch_dependents();
  int64_t u0, u1;
  {
    const int64_t total = paged_locate<kSliceUnit, kSliceExtra, kThreads>(a, s_scan, s_start, [&](int64_t t, int k) {
      return k == 0 ? paged_first_unit(t, blockIdx.x, a.grid) : t;
    });
    u0 = paged_first_unit(total, blockIdx.x, a.grid);
    u1 = paged_first_unit(total, blockIdx.x + 1, a.grid);
  }
  if (u1 <= u0) return;

  // ---- this warp's copies: a walk of its own, ahead of the products ----
  PagedWalk<kSliceUnit, kSliceExtra> wp;
  wp.start(a, s_start[0], u1 - u0, blockIdx.x);
  int32_t p_r = 0, p_h = 0, p_key0 = 0, p_n = 0, p_s = 0, p_lo = 0, p_hi = 0;
  bool more = true;
  int32_t pg[2] = {-1, -1};
  auto look_up = [&]() {  // the pages of the slice that is copied next
    const int32_t key = p_key0 + p_s * kKeys;
    const int32_t* row = a.table + int64_t(p_r) * a.max_blocks;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int32_t k8 = key + 8 * i;
      pg[i] = k8 < p_hi && k8 + 8 > p_lo ? row[k8 >> a.page_shift] : -1;
    }
  };
  auto advance = [&](int step) {
    p_s += step;
    while (p_s >= p_n) {
      PagedPiece p;
      if (!wp.next(a, p)) {
        more = false;
        return;
      }
      slices_of(p, p_key0, p_n);
      p_r = p.r;
      p_h = p.h;
      p_lo = p.tile.lo;
      p_hi = p.tile.hi;
      p_s = warp;
    }
    look_up();
  };
  uint32_t issued = 0;
  auto issue = [&]() {
    if (more) {
      const uint32_t dst = sbase + L::kOffRing + (warp * NS + issued % NS) * L::kStageBytes;
      const int32_t key = p_key0 + p_s * kKeys;
      const int ck = lane % CH;
#pragma unroll
      for (int i = 0; i < kKeys / KPI; ++i) {
        const int kx = i * KPI + lane / CH;
        const int32_t j = key + kx;
        const int32_t page = kx < 8 ? pg[0] : pg[1];
        const bool wanted = j >= p_lo && j < p_hi;
        const bool ok = wanted && uint32_t(page) < uint32_t(a.n_pages);
        if (wanted && !ok && a.err) atomicCAS(a.err, 0, kErrBadPage);
        const int64_t off = ok ? page * a.page_stride + int64_t(j & ((1 << a.page_shift) - 1)) * a.token_stride +
                                     p_h * a.head_stride + ck * V
                               : 0;
        cp_async16(dst + S::at(kx, ck), static_cast<const T*>(a.k) + off, ok);
        cp_async16(dst + L::kStageBytes / 2 + S::at(kx, ck), static_cast<const T*>(a.v) + off, ok);
      }
      advance(W);
    }
    cp_async_commit();
    ++issued;
  };
  p_s = warp;  // p_n = 0: the first advance takes the first piece
  advance(0);
#pragma unroll
  for (int i = 0; i < NS; ++i) issue();

  // ---- pieces: one thread walks, two ahead ----
  auto walk = [&](int k) {
    PagedPiece p;
    PieceInfo i;
    i.valid = 0;
    if (s_walk.next(a, p)) i = piece_info(a, p);
    s_piece[k & 3] = i;
  };
  // Q of a tile, 16 bytes per thread and step, zeros behind its rows
  constexpr int kQSteps = (R * CH + kThreads - 1) / kThreads;
  uint4 qv[kQSteps];
  auto load_q = [&](const PieceInfo& p) {
#pragma unroll
    for (int i = 0; i < kQSteps; ++i) {
      const int e = tid + i * kThreads, r = e / CH, c = e % CH;
      qv[i] = make_uint4(0, 0, 0, 0);
      if (p.valid && r < R && r < p.nrows) {
        const int row = p.row0 + r;
        qv[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + int64_t(p.q0 + row / a.G) * a.q_stride +
                                                int64_t(p.h * a.G + row % a.G) * D + c * V);
      }
    }
  };
  auto store_q = [&](int k) {
#pragma unroll
    for (int i = 0; i < kQSteps; ++i) {
      const int e = tid + i * kThreads, r = e / CH, c = e % CH;
      if (r < R) *reinterpret_cast<uint4*>(smem + L::kOffQ + (k & 1) * L::kQBytes + S::q_at(r, c)) = qv[i];
    }
  };
  if (tid == 0) {
    s_walk.start(a, s_start[0], u1 - u0, blockIdx.x);
    walk(0);
    walk(1);
  }
  __syncthreads();
  load_q(s_piece[0]);
  store_q(0);
  __syncthreads();

  float* join = reinterpret_cast<float*>(smem + L::kOffJoin);
  constexpr int kState = S::kAcc + 2 * S::kRows;
  float* sp = reinterpret_cast<float*>(smem + L::kOffP + warp * S::kScratch);
  uint32_t used = 0;
  S st;
  for (int k = 0;; ++k) {
    const PieceInfo& p = s_piece[k & 3];
    if (!p.valid) break;
    load_q(s_piece[(k + 1) & 3]);
    if (tid == kThreads - 32) walk(k + 2);
    const uint32_t sq = sbase + L::kOffQ + (k & 1) * L::kQBytes;
    st.begin(a, p, sq, lane);
    const int key0 = p.key0, n = p.n, full_lo = p.full_lo, full_hi = p.full_hi;
    for (int s = warp; s < n; s += W) {
      cp_async_wait<NS - 1>();
      __syncwarp();
      const uint32_t sk = sbase + L::kOffRing + (warp * NS + used % NS) * L::kStageBytes;
      const int key = key0 + s * kKeys;
      st.slice(a, sq, sk, sk + L::kStageBytes / 2, sp, key, key >= full_lo && key + kKeys <= full_hi, lane);
      __syncwarp();
      ++used;
      issue();
    }
    st.end();
    // ---- the warps' states join pairwise; a writer's region was last read by itself ----
    __syncthreads();
#pragma unroll
    for (int half = W / 2; half >= 1; half >>= 1) {
      if (warp >= half && warp < 2 * half) {
        float* x = join + (half == W / 2 ? warp - half : warp) * (L::kJoinBytes / 4) + lane;
#pragma unroll
        for (int i = 0; i < S::kAcc; ++i) x[i * 32] = st.acc[i];
#pragma unroll
        for (int r = 0; r < S::kRows; ++r) {
          x[(S::kAcc + r) * 32] = st.m[r];
          x[(S::kAcc + S::kRows + r) * 32] = st.l[r];
        }
      }
      if (half == W / 2) store_q(k + 1);
      __syncthreads();
      if (warp < half) {
        const float* x = join + (half == W / 2 ? warp : warp + half) * (L::kJoinBytes / 4) + lane;
        float c0[S::kRows], c1[S::kRows];
#pragma unroll
        for (int r = 0; r < S::kRows; ++r) {
          const float mo = x[(S::kAcc + r) * 32], lo = x[(S::kAcc + S::kRows + r) * 32];
          const float t = fmaxf(st.m[r], mo);
          c0[r] = st.m[r] == -INFINITY ? 0.f : exp2f(st.m[r] - t);
          c1[r] = mo == -INFINITY ? 0.f : exp2f(mo - t);
          st.m[r] = t;
          st.l[r] = st.l[r] * c0[r] + lo * c1[r];
        }
#pragma unroll
        for (int i = 0; i < S::kAcc; ++i) {
          const int r = S::row_of(i);
          st.acc[i] = st.acc[i] * c0[r] + x[i * 32] * c1[r];
        }
      }
    }
    if (warp == 0) {
      const int G = a.G, slot = p.slot, nrows = p.nrows;
      const int64_t q0 = p.q0;
      const int row0 = p.row0, h0 = p.h * G;
      const SliceOut<T, D, R> out{a, slot, nrows, G, row0, h0, q0};
      st.write(lane, out, [&](int r, float v) {
        if (r >= nrows) return;
        if (slot < 0)
          a.lse[out.row(r)] = v * 0.69314718055994531f;
        else
          a.part_l[int64_t(slot) * R + r] = v;
      });
    }
  }
  cp_async_wait<0>();
}

// ---------------------------------------------------------------- merge ---
// One tile that starts in block c and goes on behind it: its partial states
// are the blocks' from c on.  O = sum_e w_e O_e / sum_e w_e, w_e = 2^(L_e - max L),
// L in log2 units, a warp per row; what bounds it is the launch (about 2 us).
constexpr int kMergeThreads = 128, kMergeRows = 8;

template <typename T, int D, int U, int E>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const __grid_constant__ PagedArgs a) {
  __shared__ int64_t s_scan[34];
  __shared__ PagedStart s_start[2];
  const int c = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t total = paged_locate<U, E, kMergeThreads>(a, s_scan, s_start, [&](int64_t t, int k) {
    return k == 0 ? paged_first_unit(t, c + 1, a.grid) : t;
  });
  grid_wait();
  const int64_t u0 = paged_first_unit(total, c, a.grid), u1 = paged_first_unit(total, c + 1, a.grid);
  if (u1 <= u0 || u1 >= total) return;
  const PagedStart st = s_start[0];
  if (st.off == 0 || u1 - st.off < u0) return;  // not cut here, or it started in an earlier block
  const PagedReq q = paged_req(a, st.r);
  const PagedTile t = paged_tile<U>(a, q, st.t);
  const int64_t begin = u1 - st.off, end = begin + t.n + E;
  // blocks c .. c + n - 1 hold a piece, the first in its first or second slot
  int last = c + 1;
  while (paged_first_unit(total, last + 1, a.grid) < end) ++last;
  // a block without units leaves no state
  const int first_slot = 2 * c + (begin == u0 ? 0 : 1);
  for (int i = warp; i < kMergeRows; i += kMergeThreads / 32) {
    const int r = blockIdx.y * kMergeRows + i;
    if (r >= t.nrows) break;
    float top = -INFINITY;
    for (int e = c + lane; e <= last; e += 32) {
      if (paged_first_unit(total, e + 1, a.grid) <= paged_first_unit(total, e, a.grid)) continue;
      const int slot = e == c ? first_slot : 2 * e;
      top = fmaxf(top, a.part_l[int64_t(slot) * a.R + r]);
    }
    top = warp_max(top);
    constexpr int N = D / 32;
    float acc[N] = {};
    float sum = 0.f;
    if (top != -INFINITY) {
      for (int e0 = c; e0 <= last; e0 += 32) {
        float w = 0.f;
        const int e = e0 + lane;
        if (e <= last && paged_first_unit(total, e + 1, a.grid) > paged_first_unit(total, e, a.grid))
          w = exp2f(a.part_l[int64_t(e == c ? first_slot : 2 * e) * a.R + r] - top);
        const int m = min(32, last - e0 + 1);
#pragma unroll 4
        for (int i2 = 0; i2 < m; ++i2) {
          const float we = __shfl_sync(0xffffffffu, w, i2);
          if (we == 0.f) continue;  // an empty state's O was not written
          const int slot = e0 + i2 == c ? first_slot : 2 * (e0 + i2);
          float x[N];
          load_vec<float, N>(a.part_o + (int64_t(slot) * a.R + r) * D + N * lane, x);
          sum += we;
#pragma unroll
          for (int j = 0; j < N; ++j) acc[j] = fmaf(we, x[j], acc[j]);
        }
      }
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] *= inv;
    const int row = t.row0 + r;
    const int64_t out = int64_t(q.q0 + row / a.G) * a.H + st.h * a.G + row % a.G;
    store_vec<T, N>(static_cast<T*>(a.o) + out * D + N * lane, acc);
    if (lane == 0) a.lse[out] = sum > 0.f ? (top + log2f(sum)) * 0.69314718055994531f : -INFINITY;
  }
}

template <typename S, int D, int R>
cp_status run_slice(const PagedArgs& a, cudaStream_t s) {
  using L = SliceLayout<S, D, R>;
  auto* kern = paged_slice_kernel<S, D, R>;
  static std::atomic<bool> ready[64] = {};  // per device (an idempotent first set-up)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CP_ERR_CUDA;
  if (!ready[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) != cudaSuccess)
      return CP_ERR_CUDA;
    ready[dev].store(true, std::memory_order_release);
  }
  kern<<<unsigned(a.grid), S::kWarps * 32, L::kBytes, s>>>(a);
  return cuda_status(cudaGetLastError());
}

template <typename T, int D, int U, int E>
cp_status run_merge(const PagedArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(unsigned(a.grid), unsigned((a.R + kMergeRows - 1) / kMergeRows));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, paged_merge_kernel<T, D, U, E>, a) != cudaSuccess) return CP_ERR_CUDA;
  return cuda_status(cudaGetLastError());
}

}  // namespace

int paged_slice_grid() { return num_sms(); }

cp_status launch_paged_slice(const PagedArgs& a, PagedKernel k, cudaStream_t s) {
  if (a.dtype == CP_BF16) {
    if (k == kPagedSlice16)
      return a.d == 128 ? run_slice<SliceBf16<128, 16>, 128, 16>(a, s) : run_slice<SliceBf16<64, 16>, 64, 16>(a, s);
    if (k == kPagedSlice32)
      return a.d == 128 ? run_slice<SliceBf16<128, 32>, 128, 32>(a, s) : run_slice<SliceBf16<64, 32>, 64, 32>(a, s);
    return CP_ERR_UNSUPPORTED;
  }
  if (k == kPagedSlice4)
    return a.d == 128 ? run_slice<SliceF32<128, 4>, 128, 4>(a, s) : run_slice<SliceF32<64, 4>, 64, 4>(a, s);
  if (k == kPagedSlice16)
    return a.d == 128 ? run_slice<SliceF32<128, 16>, 128, 16>(a, s) : run_slice<SliceF32<64, 16>, 64, 16>(a, s);
  return CP_ERR_UNSUPPORTED;
}

cp_status launch_paged_merge(const PagedArgs& a, PagedKernel k, cudaStream_t s) {
  if (k == kPagedPair) {
    if (a.d != 128 || a.dtype != CP_BF16) return CP_ERR_UNSUPPORTED;
    return run_merge<__nv_bfloat16, 128, kPairUnit, kPairExtra>(a, s);
  }
  if (a.dtype == CP_BF16)
    return a.d == 128 ? run_merge<__nv_bfloat16, 128, kSliceUnit, kSliceExtra>(a, s)
                      : run_merge<__nv_bfloat16, 64, kSliceUnit, kSliceExtra>(a, s);
  return a.d == 128 ? run_merge<float, 128, kSliceUnit, kSliceExtra>(a, s)
                    : run_merge<float, 64, kSliceUnit, kSliceExtra>(a, s);
}

}  // namespace cpattn
