// Backward of cross attention in float32 (FFMA): dK, dV and the table's gradient
// by tiles of keys, dQ by tiles of queries.  The formulas stand in cross.h; no atomics,
// every sum has one owner and one order.
//
// Items of both form S and dP of a tile of 64 keys and 64 queries: thread (ty, tx) of 16 x 16 owns
// keys ty + 16 a and queries tx + 16 b, a, b < 4, and walks the head dimension in 16-byte
// steps on packed pairs (two FMAs an instruction); rows in shared memory are D + 4 floats apart, so that
// 8 lanes' rows fall on different banks.  P and dS change hands through shared memory, and in the second
// products a thread owns 4 rows and D / 16 columns.  dQ forms S and dP again (7 products instead of 5)
// rather than adding up in memory.  Measured, 4 sequences of 2048, 16 heads of 64: 8465 us, 28 TFLOP/s of the 7 products (FFMA
// about 78); 5 pairs of about 100 over 333, 8 heads over 2: 124 us.  The bound is the wait for a tile's rows, which come
// between two barriers with nothing under way, and in small calls items that are fewer than the SMs.
#include <atomic>

#include "cross.h"
#include "device_util.cuh"
#include "philox.cuh"
#include "tc_util.cuh"
#include "tmap.h"

namespace cpattn {

namespace {

constexpr int kB = 64;  // keys and queries of a tile
constexpr int kThreads = 256;
constexpr int kPad = 4;

template <int D>
struct Smem {
  float k[kB][D + kPad], v[kB][D + kPad], q[kB][D + kPad], o[kB][D + kPad];
  float p[kB][kB + kPad], s[kB][kB + kPad];  // [key][query]: keep P, dS / r
  float l[kB], d[kB];                         // L2 and D / r of the queries
  float diag[2 * kB];
};

// Rows of a [rows][heads][D] tensor into shared memory, zeros behind the last.
template <int D>
__device__ __forceinline__ void load_rows(float (*to)[D + kPad], const void* from, int64_t stride, int64_t row, int head,
                                          int n) {
  for (int e = threadIdx.x; e < kB * (D / 4); e += kThreads) {
    const int r = e / (D / 4), c = e % (D / 4);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < n)
      x = *reinterpret_cast<const float4*>(static_cast<const float*>(from) + (row + r) * stride + int64_t(head) * D + 4 * c);
    *reinterpret_cast<float4*>(&to[r][4 * c]) = x;
  }
}

// What a tile of keys and queries needs to know.
struct Tile {
  int seq, head;
  int key0, keys, query0, queries, off;  // off: position of query 0
};

// P (under dropout the kept ones) and dS / r of a tile into shared memory.
template <int D>
__device__ __forceinline__ void probabilities(const CrossBwd& a, Smem<D>& m, const Tile& t, const DropKey& dkey) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  uint64_t s2[4][4] = {}, d2[4][4] = {};
#pragma unroll 2
  for (int c = 0; c < D; c += 4) {
    ulonglong2 k[4], v[4], q[4], o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      k[i] = *reinterpret_cast<const ulonglong2*>(&m.k[ty + 16 * i][c]);
      v[i] = *reinterpret_cast<const ulonglong2*>(&m.v[ty + 16 * i][c]);
      q[i] = *reinterpret_cast<const ulonglong2*>(&m.q[tx + 16 * i][c]);
      o[i] = *reinterpret_cast<const ulonglong2*>(&m.o[tx + 16 * i][c]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s2[i][j] = tc::ffma2(k[i].x, q[j].x, s2[i][j]);
        d2[i][j] = tc::ffma2(v[i].x, o[j].x, d2[i][j]);
        s2[i][j] = tc::ffma2(k[i].y, q[j].y, s2[i][j]);
        d2[i][j] = tc::ffma2(v[i].y, o[j].y, d2[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = ty + 16 * i, c = tx + 16 * j, key = t.key0 + r, query = t.query0 + c;
      float x, y, d, e;
      tc::f32x2_split(s2[i][j], x, y);
      tc::f32x2_split(d2[i][j], d, e);
      d += e;
      const bool see = r < t.keys && c < t.queries && (!a.causal || key <= query + t.off);
      const float bias = a.rel ? rel_bias(a, t.head, key - query - t.off) : 0.f;
      const float p = see ? exp2f(fmaf(x + y, a.scale_log2, bias) - m.l[c]) : 0.f;
      bool keep = true;
      if (a.rng) {
        const Draw dr = draw(dkey, uint32_t(key) >> 3, uint32_t(query), uint32_t(t.seq) * uint32_t(a.H) + uint32_t(t.head));
        keep = (keep_bits(dr, dkey.add) >> (key & 7)) & 1u;
      }
      m.p[r][c] = keep ? p : 0.f;
      m.s[r][c] = see ? p * ((keep ? d : 0.f) - m.d[c]) : 0.f;
    }
}

__device__ __forceinline__ void load_l_d(const CrossBwd& a, float* l, float* d, int head, int64_t row, int n) {
  const int i = threadIdx.x;
  if (i < kB) {
    l[i] = i < n ? a.lse2[int64_t(head) * a.rows + row + i] : INFINITY;
    d[i] = i < n ? a.delta[int64_t(head) * a.rows + row + i] : 0.f;
  }
}

// acc[4 rows][D / 16 columns] += sum_x w(x, row) b[x][column]: rows ty + 16 i, columns 4 tx + 64 c ..  A tile's
// sum is formed apart: one chain over all keys would be off by sqrt(n) roundings of what it holds (dQ of
// 65536 keys by 4.7e-6 of its norm).
template <int D, typename W>
__device__ __forceinline__ void second(uint64_t (*acc)[D / 32], const float (*b)[D + kPad], W w) {
  const int tx = threadIdx.x & 15;
  uint64_t sum[4][D / 32] = {};
#pragma unroll 4
  for (int x = 0; x < kB; ++x) {
    ulonglong2 y[D / 64];
#pragma unroll
    for (int c = 0; c < D / 64; ++c) y[c] = *reinterpret_cast<const ulonglong2*>(&b[x][4 * tx + 64 * c]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = w(x, i);
      const uint64_t f2 = tc::f32x2(f, f);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        sum[i][2 * c] = tc::ffma2(f2, y[c].x, sum[i][2 * c]);
        sum[i][2 * c + 1] = tc::ffma2(f2, y[c].y, sum[i][2 * c + 1]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < D / 32; ++c) acc[i][c] = tc::fadd2(acc[i][c], sum[i][c]);
}
template <int D>
__device__ __forceinline__ void store(void* to, int64_t row, int heads, int head, int n, const uint64_t (*acc)[D / 32],
                                      float mul) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (ty + 16 * i >= n) continue;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      float x[4];
      tc::f32x2_split(acc[i][2 * c], x[0], x[1]);
      tc::f32x2_split(acc[i][2 * c + 1], x[2], x[3]);
      *reinterpret_cast<float4*>(static_cast<float*>(to) + ((row + ty + 16 * i) * heads + head) * D + 4 * tx + 64 * c) =
          make_float4(x[0] * mul, x[1] * mul, x[2] * mul, x[3] * mul);
    }
  }
}

// dK, dV and the table's gradient of a tile of keys and a kv-head.
template <int D>
__device__ __forceinline__ void key_item(const CrossBwd& a, Smem<D>& m, int64_t w, const DropKey& dkey) {
  const int ty = threadIdx.x >> 4, tid = threadIdx.x;
  const CrossTile ct = a.k_tiles.list[w / a.Hkv];
  const int g = int(w % a.Hkv);
  const PagedReq q = paged_req(a, ct.seq);
  Tile t;
  t.seq = ct.seq;
  t.key0 = ct.first;
  t.keys = min(kB, q.kv - ct.first);
  t.off = q.kv - q.nq;
  const int64_t krow = paged_key_row(a, ct.seq) + ct.first;
  const int qlo = cross_first_query(a, q, ct.first);
  uint64_t dk[4][D / 32] = {}, dv[4][D / 32] = {};
  __syncthreads();
  load_rows<D>(m.k, a.k, a.k_stride, krow, g, t.keys);
  load_rows<D>(m.v, a.v, a.v_stride, krow, g, t.keys);
  for (int hj = 0; hj < a.G; ++hj) {
    t.head = g * a.G + hj;
    float sum = 0.f;  // thread b: the table's gradient of bucket b
    int lo = 1, hi = 0;
    if (a.rel && tid < a.buckets) rel_range(a.starts, tid, &lo, &hi);
    for (t.query0 = qlo; t.query0 < q.nq; t.query0 += kB) {
      t.queries = min(kB, q.nq - t.query0);
      const int64_t row = q.q0 + t.query0;
      load_rows<D>(m.q, a.q, a.q_stride, row, t.head, t.queries);
      load_rows<D>(m.o, a.dout, a.do_stride, row, t.head, t.queries);
      load_l_d(a, m.l, m.d, t.head, row, t.queries);
      __syncthreads();
      probabilities<D>(a, m, t, dkey);
      __syncthreads();
      second<D>(dv, m.o, [&](int x, int i) { return m.p[ty + 16 * i][x]; });
      second<D>(dk, m.q, [&](int x, int i) { return m.s[ty + 16 * i][x]; });
      if (a.rel) {  // diagonals of dS, then each bucket's of them
        const int x0 = t.key0 - t.query0 - t.off - (kB - 1);  // relative position of diagonal 0
        if (tid < 2 * kB - 1) {
          float s = 0.f;
          const int d = tid - (kB - 1);  // key - query
          for (int i = max(0, -d); i < min(kB, kB - d); ++i) s += m.s[i + d][i];
          m.diag[tid] = s;
        }
        __syncthreads();
        const int d1 = min(hi - x0, 2 * kB - 2);
        float s = 0.f;
        for (int d = max(lo - x0, 0); d <= d1; ++d) s += m.diag[d];
        sum += s;
      }
      __syncthreads();
    }
    if (a.rel && tid < a.bucket_stride) a.part[(int64_t(ct.id) * a.H + t.head) * a.bucket_stride + tid] = sum;
  }
  store<D>(a.dk, krow, a.Hkv, g, t.keys, dk, a.scale * a.drop_scale);
  store<D>(a.dv, krow, a.Hkv, g, t.keys, dv, a.drop_scale);
}

// dQ of a tile of queries and a head.
template <int D>
__device__ __forceinline__ void query_item(const CrossBwd& a, Smem<D>& m, int64_t w, const DropKey& dkey) {
  const int ty = threadIdx.x >> 4;
  const CrossTile ct = a.q_tiles.list[w / a.H];
  const PagedReq q = paged_req(a, ct.seq);
  Tile t;
  t.seq = ct.seq;
  t.head = int(w % a.H);
  t.query0 = ct.first;
  t.queries = min(kB, q.nq - ct.first);
  t.off = q.kv - q.nq;
  const int64_t row = q.q0 + ct.first, krow = paged_key_row(a, ct.seq);
  const int end = a.causal ? min(q.kv, ct.first + t.queries + t.off) : q.kv;  // keys that some query sees
  uint64_t dq[4][D / 32] = {};
  __syncthreads();
  load_rows<D>(m.q, a.q, a.q_stride, row, t.head, t.queries);
  load_rows<D>(m.o, a.dout, a.do_stride, row, t.head, t.queries);
  load_l_d(a, m.l, m.d, t.head, row, t.queries);
  for (t.key0 = 0; t.key0 < end; t.key0 += kB) {
    t.keys = min(kB, q.kv - t.key0);
    load_rows<D>(m.k, a.k, a.k_stride, krow + t.key0, t.head / a.G, t.keys);
    load_rows<D>(m.v, a.v, a.v_stride, krow + t.key0, t.head / a.G, t.keys);
    __syncthreads();
    probabilities<D>(a, m, t, dkey);
    __syncthreads();
    second<D>(dq, m.k, [&](int x, int i) { return m.s[x][ty + 16 * i]; });
    __syncthreads();
  }
  store<D>(a.dq, row, a.H, t.head, t.queries, dq, a.scale * a.drop_scale);
}

// Items of keys (the longer ones) in front of items of queries, in one launch: few short sequences fill
// the SMs with neither alone (5 pairs of about 100 over 333, 8 heads over 2: 228 us as two launches).
template <int D>
__global__ void __launch_bounds__(kThreads, 1) cross_bwd_f32_kernel(const __grid_constant__ CrossBwd a) {
  extern __shared__ __align__(16) uint8_t raw[];
  Smem<D>& m = *reinterpret_cast<Smem<D>*>(raw);
  DropKey dkey{};
  if (a.rng) dkey = drop_key(a.rng, a.drop_min);
  const int64_t nk = int64_t(*a.k_tiles.count) * a.Hkv, n = nk + int64_t(*a.q_tiles.count) * a.H;
  for (int64_t w = blockIdx.x; w < n; w += gridDim.x) {
    if (w < nk)
      key_item<D>(a, m, w, dkey);
    else
      query_item<D>(a, m, w - nk, dkey);
  }
}

template <int D>
cp_status run(const CrossBwd& a, cudaStream_t s) {
  static std::atomic<bool> ready[64] = {};  // per device (an idempotent first set-up)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CP_ERR_CUDA;
  const int bytes = int(sizeof(Smem<D>));
  if (!ready[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(cross_bwd_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
      return CP_ERR_CUDA;
    ready[dev].store(true, std::memory_order_release);
  }
  const int64_t blocks = num_sms();
  const int64_t most = int64_t(a.k_tiles.most) * a.Hkv + int64_t(a.q_tiles.most) * a.H;
  cross_bwd_f32_kernel<D><<<unsigned(most < blocks ? most : blocks), kThreads, bytes, s>>>(a);
  return cuda_status(cudaGetLastError());
}

}  // namespace

cp_status launch_cross_bwd_f32(const CrossBwd& a, cudaStream_t s) {
  if (a.dtype != CP_F32) return CP_ERR_UNSUPPORTED;
  return a.d == 128 ? run<128>(a, s) : run<64>(a, s);
}

}  // namespace cpattn
