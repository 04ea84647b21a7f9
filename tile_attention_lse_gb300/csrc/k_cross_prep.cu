// What cross attention makes ready before its products and brings home behind
// them: the bias table spread over the relative positions; for the backward the
// lists of tiles, D and L2, zeros; dQ from its float32 sums and the sums of the
// table's gradient.
#include <cuda_bf16.h>

#include "cross.h"
#include "device_util.cuh"
#include "paged_dev.cuh"
#include "tc_util.cuh"
#include "tmap.h"

namespace cpattn {

namespace {

// Bucket of a relative position.
__device__ __forceinline__ int rel_bucket(const RelStarts& s, int x) {
  const int away = s.both ? abs(x) : max(-x, 0);
  int lo = 0, hi = s.per;  // start[lo] <= away; start[hi], if there is one, is not
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s.start[mid] <= away)
      lo = mid;
    else
      hi = mid;
  }
  return lo + (s.both && x > 0 ? s.per : 0);
}

// rel[h][x] = log2(e) table[bucket(x)][h].  A word a thread, written side by side;
// the table is read from the caches.
template <typename T>
__global__ void __launch_bounds__(256) rel_spread_kernel(const __grid_constant__ RelSpread a) {
  grid_launch_dependents();
  const int i = int(blockIdx.x) * 256 + int(threadIdx.x), h = int(blockIdx.y);
  if (i >= a.rel_stride) return;
  const int b = rel_bucket(a.starts, i - a.rel_zero);
  float x;
  load_vec<T, 1>(static_cast<const T*>(a.table) + int64_t(b) * a.heads + h, &x);
  // entries that stand for "never" do so exactly, whatever is added to them
  a.rel[int64_t(h) * a.rel_stride + i] = x < -1e30f ? -INFINITY : x * 1.4426950408889634f;
}

// ---------------------------------------------------------- tile lists ---
constexpr int kListThreads = 512, kBins = 512;

// Tiles of a sequence, and the cost of one: the other side's tiles that it meets, and 1.
__device__ __forceinline__ int list_tiles(const PagedReq& q, bool of_k, int size) {
  return ((of_k ? q.kv : q.nq) + size - 1) / size;
}
__device__ __forceinline__ int list_cost(const CrossBwd& a, const PagedReq& q, bool of_k, int first, int size) {
  if (of_k) return (q.nq - cross_first_query(a, q, first) + size - 1) / size + 1;
  int seen = q.kv;
  if (a.causal) seen = clamp_i32(first + size + q.kv - q.nq, 0, q.kv);
  return (seen + size - 1) / size + 1;
}

// One block lists all tiles, the costly ones first (a counting sort by cost; what it puts
// side by side within a cost is not ordered, and nothing depends on that but which
// block runs a tile).  Sequences are taken kListThreads at a time, tiles found by bisection.
__device__ void list_block(const CrossBwd& a, const CrossTiles& to, bool of_k) {
  __shared__ int s_upto[kListThreads];  // tiles up to and with the sequence
  __shared__ int s_bin[kBins], s_warp[kListThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kBins; i += kListThreads) s_bin[i] = 0;
  int total = 0;
  for (int pass = 0; pass < 2; ++pass) {  // counts, then places
    int base = 0;
    for (int r0 = 0; r0 < a.n_reqs; r0 += kListThreads) {
      int n = 0;
      if (r0 + tid < a.n_reqs) n = list_tiles(paged_req(a, r0 + tid), of_k, to.size);
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();
      if (lane == 31) s_warp[warp] = x;
      __syncthreads();
      int before = 0, all = 0;
      for (int w = 0; w < kListThreads / 32; ++w) {
        if (w < warp) before += s_warp[w];
        all += s_warp[w];
      }
      s_upto[tid] = before + x;
      __syncthreads();
      for (int t = tid; t < all; t += kListThreads) {
        int lo = 0, hi = kListThreads - 1;  // the first sequence whose tiles go beyond t
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (s_upto[mid] > t)
            hi = mid;
          else
            lo = mid + 1;
        }
        const int first = (t - (lo > 0 ? s_upto[lo - 1] : 0)) * to.size;
        const int cost = list_cost(a, paged_req(a, r0 + lo), of_k, first, to.size);
        const int bin = kBins - 1 - min(cost, kBins - 1);
        const int at = atomicAdd(&s_bin[bin], 1);
        // (a place and an id within the list whatever cu_q and cu_k hold)
        if (pass == 1 && at < to.most) to.list[at] = CrossTile{r0 + lo, first, min(base + t, to.most - 1), 0};
      }
      base += all;
      __syncthreads();
    }
    total = base;
    if (pass == 0) {  // where each bin begins
      __syncthreads();
      int x = s_bin[tid];
      const int own = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) s_warp[warp] = x;
      __syncthreads();
      int before = 0;
      for (int w = 0; w < warp; ++w) before += s_warp[w];
      s_bin[tid] = before + x - own;
      __syncthreads();
    }
  }
  if (tid == 0) *to.count = min(total, to.most);
}
static_assert(kBins == kListThreads, "a thread a bin");

// Quotient of numbers of rows; the 32-bit division where both fit is several times faster.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  return ((x | y) >> 31) == 0 ? int64_t(uint32_t(x) / uint32_t(y)) : x / y;
}

// ------------------------------------------------------------ D and L2 ---
// A (row, head) of d elements is kLanes lanes of 16 bytes; a warp has two such groups
// under way.  Bound by the bytes of o and dO and of the sums' zeros (9335 rows of 32 heads of 128: 306 MB, 55 us).
template <typename T, int D>
__device__ __forceinline__ void delta_rows(const CrossBwd& a, int64_t warp, int64_t n_warps) {
  constexpr int kVec = 16 / int(sizeof(T)), kLanes = D / kVec, kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31, sub = lane / kLanes, sl = lane % kLanes;
  const int64_t n = a.rows * a.H;
  const float keep = 1.f / a.drop_scale;
  for (int64_t r0 = warp * 2 * kRows; r0 < n; r0 += n_warps * 2 * kRows) {
    float x[2][kVec], y[2][kVec], z[2][kVec];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t rh = r0 + u * kRows + sub;
      if (rh < n) {
        const int64_t row = quotient(rh, a.H), h = rh - row * a.H;
        load_vec<T, kVec>(static_cast<const T*>(a.o) + rh * D + sl * kVec, x[u]);
        load_vec<T, kVec>(static_cast<const T*>(a.dout) + row * a.do_stride + h * D + sl * kVec, y[u]);
        if (sizeof(T) == 2 && a.rest) {
          load_vec<T, kVec>(static_cast<const T*>(a.rest) + rh * D + sl * kVec, z[u]);
#pragma unroll
          for (int i = 0; i < kVec; ++i) x[u][i] += z[u][i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[u][i] = y[u][i] = 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t rh = r0 + u * kRows + sub;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kVec; ++i) sum = fmaf(x[u][i], y[u][i], sum);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (rh >= n) continue;
      const int64_t row = quotient(rh, a.H), h = rh - row * a.H;
      if (a.dq_acc) {
        float4* zero = reinterpret_cast<float4*>(a.dq_acc + (h * a.rows + row) * D);
        for (int i = sl; i < D / 4; i += kLanes) zero[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (sl == 0) {
        const float l = a.lse[rh];
        a.delta[h * a.rows + row] = sum * keep;
        a.lse2[h * a.rows + row] = l == -INFINITY ? INFINITY : l * 1.4426950408889634f;
      }
    }
  }
}

// Zeros in rows lo .. hi - 1 of a [rows][width] tensor.
template <typename T>
__device__ __forceinline__ void zero_rows(void* x, int64_t lo, int64_t hi, int64_t width, int64_t t, int64_t n) {
  uint4* to = reinterpret_cast<uint4*>(static_cast<T*>(x) + lo * width);
  const int64_t n16 = (hi - lo) * width * int64_t(sizeof(T)) / 16;
  for (int64_t i = t; i < n16; i += n) to[i] = make_uint4(0, 0, 0, 0);
}

// Blocks 0 and 1 list tiles; the others form D and L2, and clear the gradients' rows that no sequence owns.
template <typename T, int D>
__global__ void __launch_bounds__(kListThreads) cross_bwd_prep_kernel(const __grid_constant__ CrossBwd a) {
  if (blockIdx.x == 0) return list_block(a, a.k_tiles, true);
  if (blockIdx.x == 1) {
    if (a.q_tiles.most > 0) list_block(a, a.q_tiles, false);
    return;
  }
  const int64_t block = blockIdx.x - 2, blocks = gridDim.x - 2;
  delta_rows<T, D>(a, block * (kListThreads / 32) + (threadIdx.x >> 5), blocks * (kListThreads / 32));
  // gap g lies behind the keys (queries) of sequence g - 1, gap 0 before the first: a
  // block each, and all blocks for the last one (a tensor longer than its sequences)
  const int64_t kw = int64_t(a.Hkv) * D, qw = int64_t(a.H) * D;
  auto clear = [&](int g, int64_t t, int64_t n) {
    int64_t klo = 0, qlo = 0;
    if (g > 0) {
      const PagedReq q = paged_req(a, g - 1);
      klo = paged_key_row(a, g - 1) + q.kv;
      qlo = q.q0 + q.nq;
    }
    const int64_t khi = g < a.n_reqs ? paged_key_row(a, g) : a.rows_k;
    const int64_t qhi = g < a.n_reqs ? clamp_i32(a.cu[g], 0, int32_t(a.rows)) : a.rows;
    if (khi > klo) {
      zero_rows<T>(a.dk, klo, khi, kw, t, n);
      zero_rows<T>(a.dv, klo, khi, kw, t, n);
    }
    if (!a.dq_acc && qhi > qlo) zero_rows<T>(a.dq, qlo, qhi, qw, t, n);
  };
  for (int64_t g = block; g < a.n_reqs; g += blocks) clear(int(g), threadIdx.x, kListThreads);
  clear(a.n_reqs, block * kListThreads + threadIdx.x, blocks * kListThreads);
}

// ---------------------------------------------------------------- behind ---
// dQ = scale r sums, from [H][rows][d] to [rows][H][d] (four float4 a thread under way),
// and the table's gradient: one block a head, its partial sums in the order of the key tiles.
constexpr int kPostThreads = 512;

template <int D>
__device__ __forceinline__ void dq_rows(const CrossBwd& a, int64_t block, int64_t blocks) {
  const int64_t n4 = a.rows * a.H * (D / 4), stride = blocks * kPostThreads;
  const float mul = a.scale * a.drop_scale;
  const float4* acc = reinterpret_cast<const float4*>(a.dq_acc);
  for (int64_t i0 = block * kPostThreads + threadIdx.x; i0 < n4; i0 += 4 * stride) {
    float4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) x[u] = i0 + u * stride < n4 ? acc[i0 + u * stride] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t i = i0 + u * stride;
      if (i >= n4) break;
      const int64_t hr = i / (D / 4), h = quotient(hr, a.rows), row = hr - h * a.rows;
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.dq) + (row * a.H + h) * D + (i % (D / 4)) * 4) =
          make_uint2(tc::pack_bf16x2(x[u].x * mul, x[u].y * mul), tc::pack_bf16x2(x[u].z * mul, x[u].w * mul));
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kPostThreads) cross_bwd_post_kernel(const __grid_constant__ CrossBwd a, int table_blocks) {
  if (int(blockIdx.x) >= table_blocks) {
    if constexpr (sizeof(T) == 2) dq_rows<D>(a, blockIdx.x - table_blocks, gridDim.x - table_blocks);
    return;
  }
  // Bound by the latency of its loads: a thread has eight under way (16 heads, 136 key tiles: 86 us with
  // 256 threads and four).
  __shared__ float s_sum[kPostThreads];
  const int h = blockIdx.x, bs = a.bucket_stride, b = threadIdx.x % bs, s = threadIdx.x / bs, ns = kPostThreads / bs;
  const uint32_t parts = uint32_t(a.parts), n = uint32_t(*a.k_tiles.count) * parts;  // parts: a power of two
  const int shift = 31 - __clz(int(parts));
  float sum[8] = {};
  for (uint32_t i = s; i < n; i += 8 * ns) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t e = i + u * ns;
      if (e < n) sum[u] += a.part[((int64_t(e >> shift) * a.H + h) * parts + (e & (parts - 1))) * bs + b];
    }
  }
  s_sum[threadIdx.x] = ((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7]));
  __syncthreads();
  if (s > 0 || b >= a.buckets) return;
  float x = 0.f;
  for (int i = 0; i < ns; ++i) x += s_sum[i * bs + b];
  x *= a.drop_scale;
  store_vec<T, 1>(static_cast<T*>(a.dtable) + int64_t(b) * a.H + h, &x);
}

template <typename T, int D>
cp_status run_prep(const CrossBwd& a, cudaStream_t s) {
  const int64_t per = 2 * (kListThreads / 32) * (32 * 16 / int(sizeof(T)) / D);  // (row, head)s of a block's step
  int64_t blocks = (a.rows * a.H + per - 1) / per;
  const int64_t gaps = (a.rows_k * a.Hkv * D * int64_t(sizeof(T)) / 16 + kListThreads * 8 - 1) / (kListThreads * 8);
  blocks = blocks > gaps ? blocks : gaps;
  const int64_t most = int64_t(num_sms()) * 4;
  blocks = blocks > most ? most : (blocks < 1 ? 1 : blocks);
  cross_bwd_prep_kernel<T, D><<<unsigned(2 + blocks), kListThreads, 0, s>>>(a);
  return cuda_status(cudaGetLastError());
}

template <typename T, int D>
cp_status run_post(const CrossBwd& a, cudaStream_t s) {
  const int tables = a.rel ? a.H : 0;
  int64_t blocks = sizeof(T) == 2 ? (a.rows * a.H * (D / 4) + 4 * kPostThreads - 1) / (4 * kPostThreads) : 0;
  const int64_t most = int64_t(num_sms()) * 4;
  blocks = blocks > most ? most : blocks;
  if (tables + blocks == 0) return CP_OK;
  cross_bwd_post_kernel<T, D><<<unsigned(tables + blocks), kPostThreads, 0, s>>>(a, tables);
  return cuda_status(cudaGetLastError());
}

}  // namespace

cp_status launch_rel_spread(const RelSpread& a, cp_dtype dtype, cudaStream_t s) {
  const dim3 grid(unsigned((a.rel_stride + 255) / 256), unsigned(a.heads));
  if (dtype == CP_BF16)
    rel_spread_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a);
  else
    rel_spread_kernel<float><<<grid, 256, 0, s>>>(a);
  return cuda_status(cudaGetLastError());
}

cp_status launch_cross_bwd_prep(const CrossBwd& a, cudaStream_t s) {
  if (a.dtype == CP_BF16) return a.d == 128 ? run_prep<__nv_bfloat16, 128>(a, s) : run_prep<__nv_bfloat16, 64>(a, s);
  return a.d == 128 ? run_prep<float, 128>(a, s) : run_prep<float, 64>(a, s);
}

cp_status launch_cross_bwd_post(const CrossBwd& a, cudaStream_t s) {
  if (a.dtype == CP_BF16) return a.d == 128 ? run_post<__nv_bfloat16, 128>(a, s) : run_post<__nv_bfloat16, 64>(a, s);
  return a.d == 128 ? run_post<float, 128>(a, s) : run_post<float, 64>(a, s);
}

}  // namespace cpattn
