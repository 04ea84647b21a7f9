// Request tables of a paged K/V cache, and rows of heads on their way into it.
//
// kv_extend_kernel: request r holds have = ceil(len / p) pages and needs need =
//   ceil((len + add) / p) - have more.  One scan over the requests gives the
//   pages and rows before each of them; the requests in front of the first one
//   that does not fit (free pages, table width, rows) are granted.  Every block
//   repeats the scan (a few hundred requests: one step of 1024 threads) and
//   fills its own rows, so one launch does without a second pass over the
//   results; what bounds it is the chain of dependent loads, about 4 us.
// head_rows_kernel: a warp takes one row and a few of its heads.  The turn
//   of pair i at position n is n * turn[i] mod 1, exact in 64-bit integers
//   (turn is base^-e / 2 pi as a binary fraction, so the product wraps at whole
//   turns: no float64 and no range reduction), rounded once to float32 half
//   turns: the angle is off by at most 2^-25 half turns, 9.4e-8 rad.  Each lane forms two
//   pairs' sine and cosine and the lanes exchange them; every element is read
//   and written once, 16 bytes at a time.
#include <cuda_bf16.h>

#include "device_util.cuh"
#include "paged.h"
#include "tmap.h"

namespace cpattn {

namespace {

constexpr int kTabThreads = 1024;

// Inclusive scan of two values over the block (all threads call it).
__device__ __forceinline__ void block_scan2(int64_t& x, int64_t& y, int64_t* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, x, o), b = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += a;
      y += b;
    }
  }
  if (lane == 31) {
    sh[warp] = x;
    sh[32 + warp] = y;
  }
  __syncthreads();
  if (warp == 0) {
    int64_t u = sh[lane], w = sh[32 + lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, u, o), b = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) {
        u += a;
        w += b;
      }
    }
    sh[lane] = u;
    sh[32 + lane] = w;
  }
  __syncthreads();
  if (warp > 0) {
    x += sh[warp - 1];
    y += sh[32 + warp - 1];
  }
}

constexpr int kRowsPerTabBlock = 4096;

__global__ void __launch_bounds__(kTabThreads) kv_extend_kernel(KvTables a) {
  extern __shared__ int32_t sm[];  // [n_reqs] first row, [n_reqs] free pages taken before
  int32_t* s_cu = sm;
  int32_t* s_before = sm + a.n_reqs;
  __shared__ int64_t sh[64];
  __shared__ int s_stop;
  __shared__ int32_t s_rows;
  const int tid = threadIdx.x;
  const int32_t p = a.page_size;
  const int64_t n_free = min(int64_t(max(*a.n_free, 0)), int64_t(a.pool));
  if (tid == 0) s_stop = a.n_reqs;
  int64_t pages0 = 0, rows0 = 0;  // before this step of the scan
  for (int r0 = 0; r0 < a.n_reqs; r0 += kTabThreads) {
    const int r = r0 + tid;
    int64_t need = 0, add = 0;
    bool fits = true;
    if (r < a.n_reqs) {
      const int64_t len = a.lens[r], n = a.add[r];
      fits = len >= 0 && n >= 0;
      if (fits) {
        const int64_t have = (len + p - 1) / p, end = (len + n + p - 1) / p;
        need = end - have;
        add = n;
        fits = end <= a.max_blocks;
      }
    }
    int64_t x = need, y = add;
    __syncthreads();
    block_scan2(x, y, sh);
    if (r < a.n_reqs) {
      fits = fits && pages0 + x <= n_free && rows0 + y <= a.max_rows;
      if (!fits) atomicMin(&s_stop, r);
      // exact where the request is granted; behind the first refusal unused
      s_cu[r] = int32_t(min(rows0 + y - add, int64_t(INT32_MAX)));
      s_before[r] = int32_t(min(pages0 + x - need, int64_t(INT32_MAX)));
    }
    pages0 += sh[31];
    rows0 += sh[63];
  }
  __syncthreads();
  const int stop = s_stop;
  if (tid == 0) {
    s_rows = 0;
    if (stop > 0) s_rows = s_cu[stop - 1] + a.add[stop - 1];
  }
  __syncthreads();
  const int32_t rows = s_rows;
  // tables, lengths and row offsets: block b takes every gridDim.x-th request
  for (int r = blockIdx.x * kTabThreads + tid; r < a.n_reqs; r += gridDim.x * kTabThreads) {
    const bool ok = r < stop;
    const int32_t len = a.lens[r], add = ok ? a.add[r] : 0;
    a.lens_out[r] = len + add;
    a.cu[r] = ok ? s_cu[r] : rows;
    if (add > 0) {
      const int32_t have = int32_t((int64_t(len) + p - 1) / p);
      const int32_t end = int32_t((int64_t(len) + add + p - 1) / p);
      for (int32_t j = have; j < end; ++j)
        a.table[int64_t(r) * a.max_blocks + j] = a.free_pages[n_free - 1 - (s_before[r] + j - have)];
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.cu[a.n_reqs] = rows;
    int64_t taken = 0;
    if (stop > 0) {
      const int64_t len = a.lens[stop - 1];
      taken = s_before[stop - 1] + (len + a.add[stop - 1] + p - 1) / p - (len + p - 1) / p;
    }
    *a.n_free_out = int32_t(n_free - taken);
  }
  // rows: slot and position; -1 and 0 behind the last
  const int64_t t1 = min(a.max_rows, int64_t(blockIdx.x + 1) * kRowsPerTabBlock);
  for (int64_t t = int64_t(blockIdx.x) * kRowsPerTabBlock + tid; t < t1; t += kTabThreads) {
    int32_t slot = -1, pos = 0;
    if (t < rows) {
      // the last granted request that starts at or before t (requests that
      // add nothing start where the next does)
      int lo = 0, hi = stop - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_cu[mid] <= t) lo = mid; else hi = mid - 1;
      }
      const int32_t len = a.lens[lo];
      pos = len + int32_t(t - s_cu[lo]);
      const int32_t have = int32_t((int64_t(len) + p - 1) / p), b = pos / p;
      const int64_t page = b < have ? a.table[int64_t(lo) * a.max_blocks + b]
                                    : a.free_pages[n_free - 1 - (s_before[lo] + b - have)];
      const int64_t at = page * p + pos % p;
      if (page >= 0 && at <= INT32_MAX) slot = int32_t(at);
    }
    a.slots[t] = slot;
    a.pos[t] = pos;
  }
}

__global__ void __launch_bounds__(kTabThreads) kv_release_kernel(KvTables a) {
  __shared__ int64_t sh[64];
  const int tid = threadIdx.x;
  const int32_t p = a.page_size;
  const int64_t n_free = min(int64_t(max(*a.n_free, 0)), int64_t(a.pool));
  int64_t pages0 = 0;
  for (int r0 = 0; r0 < a.n_reqs; r0 += kTabThreads) {
    const int r = r0 + tid;
    int64_t have = 0;
    int32_t len = 0;
    bool done = false;
    if (r < a.n_reqs) {
      len = a.lens[r];
      done = a.add[r] != 0;
      if (done && len > 0) have = min((int64_t(len) + p - 1) / p, int64_t(a.max_blocks));
    }
    int64_t x = have, y = 0;
    __syncthreads();
    block_scan2(x, y, sh);
    if (r < a.n_reqs) {
      a.lens_out[r] = done ? 0 : len;
      const int64_t at = n_free + pages0 + x - have;
      for (int64_t j = 0; j < have; ++j) {
        int32_t* e = a.table + int64_t(r) * a.max_blocks + j;
        if (at + j < a.pool) a.free_pages[at + j] = *e;
        *e = -1;
      }
    }
    pages0 += sh[31];
  }
  if (tid == 0) *a.n_free_out = int32_t(min(n_free + pages0, int64_t(a.pool)));
}

template <typename T>
union Vec16 {
  uint4 u;
  T e[16 / sizeof(T)];
};
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float x, float& y) { y = x; }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16& y) { y = __float2bfloat16_rn(x); }

template <typename T, int D, bool kAdjacent>
__global__ void __launch_bounds__(256) head_rows_kernel(const __grid_constant__ HeadRows a, int32_t heads_per_task,
                                                        int32_t tasks_per_row, int64_t tasks) {
  constexpr int V = 16 / int(sizeof(T));  // elements of one load
  constexpr int LPH = D / 2 / V;          // lanes of a head: each holds two vectors
  constexpr int HPI = 32 / LPH;           // heads of one step of a warp
  const int lane = threadIdx.x & 31;
  const int c = lane % LPH, sub = lane / LPH;
  const int pairs = a.turns.pairs;
  const bool turns = c * V < pairs;
  // this lane's vectors: its pairs' two halves, or two vectors side by side
  const int off0 = (kAdjacent || !turns) ? 2 * c * V : c * V;
  const int off1 = (kAdjacent || !turns) ? off0 + V : pairs + c * V;
  const int heads = a.heads_q + a.heads_k + a.heads_v;
  const int64_t stride = (int64_t(gridDim.x) * blockDim.x) >> 5;
  for (int64_t task = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; task < tasks; task += stride) {
    const int64_t row = task / tasks_per_row;
    const int h0 = int(task - row * tasks_per_row) * heads_per_task;
    const int h1 = min(heads, h0 + heads_per_task);
    int64_t cache_off = 0;
    if (a.slots) {
      const int32_t slot = a.slots[row];
      const int32_t page = slot >> a.page_shift;
      if (slot < 0 || page >= a.n_pages) continue;
      cache_off = page * a.page_stride + int64_t(slot & ((1 << a.page_shift) - 1)) * a.token_stride;
    }
    float cs[V], sn[V];
    if (pairs > 0 && h0 < a.heads_q + a.heads_k) {
      float c2[D / 64], s2[D / 64];
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const int i = lane + 32 * j;
        float s_ = 0.f, c_ = 1.f;
        if (i < pairs) {
          const int64_t n = a.pos[int64_t(a.turns.axis[i]) * a.rows + row];
          const uint64_t t = uint64_t(n) * a.turns.turn[i];
          sincospif(float(int32_t(uint32_t(t >> 32))) * 4.656612873077393e-10f, &s_, &c_);  // * 2^-31: half turns
        }
        c2[j] = c_;
        s2[j] = a.turns.inverse ? -s_ : s_;
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int i = c * V + j;
        float x = __shfl_sync(0xffffffffu, c2[0], i & 31), y = __shfl_sync(0xffffffffu, s2[0], i & 31);
        if constexpr (D == 128) {
          const float x1 = __shfl_sync(0xffffffffu, c2[1], i & 31), y1 = __shfl_sync(0xffffffffu, s2[1], i & 31);
          if (i >= 32) {
            x = x1;
            y = y1;
          }
        }
        cs[j] = x;
        sn[j] = y;
      }
    }
    for (int h = h0 + sub; h < h1; h += HPI) {
      const T* src;
      T* dst;
      bool rotate = turns;
      if (h < a.heads_q) {
        src = static_cast<const T*>(a.q) + row * a.q_stride + int64_t(h) * D;
        dst = static_cast<T*>(a.q_out) + (row * a.heads_q + h) * D;
      } else if (h < a.heads_q + a.heads_k) {
        const int g = h - a.heads_q;
        src = static_cast<const T*>(a.k) + row * a.k_stride + int64_t(g) * D;
        dst = static_cast<T*>(a.k_out) + (a.slots ? cache_off + g * a.head_stride : (row * a.heads_k + g) * D);
      } else {
        const int g = h - a.heads_q - a.heads_k;
        src = static_cast<const T*>(a.v) + row * a.v_stride + int64_t(g) * D;
        dst = static_cast<T*>(a.v_out) + cache_off + g * a.head_stride;
        rotate = false;
      }
      const int o0 = rotate ? off0 : 2 * c * V;
      const int o1 = rotate ? off1 : 2 * c * V + V;
      Vec16<T> x0, x1;
      x0.u = *reinterpret_cast<const uint4*>(src + o0);
      x1.u = *reinterpret_cast<const uint4*>(src + o1);
      if (rotate) {
        if (kAdjacent) {
#pragma unroll
          for (int j = 0; j < V; ++j) {  // pair j: elements 2 j, 2 j + 1 of the lane's 2 V
            Vec16<T>& x = 2 * j < V ? x0 : x1;
            const int e = (2 * j) % V;
            const float u = to_f(x.e[e]), w = to_f(x.e[e + 1]);
            from_f(u * cs[j] - w * sn[j], x.e[e]);
            from_f(w * cs[j] + u * sn[j], x.e[e + 1]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float u = to_f(x0.e[j]), w = to_f(x1.e[j]);
            from_f(u * cs[j] - w * sn[j], x0.e[j]);
            from_f(w * cs[j] + u * sn[j], x1.e[j]);
          }
        }
      }
      *reinterpret_cast<uint4*>(dst + o0) = x0.u;
      *reinterpret_cast<uint4*>(dst + o1) = x1.u;
    }
  }
}

template <typename T, int D>
cp_status head_rows(const HeadRows& a, cudaStream_t s) {
  const int heads = a.heads_q + a.heads_k + a.heads_v;
  // few rows: one step of heads per warp, so that the rows spread over the SMs;
  // many rows: more heads share one set of sines and cosines
  const int per = a.rows >= 4096 ? 16 : 8;
  const int tasks_per_row = (heads + per - 1) / per;
  const int64_t tasks = a.rows * tasks_per_row;
  int64_t blocks = (tasks + 7) / 8;
  const int64_t cap = int64_t(num_sms()) * 8;
  if (blocks > cap) blocks = cap;
  auto* kern = a.turns.adjacent ? head_rows_kernel<T, D, true> : head_rows_kernel<T, D, false>;
  kern<<<unsigned(blocks), 256, 0, s>>>(a, per, tasks_per_row, tasks);
  return cuda_status(cudaGetLastError());
}

}  // namespace

cp_status launch_head_rows(const HeadRows& a, cp_dtype dtype, cudaStream_t s) {
  if (a.rows == 0 || a.heads_q + a.heads_k + a.heads_v == 0) return CP_OK;
  if (dtype == CP_BF16) return a.d == 128 ? head_rows<__nv_bfloat16, 128>(a, s) : head_rows<__nv_bfloat16, 64>(a, s);
  return a.d == 128 ? head_rows<float, 128>(a, s) : head_rows<float, 64>(a, s);
}

cp_status launch_kv_extend(const KvTables& a, cudaStream_t s) {
  const size_t smem = size_t(a.n_reqs) * 8;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kv_extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxTableReqs * 8) !=
          cudaSuccess)
    return CP_ERR_CUDA;
  const int64_t blocks = (a.max_rows + kRowsPerTabBlock - 1) / kRowsPerTabBlock;
  kv_extend_kernel<<<unsigned(blocks > 0 ? blocks : 1), kTabThreads, smem, s>>>(a);
  return cuda_status(cudaGetLastError());
}

cp_status launch_kv_release(const KvTables& a, cudaStream_t s) {
  kv_release_kernel<<<1, kTabThreads, 0, s>>>(a);
  return cuda_status(cudaGetLastError());
}

}  // namespace cpattn
