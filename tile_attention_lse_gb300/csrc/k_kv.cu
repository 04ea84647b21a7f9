// Request tables of a paged K/V cache, and rows of heads on their way into it.
//
// kv_extend_kernel: request r holds have = ceil(len / p) pages and needs need =
//   ceil((len + add) / p) - have more.  One scan over the requests gives the
//   pages and rows before each of them; the requests in front of the first one
//   that does not fit (free pages, table width, rows) are granted.  Every block
//   repeats the scan (a few hundred requests: one step of 1024 threads) and
//   fills its own rows, so one launch does without a second pass over the
//   results; what bounds it is the chain of dependent loads, about 4 us.
// head_rows_kernel: a warp takes one row and a few heads of one tensor.  The turn
//   of pair i at position n is n * turn[i] mod 1, exact in 64-bit integers for
//   the table's turn (base^-e / 2 pi as a binary fraction, formed in float64 on the host, so the
//   product wraps at whole turns: no float64 and no range reduction here).  Its upper 32
//   bits become float32 half turns.  The angle is off by the rounding to float32, at most 2^-25
//   half turns (9.4e-8 rad), by 2^-32 turns for the bits cut off, and by the
//   position times the table's own error, 2^-53 turns for bases from 1 on (power, exponent,
//   1 / 2 pi and product: (4 + e ln base) 2^-53 of a turn of 0.16 base^-e): 7e-10 rad
//   at 2^20, 1.5e-6 at 2^31.  Each lane forms two
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

__global__ void __launch_bounds__(kTabThreads) kv_extend_kernel(KvTables a) {
  extern __shared__ int32_t sm[];  // [n_reqs] first row, [n_reqs] free pages taken before
  int32_t* s_cu = sm;
  int32_t* s_before = sm + a.n_reqs;
  __shared__ int64_t sh[64];
  __shared__ int s_stop;
  __shared__ int32_t s_rows, s_taken;
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
    s_rows = s_taken = 0;
    if (stop > 0) {
      const int64_t len = a.lens[stop - 1], n = a.add[stop - 1];
      s_rows = s_cu[stop - 1] + int32_t(n);
      s_taken = s_before[stop - 1] + int32_t((len + n + p - 1) / p - (len + p - 1) / p);
    }
  }
  __syncthreads();
  const int32_t rows = s_rows, taken = s_taken;
  // the last granted request whose entry of `from` is at most x (requests that
  // add nothing share theirs with the next)
  auto find = [&](const int32_t* from, int64_t x) {
    int lo = 0, hi = stop - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (from[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  const int32_t stride = gridDim.x * kTabThreads, first = blockIdx.x * kTabThreads + tid;
  for (int r = first; r < a.n_reqs; r += stride) {
    const bool ok = r < stop;
    a.lens_out[r] = a.lens[r] + (ok ? a.add[r] : 0);
    a.cu[r] = ok ? s_cu[r] : rows;
  }
  for (int64_t i = first; i < taken; i += stride) {  // page i of those taken
    const int r = find(s_before, i);
    const int32_t have = int32_t((int64_t(a.lens[r]) + p - 1) / p);
    a.table[int64_t(r) * a.max_blocks + have + i - s_before[r]] = a.free_pages[n_free - 1 - i];
  }
  if (first == 0) {
    a.cu[a.n_reqs] = rows;
    *a.n_free_out = int32_t(n_free - taken);
  }
  // rows: slot and position; -1 and 0 behind the last
  for (int64_t t = first; t < a.max_rows; t += stride) {
    int32_t slot = -1, pos = 0;
    if (t < rows) {
      const int lo = find(s_cu, t);
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

// A thread a request: its entries at or above zero are counted, the scan gives
// their place in the pool, and they move there in table order (one below
// zero holds no page: it was given back before).  A load cannot pass the stores
// in front of it, so 16 entries are read at a time, the first 16 once for both
// (256 requests of 2000 tokens in pages of 16: 46 us, one of 131072: 400; 8 at
// a time 48 and 490).  One block: its long requests are bound by their threads'
// chains of loads.
__global__ void __launch_bounds__(kTabThreads) kv_release_kernel(KvTables a) {
  __shared__ int64_t sh[64];
  constexpr int kAhead = 16;
  const int tid = threadIdx.x;
  const int32_t p = a.page_size;
  const int64_t n_free = min(int64_t(max(*a.n_free, 0)), int64_t(a.pool));
  int64_t pages0 = 0;
  for (int r0 = 0; r0 < a.n_reqs; r0 += kTabThreads) {
    const int r = r0 + tid;
    int32_t have = 0, given = 0, len = 0;
    bool done = false;
    int32_t* row = a.table + int64_t(r) * a.max_blocks;
    int32_t page[kAhead];
    auto load = [&](int32_t j0) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) page[j] = j0 + j < have ? row[j0 + j] : -1;
    };
    if (r < a.n_reqs) {
      len = a.lens[r];
      done = a.add[r] != 0;
      if (done && len > 0) have = int32_t(min((int64_t(len) + p - 1) / p, int64_t(a.max_blocks)));
    }
    for (int32_t j0 = (have - 1) / kAhead * kAhead; j0 >= 0; j0 -= kAhead) {  // the first ones last: they stay
      load(j0);
#pragma unroll
      for (int j = 0; j < kAhead; ++j) given += page[j] >= 0;
    }
    int64_t x = given, y = 0;
    __syncthreads();
    block_scan2(x, y, sh);
    if (r < a.n_reqs) {
      a.lens_out[r] = done ? 0 : len;
      int32_t at = int32_t(min(n_free + pages0 + x - given, int64_t(a.pool)));
      for (int32_t j0 = 0; j0 < have; j0 += kAhead) {
        if (j0 > 0) load(j0);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (j0 + j >= have) break;
          row[j0 + j] = -1;
          const bool put = page[j] >= 0 && at < a.pool;
          if (put) a.free_pages[at] = page[j];
          at += put;
        }
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

// Sine and cosine of `turn` / 2^32 turns.  bfloat16 takes the hardware's (off
// by 2^-21 at most for angles within a half turn either way, 2^-13 of the
// output's own rounding), float32 the accurate ones.
template <typename T>
__device__ __forceinline__ void turn_sincos(int32_t turn, float* s, float* c) {
  if constexpr (sizeof(T) == 2)
    __sincosf(float(turn) * 1.4629180792671596e-9f, s, c);  // * 2 pi / 2^32
  else
    sincospif(float(turn) * 4.656612873077393e-10f, s, c);  // * 2^-31: half turns
}

// Tasks of a row: its q heads, k heads and v heads, `per` at a time.
struct RowTasks {
  int32_t per, of_q, of_k, all;
};

constexpr int kRowBlocks = 4;  // resident blocks of 256 threads: 64 registers

template <typename T, int D, bool kAdjacent>
__global__ void __launch_bounds__(256, kRowBlocks) head_rows_kernel(const __grid_constant__ HeadRows a, RowTasks rt, int64_t tasks) {
  constexpr int V = 16 / int(sizeof(T));  // elements of one load
  constexpr int LPH = D / 2 / V;          // lanes of a head: each holds two vectors
  constexpr int HPI = 32 / LPH;           // heads of one step of a warp
  const int lane = threadIdx.x & 31;
  const int c = lane % LPH, sub = lane / LPH;
  const int pairs = a.turns.pairs;
  // this lane's pairs' turns and positions (by lane from constant memory: once)
  uint64_t turn[D / 64];
  const int32_t* pos[D / 64];
#pragma unroll
  for (int j = 0; j < D / 64; ++j) {
    const int i = min(lane + 32 * j, 63);
    turn[j] = a.turns.turn[i];
    pos[j] = lane + 32 * j < pairs ? a.pos + int64_t(a.turns.axis[i]) * a.rows : nullptr;
  }
  const int64_t stride = (int64_t(gridDim.x) * blockDim.x) >> 5;
  // a row's tasks differ in length: where a warp would always meet the same
  // kind, it moves on by one each time (its row's tasks are all in this step then)
  const int turn_by = stride % rt.all == 0 ? 1 : 0;
  int skew = 0;
  for (int64_t task = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; task < tasks; task += stride) {
    const int64_t row = tasks >> 31 ? task / rt.all : int64_t(uint32_t(task) / uint32_t(rt.all));
    int part = int(task - row * rt.all) + skew;
    if (part >= rt.all) part -= rt.all;
    skew = skew + turn_by == rt.all ? 0 : skew + turn_by;
    int64_t cache_off = 0;
    if (a.slots) {
      const int32_t slot = a.slots[row];
      const int32_t page = slot >> a.page_shift;
      if (slot < 0 || page >= a.n_pages) continue;
      cache_off = page * a.page_stride + int64_t(slot & ((1 << a.page_shift) - 1)) * a.token_stride;
    }
    // the task's heads of one tensor
    const T* src;
    T* dst;
    int64_t step = D;  // elements between heads of dst
    int heads;
    const bool of_v = part >= rt.of_q + rt.of_k;
    if (part < rt.of_q) {
      heads = a.heads_q;
      src = static_cast<const T*>(a.q) + row * a.q_stride;
      dst = static_cast<T*>(a.q_out) + row * a.heads_q * D;
    } else if (!of_v) {
      part -= rt.of_q;
      heads = a.heads_k;
      src = static_cast<const T*>(a.k) + row * a.k_stride;
      dst = static_cast<T*>(a.k_out) + (a.slots ? cache_off : row * a.heads_k * D);
      if (a.slots) step = a.head_stride;
    } else {
      part -= rt.of_q + rt.of_k;
      heads = a.heads_v;
      src = static_cast<const T*>(a.v) + row * a.v_stride;
      dst = static_cast<T*>(a.v_out) + cache_off;
      step = a.head_stride;
    }
    const bool rotate = !of_v && c * V < pairs;
    // this lane's vectors: its pairs' two halves, or two vectors side by side
    const int off0 = kAdjacent || !rotate ? 2 * c * V : c * V;
    const int off1 = kAdjacent || !rotate ? off0 + V : pairs + c * V;
    const int h1 = min(heads, (part + 1) * rt.per);
    int h = part * rt.per + sub;
    // the loads of a step of heads are under way while the angles are formed,
    // and then while the step before it is turned
    Vec16<T> n0, n1;
    auto load = [&](int at) {
      if (at < h1) {
        n0.u = *reinterpret_cast<const uint4*>(src + at * D + off0);
        n1.u = *reinterpret_cast<const uint4*>(src + at * D + off1);
      }
    };
    load(h);
    float cs[V], sn[V];
    if (!of_v && pairs > 0) {
      float c2[D / 64], s2[D / 64];
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        float s_ = 0.f, c_ = 1.f;
        if (pos[j]) {
          const int64_t n = pos[j][row];
          turn_sincos<T>(int32_t(uint32_t((uint64_t(n) * turn[j]) >> 32)), &s_, &c_);
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
    for (; h < h1; h += HPI) {
      Vec16<T> x0 = n0, x1 = n1;
      load(h + HPI);
      if (rotate) {
        if (kAdjacent) {
#pragma unroll
          for (int j = 0; j < V; ++j) {  // pair j: elements 2 j, 2 j + 1 of the lane's 2 V
            Vec16<T>& x = 2 * j < V ? x0 : x1;
            const int e = (2 * j) % V;
            const float y = to_f(x.e[e]), w = to_f(x.e[e + 1]);
            from_f(y * cs[j] - w * sn[j], x.e[e]);
            from_f(w * cs[j] + y * sn[j], x.e[e + 1]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float y = to_f(x0.e[j]), w = to_f(x1.e[j]);
            from_f(y * cs[j] - w * sn[j], x0.e[j]);
            from_f(w * cs[j] + y * sn[j], x1.e[j]);
          }
        }
      }
      *reinterpret_cast<uint4*>(dst + h * step + off0) = x0.u;
      *reinterpret_cast<uint4*>(dst + h * step + off1) = x1.u;
    }
  }
}

template <typename T, int D>
cp_status head_rows(const HeadRows& a, cudaStream_t s) {
  // few rows: one or two steps of heads per warp, so that the rows spread over
  // the SMs; many rows: more heads share one set of sines and cosines.  Rotation
  // of 32/8 heads of 128, 8 and 16 heads a task: bf16 64 rows 3.7 and 4.2 us, 2048 rows 13.1
  // and 13.7, 4096 19.8 and 18.5, 32768 116 and 106; float32 64 rows 4.6 and 5.4, 2048
  // 19.5 and 20.5, 4096 32.2 and 31.7, 32768 211 and 215.
  RowTasks rt;
  rt.per = a.rows >= 4096 ? 16 : 8;
  rt.of_q = (a.heads_q + rt.per - 1) / rt.per;
  rt.of_k = (a.heads_k + rt.per - 1) / rt.per;
  rt.all = rt.of_q + rt.of_k + (a.heads_v + rt.per - 1) / rt.per;
  const int64_t tasks = a.rows * rt.all;
  int64_t blocks = (tasks + 7) / 8;
  const int64_t cap = int64_t(num_sms()) * kRowBlocks;
  if (blocks > cap) blocks = cap;
  auto* kern = a.turns.adjacent ? head_rows_kernel<T, D, true> : head_rows_kernel<T, D, false>;
  kern<<<unsigned(blocks), 256, 0, s>>>(a, rt, tasks);
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
  // what needs no opt-in is 48 KB of dynamic and static shared memory together;
  // the kernel's static arrays are less than 1 KB
  if (smem > 47 * 1024 &&
      cudaFuncSetAttribute(kv_extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxTableReqs * 8) !=
          cudaSuccess)
    return CP_ERR_CUDA;
  int64_t blocks = (a.max_rows + kTabThreads - 1) / kTabThreads;
  const int64_t cap = int64_t(num_sms()) * 2;
  blocks = blocks < 1 ? 1 : blocks > cap ? cap : blocks;
  kv_extend_kernel<<<unsigned(blocks), kTabThreads, smem, s>>>(a);
  return cuda_status(cudaGetLastError());
}

cp_status launch_kv_release(const KvTables& a, cudaStream_t s) {
  kv_release_kernel<<<1, kTabThreads, 0, s>>>(a);
  return cuda_status(cudaGetLastError());
}

}  // namespace cpattn
