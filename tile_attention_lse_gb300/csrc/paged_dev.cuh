// Device side of the paged attention's work division: where a unit lies.
#pragma once

#include "paged.h"

namespace cpattn {

// Finds where the first unit of block c lies and returns the shares; the whole
// block calls it, `sh` holds 32 int64 and `out` a PagedStart in shared memory
// (not written where c has no first unit).  The threads share the requests in runs.
template <int U, int E, int kThreads>
__device__ __forceinline__ PagedShare paged_locate(const PagedArgs& a, int64_t* sh, PagedStart* out, int c) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (a.n_reqs + kThreads - 1) / kThreads;
  const int r0 = min(tid * run, a.n_reqs), r1 = min(r0 + run, a.n_reqs);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) mine += paged_req_units<U, E>(a, paged_req(a, r)) * a.Hkv;
  int64_t x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  int64_t total = 0, before = x - mine;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sh[w];
    total += sh[w];
  }
  const PagedShare share(total, a.grid);
  const int64_t u = share.first(c);
  if (u >= before && u < before + mine) {
    int64_t base = before;
    for (int r = r0; r < r1; ++r) {
      const PagedReq q = paged_req(a, r);
      const int64_t per = paged_req_units<U, E>(a, q);
      if (u >= base + per * a.Hkv) {
        base += per * a.Hkv;
        continue;
      }
      const int h = int(paged_div(u - base, per));
      int64_t rest = u - base - h * per;
      const int nt = paged_tiles(a, q);
      for (int t = 0; t < nt; ++t) {
        const int cost = paged_tile<U>(a, q, t).n + E;
        if (rest < cost) {
          *out = PagedStart{r, h, t, int32_t(rest)};
          break;
        }
        rest -= cost;
      }
      break;
    }
  }
  __syncthreads();
  return share;
}

// The merge kernel may start early; it waits for its predecessor here.
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace cpattn
