// Device side of the paged attention's work division (where a unit lies), and
// what its kernels share.
#pragma once

#include <type_traits>

#include "paged.h"

namespace cpattn {

// Tiles that a thread sums by itself; a request of more is summed by its whole warp.
constexpr int kOwnTiles = 16;

// Finds where the first unit of block c lies and returns the shares; the whole
// block calls it, `sh` holds 64 int64 and `out` a PagedStart in shared memory
// (not written where c has no first unit).  The threads share the requests in
// runs; the loops are warp-uniform so that lanes can help one another.
template <int U, int E, int kThreads, class A>
__device__ __forceinline__ PagedShare paged_locate(const A& a, int64_t* sh, PagedStart* out, int c) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (a.n_reqs + kThreads - 1) / kThreads;
  const int r0 = tid * run;
  // units of one kv-head of this lane's i-th request
  auto units = [&](const A& a, auto unit, auto extra, int i, PagedReq& q, int& nt) -> int64_t {
    constexpr int kU = decltype(unit)::value, kE = decltype(extra)::value;
    q = PagedReq{0, 0, 0};
    if (r0 + i < a.n_reqs) q = paged_req(a, r0 + i);
    nt = paged_tiles(a, q);
    int64_t s = 0;
    if (nt <= kOwnTiles)
      for (int t = 0; t < nt; ++t) s += paged_tile<kU>(a, q, t).n + kE;
    for (uint32_t big = __ballot_sync(0xffffffffu, nt > kOwnTiles); big; big &= big - 1) {
      const int from = __ffs(big) - 1;
      const PagedReq x{__shfl_sync(0xffffffffu, q.q0, from), __shfl_sync(0xffffffffu, q.nq, from),
                       __shfl_sync(0xffffffffu, q.kv, from)};
      const int n = __shfl_sync(0xffffffffu, nt, from);
      int64_t part = 0;
      for (int t = lane; t < n; t += 32) part += paged_tile<kU>(a, x, t).n + kE;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
      if (lane == from) s = part;
    }
    return s;
  };
  using Unit = std::integral_constant<int, U>;
  using Extra = std::integral_constant<int, E>;
  PagedReq q{};
  int nt = 0;
  int64_t mine = 0, last = 0, other = 0;
  for (int i = 0; i < run; ++i) {
    last = units(a, Unit{}, Extra{}, i, q, nt);
    mine += last * a.Hkv;
  }
  if (a.other_R > 0) {  // the other launch's units: how the SMs are divided
    const A b = paged_other(a);
    for (int i = 0; i < run; ++i) {
      PagedReq x;
      int n;
      other += units(b, std::integral_constant<int, PagedOther<U>::kUnit>{},
                     std::integral_constant<int, PagedOther<U>::kExtra>{}, i, x, n) * a.Hkv;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) other += __shfl_xor_sync(0xffffffffu, other, o);
    if (lane == 0) sh[32 + warp] = other;
  }
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
  int64_t others = 0;
  if (a.other_R > 0) {
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) others += sh[32 + w];
  }
  const PagedShare share(total, paged_blocks(a, U == kPairUnit, total, others));
  const int64_t u = share.first(c);
  const uint32_t who = __ballot_sync(0xffffffffu, u >= before && u < before + mine);
  if (who) {  // this warp holds it: its lane's requests, then the tiles of the one
    const int from = __ffs(who) - 1;
    int64_t base = before;
    bool found = false;
    int r = 0;
    for (int i = 0; i < run; ++i) {
      if (run > 1) last = units(a, Unit{}, Extra{}, i, q, nt);
      const bool here = lane == from && !found && u < base + last * a.Hkv;
      if (__any_sync(0xffffffffu, here)) {
        r = i;
        found = true;
        break;
      }
      base += last * a.Hkv;
    }
    base = __shfl_sync(0xffffffffu, base, from);
    const int64_t per = __shfl_sync(0xffffffffu, last, from);
    const PagedReq y{__shfl_sync(0xffffffffu, q.q0, from), __shfl_sync(0xffffffffu, q.nq, from),
                     __shfl_sync(0xffffffffu, q.kv, from)};
    const int n = __shfl_sync(0xffffffffu, nt, from);
    const int h = int(paged_div(u - base, per));
    int64_t rest = u - base - h * per;
    for (int t0 = 0; t0 < n; t0 += 32) {  // 32 tiles at a time
      const int cost = t0 + lane < n ? paged_tile<U>(a, y, t0 + lane).n + E : 0;
      int64_t upto = cost;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t z = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += z;
      }
      const uint32_t in = __ballot_sync(0xffffffffu, rest < upto);
      if (in) {
        if (lane == __ffs(in) - 1)
          *out = PagedStart{(warp * 32 + from) * run + r, h, t0 + lane, int32_t(rest - (upto - cost))};
        break;
      }
      rest -= __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  __syncthreads();
  return share;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool read) {
  const int n = read ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// The merge kernel may start early; it waits for its predecessor here.
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace cpattn
