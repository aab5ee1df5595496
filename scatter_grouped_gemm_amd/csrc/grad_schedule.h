// Which tiles of the weight gradient (gemm_grad.hip) a workgroup takes.
//
// Every expert has the same number of 256 x 256 tiles, and a tile of expert e
// costs steps(e), its rows over 64.  With popular experts a tile may cost as much
// as the average workgroup's whole share, so the tiles have to be dealt by cost.
// All of it is worked out by every workgroup from the row counts (no memory of
// the caller's, no atomics: two calls at once do not meet), in a few microseconds:
//   - Experts in order of falling row counts.  The tiles of an expert are cut in
//     eight contiguous shares, one per XCD (expert s starts with XCD -s, so that
//     odd ones even out).
//   - P workgroups of an XCD.  Whole rounds of P tiles of a share go to all of
//     them, side by side: they share panels of dC and A through the XCD's L2.
//   - The remainders of all shares form one list of items of falling cost.  Item
//     b < P goes to workgroup b; the rest is poured over them as water over
//     steps: first the workgroup with the smallest item takes items until it
//     has as much as the next one, then the two take them in turn until they have
//     as much as the third, and so on.  tm[m - 1] .. tm[m] are the items that m
//     workgroups take in turn.
// Measured (64 experts, 2048 x 1408 fp32 gradients added to, rows by a power law of
// exponent 1.2 with eight experts empty): 449 us; every 32nd tile to a workgroup
// 538; the items dealt from the first workgroup on at each level 518.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_runs.h"

namespace moe {
namespace sched {

constexpr int kMaxG = 1024;
constexpr int kMaxP = 64;       // workgroups of an XCD

struct Lds {
  int2 range[kMaxG];            // (first row, rows), rows falling
  int id[kMaxG];
  int items[kMaxG + kMaxP];     // items before expert s (the total from the last one on)
  int cost[kMaxG + kMaxP];      // and their cost
  int tm[kMaxP + 1];
  int scr[16];
};

// Hand-written reads, as the run table's in gemm_runs.h and for its reason.
__device__ __forceinline__ int lds_int(const int* p) {
  int v;
  asm volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=v"(v) : "v"(runs::lds_off(p)) : "memory");
  return v;
}
__device__ __forceinline__ int2 lds_int2(const int2* p) {
  int2 v;
  asm volatile("ds_read_b64 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=v"(v) : "v"(runs::lds_off(p)) : "memory");
  return v;
}
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

__device__ __forceinline__ int tile_steps(int rows, int step) {
  return rows > 0 ? (rows + 2 * step - 1) / (2 * step) * 2 : 2;
}

// Tiles [lo, lo + n) of expert s (in falling order) that XCD x takes.
__device__ __forceinline__ int2 share(int s, int x, int64_t tiles) {
  const int y = (x + s) & 7;
  const int lo = static_cast<int>((y * tiles) >> 3);
  return make_int2(lo, static_cast<int>(((y + 1) * tiles) >> 3) - lo);
}

struct Dealer {
  Lds* L;
  int G, P, w, xcd, tiles, total;
  int s, k;      // whole rounds: expert, round
  int m, t;      // items: workgroups that take them in turn (0: none taken yet), next one
  int at;        // the expert search goes on from here
};

// Sets up the dealing: all 64 * WAVES threads call it, `raw` is kMaxG int2 of LDS
// to work in.  A tile costs its steps and tile_cost.  skip_empty: experts without rows have no tiles.
template <int WAVES>
__device__ __forceinline__ void deal(Dealer& d, Lds* L, int2* raw, const int32_t* __restrict__ starts,
                                     const int32_t* __restrict__ counts, int64_t M, int G, int tiles,
                                     int step, int tile_cost, bool skip_empty) {
  constexpr int kThreads = 64 * WAVES;
  static_assert(2 * kThreads >= kMaxG && kThreads >= kMaxP + 1, "a thread has two experts");
  const int tid = threadIdx.x;
  const int P = static_cast<int>(gridDim.x >> 3), xcd = blockIdx.x & 7;
  for (int e = tid; e < G; e += kThreads) {
    int64_t s = starts[e], n = counts[e];
    if (s < 0 || s > M || n < 0) s = 0, n = 0;
    n = n < M - s ? n : M - s;
    raw[e] = make_int2(static_cast<int>(s), static_cast<int>(n));
  }
  __syncthreads();
  int live = 0;
  for (int e = tid; e < G; e += kThreads) {
    const int2 r = raw[e];
    int rank = 0;
    for (int j = 0; j < G; ++j) {
      const int n = raw[j].y;
      rank += n > r.y || (n == r.y && j < e);
    }
    L->range[rank] = r;
    L->id[rank] = e;
    live += r.y > 0;
  }
  int2 tot = make_int2(G, 0);
  if (skip_empty) runs::scan_excl_sum2<WAVES>(live, 0, L->scr, tot);
  d.G = uniform(tot.x);
  __syncthreads();
  int r[2], c[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = 2 * tid + i;
    r[i] = s < d.G ? share(s, xcd, tiles).y % P : 0;
    c[i] = r[i] > 0 ? r[i] * (tile_steps(L->range[s].y, step) + tile_cost) : 0;
  }
  const int2 base = runs::scan_excl_sum2<WAVES>(r[0] + r[1], c[0] + c[1], L->scr, tot);
  if (2 * tid < kMaxG) {
    L->items[2 * tid] = base.x;
    L->items[2 * tid + 1] = base.x + r[0];
    L->cost[2 * tid] = base.y;
    L->cost[2 * tid + 1] = base.y + c[0];
  }
  if (tid < kMaxP) {
    L->items[kMaxG + tid] = tot.x;
    L->cost[kMaxG + tid] = tot.y;
  }
  __syncthreads();
  // last s with a[s] <= x, of the experts that have items
  auto last = [&](const int* a, int x) -> int {
    int lo = 0, hi = d.G;  // a[lo] <= x; a[hi] is the total
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a[mid] <= x) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  if (tid < 64) {
    const int b = tid;
    int load = 0;
    if (b < P && b < tot.x) load = tile_steps(L->range[last(L->items, b)].y, step) + tile_cost;
    int sum = load;  // of the workgroups from b on (smaller items)
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_down(sum, off, 64);
      if (b + off < 64) sum += o;
    }
    const int before = __shfl(sum, 0, 64);  // cost of the first items
    if (b < P) {
      const int rho = P - 1 - b;
      const int x = before + rho * load - (sum - load);
      int t = tot.x;
      if (x < tot.y) {
        const int s = last(L->cost, x);
        const int each = tile_steps(L->range[s].y, step) + tile_cost;
        t = L->items[s] + (x - L->cost[s] + each - 1) / each;
      }
      t = t < tot.x ? t : tot.x;
      L->tm[rho] = t > P ? t : P;
    }
    if (b == 0) L->tm[P] = tot.x;
  }
  __syncthreads();
  d.L = L;
  d.P = P;
  d.w = static_cast<int>(blockIdx.x >> 3);
  d.xcd = xcd;
  d.tiles = tiles;
  d.total = uniform(tot.x);
  d.s = (tiles + 7) / 8 >= P ? 0 : d.G;  // no whole rounds: straight to the items
  d.k = 0;
  d.m = 0;
  d.t = 0;
  d.at = 0;
}

// Its first item among those that m workgroups take in turn.  The turn goes by the
// item's number and not by its place among these: they may be one or two only,
// and would always fall to the same workgroup.
__device__ __forceinline__ int first_of(const Dealer& d, int rho) {
  const int from = uniform(lds_int(&d.L->tm[d.m - 1]));
  const int ahead = rho - (from - d.P) % d.m;
  return from + (ahead < 0 ? ahead + d.m : ahead);
}

// The workgroup's next tile: expert s and tile i of it; false: none left.
__device__ __forceinline__ bool next(Dealer& d, int& s, int& i) {
  while (d.s < d.G) {
    const int2 sh = share(d.s, d.xcd, d.tiles);
    if ((d.k + 1) * d.P <= sh.y) {
      s = d.s;
      i = sh.x + d.k * d.P + d.w;
      ++d.k;
      return true;
    }
    ++d.s;
    d.k = 0;
  }
  const int rho = d.P - 1 - d.w;
  int t;
  if (d.m == 0) {
    d.m = rho + 1;
    d.t = first_of(d, rho);
    t = d.w;
    if (t >= d.total) return false;  // fewer items than workgroups
  } else {
    for (;; ) {
      if (d.m > d.P) return false;
      if (d.t < uniform(lds_int(&d.L->tm[d.m]))) break;
      if (++d.m > d.P) return false;
      d.t = first_of(d, rho);
    }
    t = d.t;
    d.t += d.m;
  }
  // its expert: the last one with no more than t items before it, 64 at a time
  const int lane = threadIdx.x & 63;
  for (;;) {
    const int n = __popcll(__ballot(d.at + lane < d.G && lds_int(&d.L->items[d.at + lane]) <= t));
    if (n < 64) {
      d.at += n - 1;
      break;
    }
    d.at += 63;
  }
  d.at = uniform(d.at);
  s = d.at;
  const int2 sh = share(s, d.xcd, d.tiles);
  i = sh.x + sh.y / d.P * d.P + t - uniform(lds_int(&d.L->items[s]));
  return true;
}

}  // namespace sched
}  // namespace moe
