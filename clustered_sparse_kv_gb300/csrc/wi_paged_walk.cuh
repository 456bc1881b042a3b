// wi_paged_walk.cuh -- how the attention kernels of the paged cache divide their work.
//
// An item is one (request, kv head, run of TILES tiles of tq tokens); its key blocks of 128 positions run from 0 to the
// last position that a row sees.  A unit is one block of one item, or one of LEAD more for its start and end; all units of
// a call, item after item, are cut into equal runs, one per CTA.  Lengths live on the device: each CTA sums the units of
// all requests itself (closed form per request) and finds its run's start.
#pragma once
#include <cuda_runtime.h>

#include "wi_common.cuh"
#include "wi_paged.h"

namespace {

constexpr int kRows = 128;  // rows of a tile, and positions of a block

// A partial result: m, then l, of every row, then O, column-major (a thread owns a row, so column-major stores of a
// warp are contiguous).
struct Parts {
  float* base;
  int rows, tiles;
  __device__ __forceinline__ float* slot(int i) const {
    return base + (long long)i * (tiles * rows * (2 + WI_D));
  }
  __device__ __forceinline__ int m(int t, int r) const { return t * rows + r; }
  __device__ __forceinline__ int l(int t, int r) const { return (tiles + t) * rows + r; }
  __device__ __forceinline__ int o(int t, int d, int r) const { return (2 * tiles + t * WI_D + d) * rows + r; }
};

// Request b as the kernel reads it; a request with impossible numbers has no tokens (CTA 0 reports it).
struct Req {
  int s0, n, kv, ok;
};

// Where a CTA stands in its run: request, kv head, tile pair, the next unit of that item (its first LEAD units stand
// for no block), and the units of the run still to come.
struct Cursor {
  int b, kh, tile, at, left;
};

// An item that CTA c begins and others go on with: what the merge needs of it.  last < 0: there is none.
struct Split {
  int row0, kh, cnt, last;  // first token (row of q), kv head, tokens, the item's last CTA
};

struct Params {
  WiPagedAttn a;
  int Hq, Hkv, G, tq;       // tq = tokens per tile
  int page, n_pages, max_pages, box;
  Parts parts;
  Split* splits;
  unsigned* tickets;        // of the items, at the CTA that begins each; zero between calls; null: a kernel of its own merges
  int* err;
};

__device__ __forceinline__ Req load_req(const Params& P, int b) {
  Req r;
  r.s0 = P.a.q_start[b];
  const int s1 = P.a.q_start[b + 1];
  r.kv = P.a.kv_len[b];
  r.ok = r.s0 >= 0 && s1 >= r.s0 && s1 <= P.a.n_tokens && r.kv >= 0 && (long long)r.kv <= (long long)P.max_pages * P.page;
  r.n = r.ok ? s1 - r.s0 : 0;
  return r;
}

// Blocks of the tile pair that ends before token `end` of a request whose token 0 sits at p0: at least one,
// so that rows that see nothing are visited too.
__device__ __forceinline__ int blocks_to(long long p0, long long end) {
  const long long e = p0 + end;
  return e <= kRows ? 1 : (int)((e + kRows - 1) / kRows);
}

// Sum over i < n of floor((a i + b) / 128), a, b >= 0, by the steps of Euclid's algorithm on a and the divisor m (the
// known way to a floor sum): whole multiples of m are taken out of a and b, and what is left counts lattice points under
// a line, which is the same problem with a and m exchanged (n <= 2^19, so that after the first step everything but the
// sum fits 32 bits).
__device__ long long floor_sum(int n, int a, long long b) {
  if (n <= 0) return 0;
  long long s = (long long)n * (n - 1) / 2 * (a >> 7) + n * (b >> 7);
  uint32_t k = (uint32_t)n, m = 128, u = (uint32_t)a & 127u, v = (uint32_t)b & 127u;
  for (;;) {
    const uint32_t y = u * k + v;
    if (y < m) return s;
    k = y / m;
    v = y % m;
    const uint32_t t = u;
    u = m;
    m = t;
    s += (long long)k * (k - 1) / 2 * (u / m) + (long long)k * (v / m);
    u %= m;
    v %= m;
  }
}

// Units of the first `m` tile pairs (none of them the last one, which may be shorter).
template <int LEAD>
__device__ long long units_before(long long p0, int tp, int m) {
  long long z = 0;  // pairs that end at or before position 0: one block each
  if (p0 < 0) z = min(-p0 / tp, (long long)m);
  return z + floor_sum((int)(m - z), tp, p0 + (z + 1) * tp + kRows - 1) + (long long)LEAD * m;
}

// a / b; 64-bit division only where 32 bits do not do.
__device__ __forceinline__ long long quot(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// The run, one item's part after the other.  LONGEST: blocks that one segment has at most, 0: as many as there are.
template <int LEAD, int TILES, int LONGEST>
struct WalkOver : Cursor {
  Req r;
  int tp, tiles;
  // the current segment: what the run holds of one item
  int cnt, single, nblk, b0, nb, took;   // tokens, one tile, blocks of the item, first block, blocks, units
  long long p0;           // position of the request's token 0

  __device__ __forceinline__ WalkOver(const Params& P, const Cursor& c, const Req& q) : Cursor(c) {
    tp = TILES * P.tq;
    set(q);
  }
  __device__ __forceinline__ void set(const Req& q) {
    r = q;
    p0 = (long long)r.kv - r.n;
    tiles = (r.n + tp - 1) / tp;
  }
  // The next segment of the run that has blocks; false at the run's end.
  __device__ __forceinline__ bool next(const Params& P) {
    while (left > 0) {
      while (tile >= tiles) {   // past the request's last pair: next kv head, next request with tokens
        tile = 0;
        if (r.n == 0 || ++kh == P.Hkv) {
          kh = 0;
          if (++b >= P.a.batch) return false;
          set(load_req(P, b));
        }
      }
      cnt = min(tp, r.n - tile * tp);
      single = cnt <= P.tq;
      nblk = blocks_to(p0, (long long)tile * tp + cnt);
      took = min(nblk + LEAD - at, left);
      if (LONGEST) took = min(took, LEAD + LONGEST);
      b0 = max(0, at - LEAD);
      nb = max(0, at + took - LEAD) - b0;
      if (nb > 0) return true;
      advance();
    }
    return false;
  }
  __device__ __forceinline__ void advance() {
    left -= took;
    at += took;
    if (at >= nblk + LEAD) {
      at = 0;
      ++tile;
    }
  }
  __device__ __forceinline__ int first_pos() const { return (int)(p0 + (long long)tile * tp); }
  // The item's first block that not all of its rows see whole.
  __device__ __forceinline__ int first_fix() const {
    const int f = first_pos();
    return f < 0 ? 0 : (f + 1) / kRows;
  }
  // The first position whose value row is cleaned: what all rows see stays as it is, in whole groups of eight.
  __device__ __forceinline__ int first_clean() const { return max(0, first_pos() + 1) & ~7; }
};

// The CTA whose run holds unit u of `total`, cut into `ctas` runs.
__device__ __forceinline__ int cta_of(long long u, long long total, int ctas) {
  return (int)quot((u + 1) * ctas - 1, total);
}

// What a place where q_start falls adds to the units: more than any grid takes, and 4096 of them fit 64 bits beside the
// most units that a call can have (2^51).
constexpr long long kFalls = 1LL << 50;

// The requests in front of the first place where q_start falls.  Those behind it may claim rows of the ones in front of
// it: they have no tokens.
__device__ __noinline__ int requests_in_order(const Params& P) {
  int b = 0;
  while (b < P.a.batch && P.a.q_start[b + 1] >= P.a.q_start[b]) ++b;
  return b;
}

// What a CTA knows of its run, in shared memory.
struct Run {
  Cursor start;
  Req req;               // start.b's
  long long end, total;  // the unit behind the run, all units
  int ctas;              // CTAs with units
};

// Units of one kv head of a request.
template <int LEAD>
__device__ __forceinline__ long long units_of(const Req& r, int tp) {
  const long long p0 = (long long)r.kv - r.n;
  return units_before<LEAD>(p0, tp, (r.n + tp - 1) / tp - 1) + LEAD + blocks_to(p0, r.n);
}

// What the threads in front of this one have, and all of them.  With a barrier of all THREADS; scan: a number per warp.
template <int THREADS>
__device__ __forceinline__ void add_up(long long mine, long long* scan, long long& before, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += t;
  }
  if (lane == 31) scan[warp] = before;
  __syncthreads();
  total = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) before += total;
    total += scan[w];
  }
  before -= mine;
}

// The run of units [u0, u1), by the one thread whose requests [rb0, rb1) hold u0; `before` units in front of those.  One
// request: r, of `cost` units per kv head.
template <int LEAD>
__device__ __forceinline__ void begin_run(const Params& P, int tp, int rb0, int rb1, bool one, Req r, long long cost,
                                          long long before, long long u0, long long u1, long long total, int ctas, Run* run) {
  long long rem = u0 - before;
  for (int b = rb0; b < rb1; ++b) {
    if (!one) r = load_req(P, b);
    if (r.n == 0) continue;
    const int tiles = (r.n + tp - 1) / tp;
    const long long p0 = (long long)r.kv - r.n;
    if (!one) cost = units_of<LEAD>(r, tp);
    if (rem >= cost * P.Hkv) {
      rem -= cost * P.Hkv;
      continue;
    }
    const int kh = (int)quot(rem, cost);
    rem -= cost * kh;
    int lo = 0, hi = tiles - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (units_before<LEAD>(p0, tp, mid) <= rem) lo = mid; else hi = mid - 1;
    }
    if (lo > 0) rem -= units_before<LEAD>(p0, tp, lo);
    run->start = {b, kh, lo, (int)rem, (int)(u1 - u0)};
    run->req = r;
    run->end = u1;
    run->total = total;
    run->ctas = ctas;
    break;
  }
}

// The run that is item i of those of requests [b0, b1): all of it.  Called by one thread.
template <int LEAD>
__device__ __noinline__ void own_item(const Params& P, int tp, int b0, int b1, int i, Run* run) {
  for (int b = b0; b < b1; ++b) {
    const Req r = load_req(P, b);
    const int tiles = (r.n + tp - 1) / tp;
    if (i >= tiles * P.Hkv) {
      i -= tiles * P.Hkv;
      continue;
    }
    const int kh = i / tiles, tile = i - kh * tiles;
    const int units = LEAD + blocks_to((long long)r.kv - r.n, min((long long)(tile + 1) * tp, (long long)r.n));
    run->start = {b, kh, tile, 0, units};
    run->req = r;
    run->end = run->total = units;
    run->ctas = 1;
    return;
  }
}

// This CTA's run of the call's units: equal ones, `least` units at least (a run of a few units would spend more on joining
// its part with the others than on the part); where there is one request, whose items are alike, and they have no more than
// `whole` units, each of them is a run.  So it is of several requests with no more items than CTAs, the largest of which has no
// more than `slack` units more than an equal run.  False, for the whole CTA, where it has none.  scan: two numbers per warp.
template <int LEAD, int TILES, int THREADS>
__device__ __forceinline__ bool find_run(const Params& P, int least, int whole, int slack, long long* scan, Run* run) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tp = TILES * P.tq;
  const int per = (P.a.batch + THREADS - 1) / THREADS;
  const int rb0 = min(tid * per, P.a.batch);
  int rb1 = min(rb0 + per, P.a.batch);
  // more than a run can count, through q_start that falls somewhere or pages shared by many requests
  const long long most = (long long)gridDim.x * 0x3fffffff;
  long long mine, before, total, cost = 0;  // cost: of one kv head of the last request looked at
  long long items, largest;  // this thread's; its largest, in units
  Req r = {0, 0, 0, 1};
  for (int again = 0;; ++again) {
    mine = items = largest = 0;
    for (int b = rb0; b < rb1; ++b) {
      r = load_req(P, b);
      if (!r.ok && !again) {
        if (blockIdx.x == 0) atomicOr(P.err, WI_DEVERR_BAD_LENGTH);
        if (P.a.q_start[b + 1] < r.s0) mine += kFalls;
      }
      if (r.n == 0) continue;
      cost = units_of<LEAD>(r, tp);
      mine += P.Hkv * cost;
      items += P.Hkv * ((r.n + tp - 1) / tp);
      largest = max(largest, (long long)LEAD + blocks_to((long long)r.kv - r.n, r.n));
    }
    if (P.a.batch > 1) {
      // of a warp: the largest item, and the items unless they are more than there are CTAs anyway
      const uint32_t units = __reduce_max_sync(0xffffffffu, (uint32_t)largest);
      const uint32_t count = __reduce_add_sync(0xffffffffu, (uint32_t)min(items, 1LL << 16));
      if (lane == 0) reinterpret_cast<uint2*>(scan)[THREADS / 32 + warp] = make_uint2(units, count);
    }
    add_up<THREADS>(mine, scan, before, total);
    if (total <= most) break;
    if (blockIdx.x == 0 && tid == 0) atomicOr(P.err, WI_DEVERR_BAD_LENGTH);
    if (again) {  // too much still: nothing is done
      total = 0;
      break;
    }
    rb1 = min(rb1, requests_in_order(P));
    __syncthreads();  // the sums are read
  }
  int ctas = (int)min((long long)gridDim.x, quot(total + least - 1, least));
  if (P.a.batch == 1 && ctas > P.Hkv && total <= (long long)P.Hkv * whole) ctas = P.Hkv;
  if (P.a.batch > 1) {
    const uint2 x = lane < THREADS / 32 ? reinterpret_cast<const uint2*>(scan)[THREADS / 32 + lane] : make_uint2(0u, 0u);
    const uint32_t most_units = __reduce_max_sync(0xffffffffu, x.x), all = __reduce_add_sync(0xffffffffu, x.y);
    if (all <= gridDim.x && total > 0 && ((long long)most_units - slack) * ctas <= total) {  // item i is CTA i's
      if (blockIdx.x >= all) return false;
      long long first = items;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, first, o);
        if (lane >= o) first += t;
      }
      const int before_warp = (int)__reduce_add_sync(0xffffffffu, lane < warp ? x.y : 0u);
      const int i = (int)(blockIdx.x - before_warp - (first - items));
      if (i >= 0 && i < items) own_item<LEAD>(P, tp, rb0, rb1, i, run);
      __syncthreads();
      return true;
    }
  }
  if ((int)blockIdx.x >= ctas) return false;
  const long long u0 = quot(total * blockIdx.x, ctas), u1 = quot(total * (blockIdx.x + 1), ctas);
  if (u0 >= before && u0 < before + mine)  // (where each thread has one request, that is at hand)
    begin_run<LEAD>(P, tp, rb0, rb1, per == 1, r, cost, before, u0, u1, total, ctas, run);
  __syncthreads();
  return true;
}

}  // namespace
