// wi_paged_merge.cuh -- partial results of the paged attention's items, added up; and fp32 pairs.
#pragma once
#include <cuda_runtime.h>

#include "wi_common.cuh"
#include "wi_paged.h"
#include "wi_paged_walk.cuh"
#include "wi_pipe.cuh"
#include "wi_tc.cuh"

namespace {

constexpr float kLn2 = 0.6931471805599453f;

// A partial result holds two tiles of 128 rows, or, where a call has no more, one of kMergeHere or kFewRows: those of
// all CTAs lie within 5 or 1.3 MB then, which a merge reads with fewer address translations.
constexpr int kFewRows = 8;
constexpr int kMergeHere = 32;  // rows per kv head of a call up to which the attention kernel merges itself
constexpr size_t kPartBytes = 2 * kRows * (2 + WI_D) * 4;
constexpr size_t kSplitBytes = kPagedMaxSms * sizeof(Split);

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Two fp32 values in one 64-bit register pair.
__device__ __forceinline__ uint64_t pair(uint32_t a, uint32_t b) {
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "r"(a), "r"(b));
  return x;
}
__device__ __forceinline__ uint64_t pair(float a, float b) { return pair(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ float lo_of(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float hi_of(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 w = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&w);
}

// ---- merge of an item that was cut between CTAs
//
// out = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c over the CTAs c that worked on it, in their order.
constexpr int kMergeThreads = 512;

// Rows of an item's tile t.
__device__ __forceinline__ int tile_rows(const Params& P, const Split& sp, int t) {
  return min(P.tq, sp.cnt - t * P.tq) * P.G;
}

// The partial result of the i-th CTA that worked on the item that CTA c0 begins.
__device__ __forceinline__ const float* part_of(const Params& P, int c0, int i) {
  return P.parts.slot(2 * (c0 + i) + (i == 0 ? 1 : 0));
}

// (token, query head) of a row of tile t.
__device__ __forceinline__ long long place_of(const Params& P, const Split& sp, int t, int r) {
  const int tok = r / P.G;
  return (long long)(sp.row0 + t * P.tq + tok) * P.Hq + sp.kh * P.G + r - tok * P.G;
}

// Rows of tile t from r0 on by THREADS threads, each two rows of one column (2 * THREADS / 128 rows in all): the parts
// ten at a time, with the running maximum.
template <int THREADS>
__device__ __noinline__ void merge_some(const Params& P, const Split& sp, int c0, int t, int r0) {
  constexpr int kPairs = THREADS / WI_D, kAtOnce = 10;
  const int r = r0 + 2 * (threadIdx.x % kPairs), d = threadIdx.x / kPairs, parts = sp.last - c0 + 1;
  float M[2] = {-INFINITY, -INFINITY}, L[2] = {0.f, 0.f}, acc[2] = {0.f, 0.f};
#pragma unroll 1
  for (int i0 = 0; i0 < parts; i0 += kAtOnce) {
    float2 m[kAtOnce], l[kAtOnce], o[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      m[k] = make_float2(-INFINITY, -INFINITY);
      l[k] = o[k] = make_float2(0.f, 0.f);
      if (i0 + k < parts) {
        const float* p = part_of(P, c0, i0 + k);
        m[k] = __ldcg(reinterpret_cast<const float2*>(p + P.parts.m(t, r)));
        l[k] = __ldcg(reinterpret_cast<const float2*>(p + P.parts.l(t, r)));
        o[k] = __ldcg(reinterpret_cast<const float2*>(p + P.parts.o(t, d, r)));
      }
    }
    float2 top = make_float2(M[0], M[1]);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) top = make_float2(fmaxf(top.x, m[k].x), fmaxf(top.y, m[k].y));
    const float ref0 = top.x == -INFINITY ? 0.f : top.x, ref1 = top.y == -INFINITY ? 0.f : top.y;
    const float f0 = ex2(M[0] - ref0), f1 = ex2(M[1] - ref1);
    M[0] = top.x;
    M[1] = top.y;
    L[0] *= f0;
    L[1] *= f1;
    acc[0] *= f0;
    acc[1] *= f1;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const float g0 = ex2(m[k].x - ref0), g1 = ex2(m[k].y - ref1);
      L[0] += g0 * l[k].x;
      L[1] += g1 * l[k].y;
      acc[0] += g0 * o[k].x;
      acc[1] += g1 * o[k].y;
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (r + k < tile_rows(P, sp, t)) {
      const long long at = place_of(P, sp, t, r + k);
      static_cast<bf16*>(P.a.out)[at * WI_D + d] = __float2bfloat16_rn(L[k] == 0.f ? 0.f : acc[k] / L[k]);
      if (P.a.lse && d == 0) P.a.lse[at] = L[k] == 0.f ? -INFINITY : M[k] * kLn2 + logf(L[k]);
    }
}

// COLS columns from d0 on of row r of tile t, added up: the parts four at a time, every load of them issued before the
// first is used, with the running maximum (ONCE: no more than four).  A lane to a row, as they were written; ROWS,
// TILES: the parts' layout.
constexpr int kWideParts = 4;
template <int COLS>
struct Merged {
  float M, L, acc[COLS];
};
template <int COLS, int ROWS, int TILES, bool ONCE = false>
__device__ __forceinline__ Merged<COLS> merge_wide(const Params& P, const Split& sp, int c0, int t, int r, int d0) {
  constexpr int kAtOnce = kWideParts;
  const int parts = sp.last - c0 + 1;
  Merged<COLS> x = {-INFINITY, 0.f, {}};
#pragma unroll 1
  for (int i0 = 0; i0 < (ONCE ? 1 : parts); i0 += kAtOnce) {
    float m[kAtOnce], l[kAtOnce], o[kAtOnce][COLS];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      m[k] = -INFINITY;
      l[k] = 0.f;
#pragma unroll
      for (int c = 0; c < COLS; ++c) o[k][c] = 0.f;
      if (i0 + k < parts) {
        const float* p = part_of(P, c0, i0 + k) + r;
        m[k] = __ldcg(p + t * ROWS);
        l[k] = __ldcg(p + (TILES + t) * ROWS);
        p += (2 * TILES + t * WI_D + d0) * ROWS;
#pragma unroll
        for (int c = 0; c < COLS; ++c) o[k][c] = __ldcg(p + c * ROWS);
      }
    }
    float top = x.M;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) top = fmaxf(top, m[k]);
    const float ref = top == -INFINITY ? 0.f : top, f = ex2(x.M - ref);
    x.M = top;
    x.L *= f;
#pragma unroll
    for (int c = 0; c < COLS; ++c) x.acc[c] *= f;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const float g = ex2(m[k] - ref);
      x.L += g * l[k];
#pragma unroll
      for (int c = 0; c < COLS; ++c) x.acc[c] += g * o[k][c];
    }
  }
  const float inv = x.L == 0.f ? 0.f : 1.f / x.L;
#pragma unroll
  for (int c = 0; c < COLS; ++c) x.acc[c] *= inv;
  return x;
}

// All rows (32 at most) of an item of one tile by WARPS warps, sixteen columns each of eight.
template <int WARPS>
__device__ __noinline__ void merge_tile(const Params& P, const Split& sp, int c0) {
  constexpr int kCols = WI_D / WARPS;
  const int r = threadIdx.x & 31, d0 = (threadIdx.x >> 5) * kCols;
  if (r >= tile_rows(P, sp, 0)) return;
  const Merged<kCols> x = merge_wide<kCols, kMergeHere, 1>(P, sp, c0, 0, r, d0);
  const long long at = place_of(P, sp, 0, r);
  uint4* out = reinterpret_cast<uint4*>(static_cast<bf16*>(P.a.out) + at * WI_D + d0);
#pragma unroll
  for (int i = 0; i < kCols / 8; ++i) {
    const float* a = x.acc + 8 * i;
    out[i] = make_uint4(pack2(a[0], a[1]), pack2(a[2], a[3]), pack2(a[4], a[5]), pack2(a[6], a[7]));
  }
  if (P.a.lse && d0 == 0) P.a.lse[at] = x.L == 0.f ? -INFINITY : x.M * kLn2 + logf(x.L);
}

// What a CTA's earlier segments of an item left in the scratch, added to a row's O in tensor memory (columns [ca, cb) at
// `to`; with `join`, of both chains, whose factors are f0 and f1).  Returns the row's new maximum and sum.
__device__ __noinline__ float2 add_earlier(const Params& P, const float* src, int t, int row, bool live, float m, float l,
                                           uint32_t to, int ca, int cb, bool join, float f0, float f1) {
  const float pm = live ? __ldcg(src + P.parts.m(t, row)) : -INFINITY, pl = live ? __ldcg(src + P.parts.l(t, row)) : 0.f;
  const float top = fmaxf(m, pm), ref = top == -INFINITY ? 0.f : top, f = ex2(m - ref), g = ex2(pm - ref);
#pragma unroll 1
  for (int c = ca; c < cb; c += 16) {
    uint32_t a[16], b[16];
    __syncwarp();
    tmem_ld16_nowait(to + c, a);
    tmem_ld16_nowait(to + (join ? WI_D : 0) + c, b);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float o = __uint_as_float(a[i]);
      if (join) o = o * f0 + __uint_as_float(b[i]) * f1;
      a[i] = __float_as_uint(live ? o * f + __ldcg(src + P.parts.o(t, c + i, row)) * g : o);
    }
    tmem_st16_nowait(to + c, a);
  }
  tmem_wait_st();
  return make_float2(top, l * f + pl * g);
}

// The merge as a kernel of its own: a block takes 32 rows of one cut item.  What counts is latency.  The rows are turned
// in shared memory for the way out; where there are few, more threads share one.
constexpr int kMergeRows = 32;

// Row base + lane of the tile, eight columns to a warp, to `to` in bf16.
template <bool ONCE>
__device__ __forceinline__ void merge_row(const Params& P, const Split& sp, int c0, int t, int base, bf16* to) {
  const int r = base + (threadIdx.x & 31), warp = threadIdx.x >> 5;
  const Merged<8> y = merge_wide<8, kRows, 2, ONCE>(P, sp, c0, t, r, warp * 8);
  uint4 x;
  x.x = pack2(y.acc[0], y.acc[1]);
  x.y = pack2(y.acc[2], y.acc[3]);
  x.z = pack2(y.acc[4], y.acc[5]);
  x.w = pack2(y.acc[6], y.acc[7]);
  *reinterpret_cast<uint4*>(to) = x;
  if (P.a.lse && warp == 0 && r < tile_rows(P, sp, t))
    P.a.lse[place_of(P, sp, t, r)] = y.L == 0.f ? -INFINITY : y.M * kLn2 + logf(y.L);
}

__device__ __noinline__ void merge_row_of_many(const Params& P, const Split& sp, int c0, int t, int base, bf16* to) {
  merge_row<false>(P, sp, c0, t, base, to);
}

__global__ void __launch_bounds__(kMergeThreads, 2) k_paged_merge(const __grid_constant__ Params P) {
  __shared__ __align__(16) bf16 turn[kMergeRows][WI_D + 8];
  pdl_wait();
  const int c0 = blockIdx.x;
  const Split sp = P.splits[c0];
  if (sp.last < 0) return;
  const int t = blockIdx.y / (kRows / kMergeRows), base = blockIdx.y % (kRows / kMergeRows) * kMergeRows;
  const int rows = tile_rows(P, sp, t);
  if (base >= rows) return;
  bf16* const to = &turn[threadIdx.x & 31][(threadIdx.x >> 5) * 8];  // (rows behind the last are read, and not stored)
  if (sp.last - c0 < kWideParts) {
    merge_row<true>(P, sp, c0, t, base, to);
  } else if (rows - base <= kFewRows) {
    for (int r0 = base; r0 < rows; r0 += 2 * kMergeThreads / WI_D) merge_some<kMergeThreads>(P, sp, c0, t, r0);
    return;
  } else {
    merge_row_of_many(P, sp, c0, t, base, to);
  }
  __syncthreads();
  static_assert(kMergeThreads / 32 * 8 == WI_D && kMergeThreads / 16 == kMergeRows, "thread maps");
  const int q = threadIdx.x >> 4, c = (threadIdx.x & 15) * 8;  // sixteen threads store a row
  if (base + q < rows)
    *reinterpret_cast<uint4*>(static_cast<bf16*>(P.a.out) + place_of(P, sp, t, base + q) * WI_D + c) =
        *reinterpret_cast<const uint4*>(&turn[q][c]);
}

}  // namespace
