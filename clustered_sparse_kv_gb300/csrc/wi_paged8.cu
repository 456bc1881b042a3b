// wi_paged8.cu -- the paged cache in 8 bits: writes and gather.
#include <cuda_runtime.h>

#include "wi_common.cuh"
#include "wi_e4m3.cuh"
#include "wi_paged.h"
#include "wi_paged_write.cuh"
#include "wi_pipe.cuh"

namespace {

// -------------------------------------------------------------------- write
//
// One launch, two kinds of CTAs.  The queries go as in the bf16 write, a warp to
// heads of one token.  Keys and values: a group of sixteen positions of a head has
// one scale, so its new rows are looked at together.  A run is what a call writes
// of one group, tokens that follow one another in rising slots; a warp takes a
// run's rows of one head's keys or values into registers (sixteen lanes hold a row
// of 128 elements, eight each), norms and turns the keys, reduces their largest
// value, and rounds.  Where the group's scale grows the rows in front of the run are
// rounded again.  A CTA takes the runs that begin in its tile of tokens, one after
// the other, with the rotation's cosines and sines of a run's rows in shared memory
// for all heads of keys.
constexpr int kApTile = 16;  // tokens of a tile, where there are many

struct Append {
  int tile;          // tokens of a tile
  int ctas;          // CTAs of keys and values
  int parts;         // ... of a tile's keys, and as many of its values
};

template <bool INTER>
__device__ __forceinline__ void append_rows(const WiPagedWrite& A, const WiPagedScales& S, const WiRope& R, int Hkv, int page,
                                            int n_slots, float eps, const Append& G, float2 (*turns)[WI_D / 2], int* err) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = lane & 15, row1 = lane >> 4;
  const int tile = G.tile, which = blockIdx.x % (2 * G.parts);  // keys' CTAs of the tile, then values'
  const bool is_key = which < G.parts;
  // lane i has the slot of token t0 - 1 + i: the tile's, the one before it, and what a run may have behind it
  const long long t0 = (long long)(blockIdx.x / (2 * G.parts)) * tile;
  const long long mine = t0 - 1 + lane;
  int slot = -1;
  if (mine >= 0 && mine < A.n_tokens && A.positions[mine] >= 0) slot = A.slots[mine];
  if (slot >= n_slots) {
    if (lane > 0 && lane <= tile && which == 0) atomicOr(err, WI_DEVERR_BAD_PAGE);
    slot = -1;
  }
  const int before = __shfl_up_sync(0xffffffffu, slot, 1);
  const bool begins = slot >= 0 && (slot % kGroup == 0 || before != slot - 1);
  uint32_t starts = __ballot_sync(0xffffffffu, begins && lane > 0 && lane <= tile);
  const uint32_t follow = __ballot_sync(0xffffffffu, slot >= 0 && !begins);
  const int half = R.rotary >> 1;
  const bool turned = INTER ? 8 * l < R.rotary : 4 * l < half;
  const int o0 = !INTER && turned ? 4 * l : 8 * l, o1 = !INTER && turned ? 4 * l + half : 8 * l + 4;
  for (; starts; starts &= starts - 1) {
    const int at = __ffs(starts) - 1;
    const int len = at < 31 ? __ffs(~(follow >> (at + 1))) : 1;  // rows of the run: kGroup at most
    const int first = __shfl_sync(0xffffffffu, slot, at), off = first % kGroup;
    const long long t = t0 - 1 + at;
    if (is_key && half) {
      __syncthreads();  // the last run's are read
      for (int i = tid; i < len * half; i += kWrThreads) {
        const int r = i / half, p = i - r * half;
        const int pos = A.positions[(long long)R.axis[p] * A.n_tokens + t + r];
        // the product's low 64 bits are the fraction of a turn, as in the bf16 write
        const long long a = (long long)(R.turn[p] * (unsigned long long)pos);
        float c, s;
        sincospif((float)(int)(a >> 32) * 4.656612873077393e-10f, &s, &c);
        turns[r][p] = make_float2(c * R.scale, s * R.scale);
      }
      __syncthreads();
    }
    const int pg = first / page, row = first - pg * page;
    for (int h = (is_key ? which : which - G.parts) * (kWrThreads / 32) + warp; h < Hkv; h += G.parts * (kWrThreads / 32)) {
      const int ea = is_key ? o0 : 8 * l, eb = is_key ? o1 : 8 * l + 4;  // this lane's elements of a row
      const bf16* from = (is_key ? static_cast<const bf16*>(A.k) + t * A.k_stride : static_cast<const bf16*>(A.v) + t * A.v_stride) +
                         h * WI_D;
      const long long step = is_key ? A.k_stride : A.v_stride;
      unsigned char* const to =
          static_cast<unsigned char*>(is_key ? A.k_out : A.v_out) + (((long long)pg * Hkv + h) * page + row - off) * WI_D;
      unsigned char* const scale =
          (is_key ? S.k : S.v) + ((long long)pg * Hkv + h) * (page / kGroup) + row / kGroup;
      float x[kGroup / 2][8];
      uint2 raw[kGroup / 2][2];
#pragma unroll
      for (int k = 0; k < kGroup / 2; ++k) {
        raw[k][0] = raw[k][1] = make_uint2(0u, 0u);
        if (2 * k + row1 < len) {
          raw[k][0] = ldg_u2(from + (2 * k + row1) * step + ea);
          raw[k][1] = ldg_u2(from + (2 * k + row1) * step + eb);
        }
      }
      const int was = off > 0 ? scale_exponent(*scale) : -128;
      float wa[4] = {1.f, 1.f, 1.f, 1.f}, wb[4] = {1.f, 1.f, 1.f, 1.f};
      const bf16* w = static_cast<const bf16*>(A.k_weight);
      if (is_key && w) {
        load_bf16x4(w + ea, wa);
        load_bf16x4(w + eb, wb);
      }
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < kGroup / 2; ++k) {
        float a[4], b[4];
        unpack_bf16x4(raw[k][0], a);
        unpack_bf16x4(raw[k][1], b);
        if (is_key) {
          if (w) {
            float ss = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) ss += a[c] * a[c] + b[c] * b[c];
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float inv = rsqrtf(ss * (1.f / WI_D) + eps);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              a[c] *= inv * wa[c];
              b[c] *= inv * wb[c];
            }
          }
          if (turned && 2 * k + row1 < len) {
            const float2* f = turns[2 * k + row1] + 4 * l;
            if (INTER) {
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const float a0 = a[2 * c], b0 = b[2 * c];
                a[2 * c] = a0 * f[c].x - a[2 * c + 1] * f[c].y;
                a[2 * c + 1] = a[2 * c + 1] * f[c].x + a0 * f[c].y;
                b[2 * c] = b0 * f[2 + c].x - b[2 * c + 1] * f[2 + c].y;
                b[2 * c + 1] = b[2 * c + 1] * f[2 + c].x + b0 * f[2 + c].y;
              }
            } else {
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const float a0 = a[c];
                a[c] = a0 * f[c].x - b[c] * f[c].y;
                b[c] = b[c] * f[c].x + a0 * f[c].y;
              }
            }
          }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          x[k][c] = a[c];
          x[k][4 + c] = b[c];
          top = max(top, max(__float_as_uint(a[c]) & 0x7fffffffu, __float_as_uint(b[c]) & 0x7fffffffu));
        }
      }
      top = __reduce_max_sync(0xffffffffu, top);
      if (top >= 0x7f800000u) {  // the largest finite value
        top = 0;
#pragma unroll
        for (int k = 0; k < kGroup / 2; ++k)
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint32_t v = __float_as_uint(x[k][c]) & 0x7fffffffu;
            top = max(top, v >= 0x7f800000u ? 0u : v);
          }
        top = __reduce_max_sync(0xffffffffu, top);
      }
      const int e = max(scale_needed(top), was);
      if (off > 0 && e > was) {  // the rows in front are rounded again
        const float f = pow2(max(was - e, -30));  // (2^-30 takes the largest value to nothing)
        for (int r = row1; r < off; r += 2) {
          uint2* p = reinterpret_cast<uint2*>(to + r * WI_D + 8 * l);
          const uint2 v = *p;
          uint32_t n[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t y = c ? v.y : v.x;
            const float2 p0 = e4m3x2_to_f32x2(y & 0xffffu), p1 = e4m3x2_to_f32x2(y >> 16);
            n[c] = e4m3x4_of(p0.x * f, p0.y * f, p1.x * f, p1.y * f);
          }
          *p = make_uint2(n[0], n[1]);
        }
      }
      if (lane == 0) *scale = (unsigned char)(e + kScaleBias);
      const float f = pow2(-e);
#pragma unroll
      for (int k = 0; k < kGroup / 2; ++k) {
        if (2 * k + row1 >= len) continue;
        float y[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) y[c] = fmaf(x[k][c], 0.f, x[k][c] * f);  // an infinity becomes NaN
        unsigned char* const d = to + (off + 2 * k + row1) * WI_D;
        *reinterpret_cast<uint32_t*>(d + ea) = e4m3x4_of(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<uint32_t*>(d + eb) = e4m3x4_of(y[4], y[5], y[6], y[7]);
      }
    }
  }
}

// INTER, FULL, AXES: as in the bf16 write.
template <bool INTER, bool FULL, bool AXES>
__global__ void __launch_bounds__(kWrThreads, 4) k_paged_write8(const __grid_constant__ WiPagedWrite A,
                                                               const WiPagedScales S, const __grid_constant__ WiRope R,
                                                               int Hq, int Hkv, int page, int n_slots, float eps, int parts,
                                                               const Append G, int* err) {
  __shared__ __align__(16) unsigned char rows[kWrThreads / 32][kWrStages * kWrBatch];
  static_assert(sizeof(rows) >= kGroup * (WI_D / 2) * sizeof(float2), "the cosines and sines of a run");
  pdl_trigger();
  pdl_wait();
  if ((int)blockIdx.x < G.ctas) {
    append_rows<INTER>(A, S, R, Hkv, page, n_slots, eps, G, reinterpret_cast<float2(*)[WI_D / 2]>(rows), err);
  } else {
    WiPagedWrite Q = A;  // no keys and values, so no slots either
    Q.slots = nullptr;
    write_rows<INTER, FULL, AXES>(Q, R, Hq, 0, page, n_slots, eps, parts,
                                  (long long)(blockIdx.x - G.ctas) * (kWrThreads / 32) + (threadIdx.x >> 5),
                                  rows[threadIdx.x >> 5], err);
  }
}

// ------------------------------------------------------------------- gather
//
// Eight lanes move one row: sixteen values each, to thirty-two bytes of bf16.
constexpr int kGaThreads = 256;
constexpr int kGaRows = 4;
constexpr int kGaStep = kGaThreads / 8;

__device__ __forceinline__ long long quot(long long a, int b) {
  return (a >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Four values times their scale, as bf16.
__device__ __forceinline__ uint2 widen(uint32_t w, float f) {
  const float2 a = e4m3x2_to_f32x2(w & 0xffffu), b = e4m3x2_to_f32x2(w >> 16);
  const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x * f, a.y * f), hi = __floats2bfloat162_rn(b.x * f, b.y * f);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

__global__ void __launch_bounds__(kGaThreads) k_paged_gather8(WiPagedGather A, WiPagedScales S, long long rows, int Hkv,
                                                             int page, int n_pages, int max_pages, int* err) {
  pdl_trigger();
  pdl_wait();
  const int l = threadIdx.x & 7, most = max_pages * page, n = (int)A.n;
  const long long r0 = (long long)blockIdx.x * (kGaStep * kGaRows);
  const long long u0 = quot(r0, n);
  const unsigned i0 = (unsigned)(r0 - u0 * n) + (threadIdx.x >> 3);
  long long cur = -1, pool = 0;  // the unit of the last row, and the pages in front of its layer's pool
  int b = 0, h = 0, len = 0, flags = 0;
  uint4 kr[kGaRows], vr[kGaRows];
  unsigned char ks[kGaRows], vs[kGaRows];
#pragma unroll
  for (int k = 0; k < kGaRows; ++k) {
    const long long r = r0 + (threadIdx.x >> 3) + k * kGaStep;
    kr[k] = vr[k] = make_uint4(0u, 0u, 0u, 0u);
    ks[k] = vs[k] = kScaleBias;
    if (r >= rows) continue;
    unsigned i = i0 + k * kGaStep;
    long long u = u0;
    if (i >= (unsigned)n) {
      u += i / (unsigned)n;
      i %= (unsigned)n;
    }
    if (u != cur) {
      cur = u;
      const long long bl = quot(u, Hkv);
      h = (int)(u - bl * Hkv);
      b = (int)quot(bl, A.layers);
      pool = (bl - (long long)b * A.layers) * n_pages;
      len = A.kv_len[b];
      if (len < 0 || len > most) {
        flags |= WI_DEVERR_BAD_LENGTH;
        len = 0;
      }
    }
    const int p = (int)A.pos0 + (int)i, j = p / page;
    const int pg = A.block_table[(long long)b * max_pages + j];  // on its way beside the length: j < max_pages always
    if (p < len) {
      if (pg < 0 || pg >= n_pages) {
        flags |= WI_DEVERR_BAD_PAGE;
      } else {
        const long long head = (pool + pg) * Hkv + h;
        const long long src = (head * page + (p - j * page)) * 8 + l;
        kr[k] = __ldcg(static_cast<const uint4*>(A.k_pages) + src);
        vr[k] = __ldcg(static_cast<const uint4*>(A.v_pages) + src);
        const long long group = head * (page / kGroup) + (p - j * page) / kGroup;
        ks[k] = S.k[group];
        vs[k] = S.v[group];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kGaRows; ++k) {
    const long long r = r0 + (threadIdx.x >> 3) + k * kGaStep;
    if (r >= rows) continue;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint4 x = c ? vr[k] : kr[k];
      const float f = pow2(scale_exponent(c ? vs[k] : ks[k]));
      const uint2 y0 = widen(x.x, f), y1 = widen(x.y, f), y2 = widen(x.z, f), y3 = widen(x.w, f);
      uint4* const to = static_cast<uint4*>(c ? A.v_out : A.k_out) + r * 16 + 2 * l;
      to[0] = make_uint4(y0.x, y0.y, y1.x, y1.y);
      to[1] = make_uint4(y2.x, y2.y, y3.x, y3.y);
    }
  }
  if (flags && l == 0) atomicOr(err, flags);
}

}  // namespace

cudaError_t wi_launch_paged_write8(const WiPagedGeom& g, const WiPagedWrite& w, const WiPagedScales& s, int sms, int* err,
                                   cudaStream_t st) {
  constexpr int kWarps = kWrThreads / 32;
  Append G;
  G.parts = (g.Hkv + kWarps - 1) / kWarps;
  // tiles of one token where that gives no more CTAs than the machine holds at once
  G.tile = 2LL * w.n_tokens * G.parts > 4LL * sms ? kApTile : 1;
  const long long ctas = 2LL * G.parts * ((w.n_tokens + G.tile - 1) / G.tile);
  const int batches = (g.Hq + 7) / 8;
  long long parts = ((long long)kWrPerSm * sms + w.n_tokens - 1) / w.n_tokens;  // as in the bf16 write
  if (parts > batches) parts = batches;
  const long long grid = ctas + (parts * w.n_tokens + kWarps - 1) / kWarps;
  if (grid > 2147483647LL) return cudaErrorInvalidConfiguration;
  G.ctas = (int)ctas;
  const bool full = g.rope.rotary == WI_D, axes = g.rope.axes > 1, inter = g.rope.interleaved;
  auto* kernel = axes ? (inter ? (full ? k_paged_write8<true, true, true> : k_paged_write8<true, false, true>)
                               : (full ? k_paged_write8<false, true, true> : k_paged_write8<false, false, true>))
                      : (inter ? (full ? k_paged_write8<true, true, false> : k_paged_write8<true, false, false>)
                               : (full ? k_paged_write8<false, true, false> : k_paged_write8<false, false, false>));
  return wi_launch_chained(kernel, dim3((unsigned)grid), kWrThreads, 0, st, w, s, g.rope, g.Hq, g.Hkv, g.page,
                           g.n_pages * g.page, g.eps, (int)parts, G, err);
}

cudaError_t wi_launch_paged_gather8(const WiPagedGeom& g, const WiPagedGather& a, const WiPagedScales& s, int* err,
                                    cudaStream_t st) {
  const int per = kGaStep * kGaRows;
  const long long rows = (long long)a.batch * a.layers * g.Hkv * a.n, grid = (rows + per - 1) / per;
  if (grid > 2147483647LL) return cudaErrorInvalidConfiguration;
  return wi_launch_chained(k_paged_gather8, dim3((unsigned)grid), kGaThreads, 0, st, a, s, rows, g.Hkv, g.page, g.n_pages,
                           g.max_pages, err);
}
