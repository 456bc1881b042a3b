// wi_paged8.cu -- the paged cache in 8 bits: writes and gather.
#include <cuda_runtime.h>

#include <type_traits>

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
// of one group, tokens that follow one another in rising slots; two warps take a
// run's rows of one head's keys or values into registers (sixteen lanes hold a row
// of 128 elements, eight each), norm and turn the keys, find their largest value
// (the one exchange between them), and round.  Where the group's scale grows the
// rows in front of the run are rounded again.  A CTA takes the runs that begin in its
// tile of tokens, one after the other, with the rotation's cosines and sines of a
// run's rows in shared memory for its heads of keys; the first head's rows are asked
// for before those are worked out.  Runs of four tokens at most, as decoding gives,
// go sixteen lanes to a run's rows of a head, the tile's at once (1000 single tokens
// 8.2 us, 24.3 one run after the other).
// 8192 tokens of 32 + 8 + 8 heads: 32.1 us, 5.8 TB/s; instruction issue (67% of the
// slots while busy) and the start and end bound it, as the bf16 write.  The queries
// alone take 26.3.  In a launch of their own behind the queries' the keys and values
// made it 75.7 us; in the same one, a warp to a run's rows of a head 50.6, two warps
// and packed arithmetic 40.5, angles a pair to a thread 32.7.
constexpr int kApTile = 16;   // tokens of a tile, at most
constexpr int kApHeads = 2;   // heads that a CTA has at once
constexpr int kShort = 4;     // tokens of a short run, at most

struct Append {
  int tile;          // tokens of a tile
  int ctas;          // CTAs of keys and values
  int parts;         // ... of a tile's keys, and as many of its values
};

// The rotation of a run, or of a tile's short ones: cosine, sine and minus sine of a pair and row.
struct Turns {
  static constexpr int kRows = kApTile + kShort - 1;
  float c[kRows][WI_D / 2], s[kRows][WI_D / 2], n[kRows][WI_D / 2];
};

// Eight elements of a row, as a lane holds them: the first and the second of its pairs (or eight that follow one another).
struct Eight {
  uint64_t a[2], b[2];
  __device__ __forceinline__ void from(const uint2 (&raw)[2]) {
    a[0] = unpack2(raw[0].x), a[1] = unpack2(raw[0].y), b[0] = unpack2(raw[1].x), b[1] = unpack2(raw[1].y);
  }
  __device__ __forceinline__ float squares() const {
    const float2 ss = unpair(fma2(a[0], a[0], fma2(a[1], a[1], fma2(b[0], b[0], mul2(b[1], b[1])))));
    return ss.x + ss.y;
  }
  __device__ __forceinline__ void norm(float inv, const Eight& w) {
    const uint64_t f = pair2(inv, inv);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      a[c] = mul2(mul2(a[c], f), w.a[c]);
      b[c] = mul2(mul2(b[c], f), w.b[c]);
    }
  }
  template <bool INTER>
  __device__ __forceinline__ void turn(const Turns& t, int r, int l) {
    const float4 c4 = *reinterpret_cast<const float4*>(&t.c[r][4 * l]), s4 = *reinterpret_cast<const float4*>(&t.s[r][4 * l]);
    const float4 n4 = *reinterpret_cast<const float4*>(&t.n[r][4 * l]);
    if (INTER) {  // both words hold whole pairs
      a[0] = fma2(a[0], pair2(c4.x, c4.x), mul2(swap2(a[0]), pair2(n4.x, s4.x)));
      a[1] = fma2(a[1], pair2(c4.y, c4.y), mul2(swap2(a[1]), pair2(n4.y, s4.y)));
      b[0] = fma2(b[0], pair2(c4.z, c4.z), mul2(swap2(b[0]), pair2(n4.z, s4.z)));
      b[1] = fma2(b[1], pair2(c4.w, c4.w), mul2(swap2(b[1]), pair2(n4.w, s4.w)));
    } else {
      const uint64_t c2[2] = {pair2(c4.x, c4.y), pair2(c4.z, c4.w)}, s2[2] = {pair2(s4.x, s4.y), pair2(s4.z, s4.w)};
      const uint64_t n2[2] = {pair2(n4.x, n4.y), pair2(n4.z, n4.w)};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint64_t x = a[c];
        a[c] = fma2(x, c2[c], mul2(b[c], n2[c]));
        b[c] = fma2(b[c], c2[c], mul2(x, s2[c]));
      }
    }
  }
  // The bits of the largest absolute value, or of the largest finite one.
  __device__ __forceinline__ uint32_t largest(bool finite) const {
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float2 x = unpair(c < 2 ? a[c & 1] : b[c & 1]);
      const uint32_t u = __float_as_uint(x.x) & 0x7fffffffu, v = __float_as_uint(x.y) & 0x7fffffffu;
      top = max(top, finite && u >= 0x7f800000u ? 0u : u);
      top = max(top, finite && v >= 0x7f800000u ? 0u : v);
    }
    return top;
  }
  // Times f as e4m3, to elements ea and eb of a row.
  template <bool KEY>
  __device__ __forceinline__ void store(unsigned char* row, int ea, int eb, float f) const {
    const uint64_t f2 = pair2(f, f);
    uint32_t y[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint64_t x0 = c ? b[0] : a[0], x1 = c ? b[1] : a[1];
      const float2 y0 = unpair(fma2(x0, 0ull, mul2(x0, f2))), y1 = unpair(fma2(x1, 0ull, mul2(x1, f2)));  // an infinity becomes NaN
      y[c] = e4m3x4_of(y0.x, y0.y, y1.x, y1.y);
    }
    if (KEY) {
      *reinterpret_cast<uint32_t*>(row + ea) = y[0];
      *reinterpret_cast<uint32_t*>(row + eb) = y[1];
    } else {
      *reinterpret_cast<uint2*>(row + ea) = make_uint2(y[0], y[1]);
    }
  }
};

// A lane's eight elements of a row of the input.
template <bool KEY>
__device__ __forceinline__ void load_eight(const bf16* row, int ea, int eb, uint2 (&raw)[2]) {
  if (KEY) {
    raw[0] = ldg_u2(row + ea);
    raw[1] = ldg_u2(row + eb);
  } else {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(row + ea));
    raw[0] = make_uint2(x.x, x.y);
    raw[1] = make_uint2(x.z, x.w);
  }
}

// Eight values in the cache rounded again, to a scale that is 1 / f as large.
__device__ __forceinline__ void round_again(unsigned char* at, float f) {
  uint2* const p = reinterpret_cast<uint2*>(at);
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

template <bool INTER, bool KEY>
__device__ __forceinline__ void append_rows(const WiPagedWrite& A, unsigned char* const scales, const WiRope& R, int Hkv,
                                            int page, int n_slots, float eps, const Append& G, int which, Turns& turns,
                                            uint32_t (*tops)[kWrThreads / 32], int* err) {
  constexpr int kRows = kGroup / 4;  // rows of a lane
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = lane & 15;
  const int row1 = 2 * (warp & 1) + (lane >> 4);  // rows row1, row1 + 4, ..
  const int tile = G.tile;
  // lane i has the slot of token t0 - 1 + i: the tile's, the one before it, and what a run may have behind it
  const long long t0 = (long long)(blockIdx.x / (2 * G.parts)) * tile;
  const long long mine = t0 - 1 + lane;
  int slot = -1;
  if (mine >= 0 && mine < A.n_tokens) {
    const int pos = A.positions[mine];
    slot = A.slots[mine];
    if (pos < 0) slot = -1;
  }
  if (slot >= n_slots) {
    if (KEY && which == 0 && lane > 0 && lane <= tile) atomicOr(err, WI_DEVERR_BAD_PAGE);
    slot = -1;
  }
  const int before = __shfl_up_sync(0xffffffffu, slot, 1);
  const bool begins = slot >= 0 && (slot % kGroup == 0 || before != slot - 1);
  uint32_t starts = __ballot_sync(0xffffffffu, begins && lane > 0 && lane <= tile);
  const uint32_t follow = __ballot_sync(0xffffffffu, slot >= 0 && !begins);
  const int half = R.rotary >> 1;
  const bool turned = KEY && (INTER ? 8 * l < R.rotary : 4 * l < half);
  const int ea = KEY && !INTER && turned ? 4 * l : 8 * l, eb = KEY && !INTER && turned ? 4 * l + half : 8 * l + 4;
  const bf16* const w = KEY ? static_cast<const bf16*>(A.k_weight) : nullptr;
  Eight w8;
  if (KEY && w) {
    const uint2 x[2] = {ldg_u2(w + ea), ldg_u2(w + eb)};
    w8.from(x);
  }
  const long long step = KEY ? A.k_stride : A.v_stride;
  // A thread works out the angles of one pair (the table of them is in constant memory, where 32 addresses take 32 turns: read
  // per angle, it made the keys four fifths of the kernel).
  const int p = tid % (WI_D / 2);
  const unsigned long long one_turn = KEY && p < half ? R.turn[p] : 0;
  const int32_t* const at_axis = A.positions + (KEY && p < half ? (long long)R.axis[p] * A.n_tokens : 0);
  // ... of row r, for token t
  auto angle = [&](int r, long long t) {
    const int pos = at_axis[t];
    // the product's low 64 bits are the fraction of a turn, as in the bf16 write
    const long long a = (long long)(one_turn * (unsigned long long)pos);
    float c, s;
    sincospif((float)(int)(a >> 32) * 4.656612873077393e-10f, &s, &c);
    turns.c[r][p] = c * R.scale;
    turns.s[r][p] = s * R.scale;
    turns.n[r][p] = -s * R.scale;
  };
  // Runs of N tokens at most: sixteen lanes to a run's rows of a head, the tile's runs at once.
  auto short_runs = [&](auto longest) {
    constexpr int N = decltype(longest)::value;
    if (KEY && half) {
      for (int r = tid / (WI_D / 2); p < half && r < tile + N - 1; r += kWrThreads / (WI_D / 2))
        if ((N == 1 ? starts : starts | follow) >> (r + 1) & 1) angle(r, t0 + r);
      __syncthreads();
    }
    // the CTA's heads: kApHeads of every G.parts * kApHeads
    const int sets = (Hkv - which * kApHeads + G.parts * kApHeads - 1) / (G.parts * kApHeads);
    const int runs = __popc(starts), jobs = runs * sets * kApHeads;
    int nth = 0;  // lane i: where run i starts
    uint32_t left = starts;
    for (int i = 0; i < runs; ++i, left &= left - 1)
      if (i == lane) nth = __ffs(left) - 1;
    for (int j0 = 2 * warp; j0 < jobs; j0 += kWrThreads / 16) {
      const int job = j0 + (lane >> 4), hs = job / runs, r = __shfl_sync(0xffffffffu, nth, job - hs * runs) - 1;
      const int h = (hs / kApHeads * G.parts + which) * kApHeads + hs % kApHeads;
      const int at = __shfl_sync(0xffffffffu, slot, r + 1), off = at % kGroup;
      const int len = job < jobs && h < Hkv ? (N == 1 ? 1 : __ffs(~(follow >> (r + 2)))) : 0;
      const int pg = at / page, row = at - pg * page;
      const long long head = (long long)pg * Hkv + h;
      unsigned char* const scale = scales + head * (page / kGroup) + row / kGroup;
      uint2 raw[N][2];
      int held = -128;
      const bf16* const from = static_cast<const bf16*>(KEY ? A.k : A.v) + (t0 + r) * step + h * WI_D;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        raw[k][0] = raw[k][1] = make_uint2(0u, 0u);
        if (k < len) load_eight<KEY>(from + k * step, ea, eb, raw[k]);
      }
      if (len && off > 0) held = scale_exponent(*scale);
      Eight x[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        x[k].from(raw[k]);
        if (KEY && w) {
          float v = x[k].squares();
#pragma unroll
          for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          x[k].norm(rsqrtf(v * (1.f / WI_D) + eps), w8);
        }
        if (turned && k < len) x[k].template turn<INTER>(turns, r + k, l);
      }
      auto largest = [&](bool finite) -> uint32_t {
        uint32_t top = x[0].largest(finite);
#pragma unroll
        for (int k = 1; k < N; ++k) top = max(top, x[k].largest(finite));
#pragma unroll
        for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        return top;
      };
      uint32_t top = largest(false);
      if (__any_sync(0xffffffffu, top >= 0x7f800000u)) top = largest(true);
      __syncwarp();  // all have the old scale
      if (!len) continue;
      const int e = max(scale_needed(top), held);
      unsigned char* const to = static_cast<unsigned char*>(KEY ? A.k_out : A.v_out) + (head * page + row - off) * WI_D;
      if (off > 0 && e > held) {
        const float f = pow2(max(held - e, -30));
        for (int i = 0; i < off; ++i) round_again(to + i * WI_D + 8 * l, f);
      }
      if (l == 0) *scale = (unsigned char)(e + kScaleBias);
      const float f = pow2(-e);
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (k < len) x[k].template store<KEY>(to + (off + k) * WI_D, ea, eb, f);
    }
  };
  const uint32_t longer = starts & follow >> 1 & follow >> 2 & follow >> 3 & follow >> 4;
  static_assert(kShort == 4, "longer: of more tokens than that");
  starts &= ~longer;
  if (starts) {
    if (!(starts & follow >> 1))
      short_runs(std::integral_constant<int, 1>());
    else
      short_runs(std::integral_constant<int, kShort>());
    if (longer) __syncthreads();  // the short runs' cosines and sines are read
  }
  starts = longer;
  int turn = 0;  // of the exchange between two warps
  for (; starts; starts &= starts - 1) {
    const int at = __ffs(starts) - 1;
    const int len = at < 31 ? __ffs(~(follow >> (at + 1))) : 1;  // rows of the run: kGroup at most
    const int first = __shfl_sync(0xffffffffu, slot, at), off = first % kGroup;
    const long long t = t0 - 1 + at;
    const int pg = first / page, row = first - pg * page;
    uint2 raw[kRows][2];
    int was = -128;
    const int h0 = which * kApHeads;
    auto fetch = [&](int h) {
      const bf16* from = static_cast<const bf16*>(KEY ? A.k : A.v) + t * step + h * WI_D;
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        raw[k][0] = raw[k][1] = make_uint2(0u, 0u);
        if (h < Hkv && 4 * k + row1 < len) load_eight<KEY>(from + (4 * k + row1) * step, ea, eb, raw[k]);
      }
      if (off > 0 && h < Hkv) was = scale_exponent(scales[((long long)pg * Hkv + h) * (page / kGroup) + row / kGroup]);
    };
    fetch(h0 + (warp >> 1));
    if (KEY && half) {
      if (turn) __syncthreads();  // the last run's are read
      for (int r = tid / (WI_D / 2); p < half && r < len; r += kWrThreads / (WI_D / 2)) angle(r, t + r);
      __syncthreads();
    }
    for (int hp = h0; hp < Hkv; hp += G.parts * kApHeads, ++turn) {  // (the same turns for all warps)
      const int h = hp + (warp >> 1);
      Eight x[kRows];
#pragma unroll
      for (int k = 0; k < kRows; ++k) x[k].from(raw[k]);
      const int held = was;  // exponent of the scale that the rows in front of the run have
      if (hp + G.parts * kApHeads < Hkv) fetch(h + G.parts * kApHeads);
      if (KEY && w) {
        // the four rows' sums of squares are reduced together, a quarter of the lanes ending with each
        float v[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) v[k] = x[k].squares();
        const bool up8 = l & 8, up4 = l & 4;
        float k0 = up8 ? v[2] : v[0], k1 = up8 ? v[3] : v[1];
        k0 += __shfl_xor_sync(0xffffffffu, up8 ? v[0] : v[2], 8);
        k1 += __shfl_xor_sync(0xffffffffu, up8 ? v[1] : v[3], 8);
        float r = (up4 ? k1 : k0) + __shfl_xor_sync(0xffffffffu, up4 ? k0 : k1, 4);
        r += __shfl_xor_sync(0xffffffffu, r, 2);
        r += __shfl_xor_sync(0xffffffffu, r, 1);
        r = rsqrtf(r * (1.f / WI_D) + eps);
#pragma unroll
        for (int k = 0; k < kRows; ++k) x[k].norm(__shfl_sync(0xffffffffu, r, (lane & 16) + 4 * k), w8);
      }
      if (turned) {
#pragma unroll
        for (int k = 0; k < kRows; ++k)
          if (4 * k + row1 < len) x[k].template turn<INTER>(turns, 4 * k + row1, l);
      }
      auto largest = [&](bool finite) -> uint32_t {
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < kRows; ++k) top = max(top, x[k].largest(finite));
        return __reduce_max_sync(0xffffffffu, top);
      };
      uint32_t top = largest(false);
      if (top >= 0x7f800000u) top = largest(true);  // the largest finite value
      if (lane == 0) tops[turn & 1][warp] = top;
      __syncthreads();  // (the other of the two is free again: what was there was read in front of the barrier before)
      if (h >= Hkv) continue;
      const int e = max(scale_needed(max(tops[turn & 1][warp], tops[turn & 1][warp ^ 1])), held);
      unsigned char* const to =
          static_cast<unsigned char*>(KEY ? A.k_out : A.v_out) + (((long long)pg * Hkv + h) * page + row - off) * WI_D;
      if (off > 0 && e > held) {  // the rows in front are rounded again
        const float f = pow2(max(held - e, -30));  // (2^-30 takes the largest value to nothing)
        for (int r = row1; r < off; r += 4) round_again(to + r * WI_D + 8 * l, f);
      }
      if (lane == 0 && !(warp & 1))
        scales[((long long)pg * Hkv + h) * (page / kGroup) + row / kGroup] = (unsigned char)(e + kScaleBias);
      const float f = pow2(-e);
#pragma unroll
      for (int k = 0; k < kRows; ++k)
        if (4 * k + row1 < len) x[k].template store<KEY>(to + (off + 4 * k + row1) * WI_D, ea, eb, f);
    }
  }
}

// INTER, FULL, AXES: as in the bf16 write.
template <bool INTER, bool FULL, bool AXES>
__global__ void __launch_bounds__(kWrThreads, 6) k_paged_write8(const __grid_constant__ WiPagedWrite A,
                                                               const WiPagedScales S, const __grid_constant__ WiRope R,
                                                               int Hq, int Hkv, int page, int n_slots, float eps, int parts,
                                                               const Append G, int* err) {
  __shared__ __align__(16) unsigned char rows[kWrThreads / 32][kWrStages * kWrBatch];
  __shared__ uint32_t tops[2][kWrThreads / 32];
  static_assert(sizeof(rows) >= sizeof(Turns) && kApTile >= kGroup, "the cosines and sines of a run");
  pdl_trigger();
  pdl_wait();
  if ((int)blockIdx.x < G.ctas) {
    const int which = blockIdx.x % (2 * G.parts);  // a tile's CTAs of keys, then of values
    Turns& turns = *reinterpret_cast<Turns*>(rows);
    if (which < G.parts)
      append_rows<INTER, true>(A, S.k, R, Hkv, page, n_slots, eps, G, which, turns, tops, err);
    else
      append_rows<false, false>(A, S.v, R, Hkv, page, n_slots, eps, G, which - G.parts, turns, tops, err);
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
// Sixteen lanes move one row, eight values each, so that what they store is whole sectors in a row (137 us with eight lanes
// of sixteen values).
constexpr int kGaThreads = 128;
// Rows of a thread, where there are many (a 131K prompt of 8 kv heads 126.2 us with four, 127.8, 129.7 and 130.2 with five, six
// and eight); one where the machine holds them all at once (sixteen requests' rows 2.6 us, 4.4 with four).
constexpr int kGaMany = 4;
constexpr int kGaLanes = 16;
constexpr int kGaStep = kGaThreads / kGaLanes;
static_assert(kGaStep <= kGroup, "a step is less than a page");

__device__ __forceinline__ long long quot(long long a, int b) {
  return (a >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Four values times their scale, as bf16.
__device__ __forceinline__ uint2 widen(uint32_t w, float f) {
  const float2 a = e4m3x2_to_f32x2(w & 0xffffu), b = e4m3x2_to_f32x2(w >> 16);
  const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x * f, a.y * f), hi = __floats2bfloat162_rn(b.x * f, b.y * f);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

template <int kGaRows>
__global__ void __launch_bounds__(kGaThreads) k_paged_gather8(WiPagedGather A, WiPagedScales S, long long rows, int Hkv,
                                                             int page, int n_pages, int max_pages, int* err) {
  pdl_trigger();
  pdl_wait();
  const int l = threadIdx.x % kGaLanes, most = max_pages * page, n = (int)A.n;
  const long long r0 = (long long)blockIdx.x * (kGaStep * kGaRows);
  const long long u0 = quot(r0, n);
  const unsigned i0 = (unsigned)(r0 - u0 * n) + (threadIdx.x / kGaLanes);
  long long cur = -1, pool = 0;  // the unit of the last row, and the pages in front of its layer's pool
  int b = 0, h = 0, len = 0, flags = 0, j = 0, off = 0;
  unsigned i = i0;
  long long u = u0;
  uint2 kr[kGaRows], vr[kGaRows];
  unsigned char ks[kGaRows], vs[kGaRows];
#pragma unroll
  for (int k = 0; k < kGaRows; ++k, i += kGaStep, off += kGaStep) {
    const long long r = r0 + (threadIdx.x / kGaLanes) + k * kGaStep;
    kr[k] = vr[k] = make_uint2(0u, 0u);
    ks[k] = vs[k] = kScaleBias;
    if (r >= rows) continue;
    if (i >= (unsigned)n) {
      u += i / (unsigned)n;
      i %= (unsigned)n;
    }
    const int p = (int)A.pos0 + (int)i;
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
      j = p / page;
      off = p - j * page;
    } else if (off >= page) {  // a step is less than a page
      ++j;
      off -= page;
    }
    const int pg = A.block_table[(long long)b * max_pages + j];  // on its way beside the length: j < max_pages always
    if (p < len) {
      if (pg < 0 || pg >= n_pages) {
        flags |= WI_DEVERR_BAD_PAGE;
      } else {
        const long long head = (pool + pg) * Hkv + h;
        const long long row = head * page + off;
        kr[k] = __ldcg(static_cast<const uint2*>(A.k_pages) + row * kGaLanes + l);
        vr[k] = __ldcg(static_cast<const uint2*>(A.v_pages) + row * kGaLanes + l);
        ks[k] = S.k[row / kGroup];  // (a page is whole groups)
        vs[k] = S.v[row / kGroup];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kGaRows; ++k) {
    const long long r = r0 + (threadIdx.x / kGaLanes) + k * kGaStep;
    if (r >= rows) continue;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint2 x = c ? vr[k] : kr[k];
      const float f = pow2(scale_exponent(c ? vs[k] : ks[k]));
      const uint2 y0 = widen(x.x, f), y1 = widen(x.y, f);
      static_cast<uint4*>(c ? A.v_out : A.k_out)[r * kGaLanes + l] = make_uint4(y0.x, y0.y, y1.x, y1.y);
    }
  }
  if (flags && l == 0) atomicOr(err, flags);
}

}  // namespace

cudaError_t wi_launch_paged_write8(const WiPagedGeom& g, const WiPagedWrite& w, const WiPagedScales& s, int sms, int* err,
                                   cudaStream_t st) {
  constexpr int kWarps = kWrThreads / 32;
  Append G;
  // A CTA takes a tile's long runs one after the other and its short ones at once, kApHeads heads after the other.  Small tiles
  // of few heads spread few tokens over the machine; large ones share a run's angles between heads, and what is known of a tile
  // between its runs.  8 kv heads: up to half an SM's tokens, one to a tile (16 single tokens 3.0 us, 3.8 by fours); fours while
  // all CTAs run at once (256 single tokens 4.7, 5.9 by eights; 500 of one request 5.9, 7.2 by more fours); eights up to the
  // tokens that a call may have of single ones (500 requests' four 10.7 us, 13.0 by fours, 12.7 by sixteens; 4000 single ones 23.5
  // and 26.2), with four heads where two would not run at once (600 tokens of 200 requests 7.1 with two, 8.5 with four); sixteens
  // of eight heads for chunks (8192 tokens 32.2 us, 40.8 by fours).
  const int two = (g.Hkv + kApHeads - 1) / kApHeads;
  auto ctas_of = [&](int tile, int parts) { return 2LL * parts * ((w.n_tokens + tile - 1) / tile); };
  const long long at_once = 6LL * sms;
  G.parts = two;
  if (ctas_of(1, two) <= 4LL * sms) {
    G.tile = 1;
  } else if (ctas_of(4, two) <= at_once) {
    G.tile = 4;
  } else if (w.n_tokens <= kPagedMaxBatch) {
    G.tile = 8;
    if (ctas_of(8, two) > at_once) G.parts = (g.Hkv + 3) / 4;
  } else {
    G.tile = kApTile;
    G.parts = (g.Hkv + 7) / 8;
  }
  const long long ctas = ctas_of(G.tile, G.parts);
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

cudaError_t wi_launch_paged_gather8(const WiPagedGeom& g, const WiPagedGather& a, const WiPagedScales& s, int sms, int* err,
                                    cudaStream_t st) {
  const long long rows = (long long)a.batch * a.layers * g.Hkv * a.n;
  // a row to a thread where the machine holds them all at once, else four
  const int each = rows <= 16LL * sms * kGaStep ? 1 : kGaMany, per = kGaStep * each;
  const long long grid = (rows + per - 1) / per;
  if (grid > 2147483647LL) return cudaErrorInvalidConfiguration;
  return wi_launch_chained(each == 1 ? k_paged_gather8<1> : k_paged_gather8<kGaMany>, dim3((unsigned)grid), kGaThreads, 0, st,
                           a, s, rows, g.Hkv, g.page, g.n_pages, g.max_pages, err);
}
