// wi_paged_write.cuh -- norms, rotation and the write of a token's heads, for the writes into bf16 and into 8-bit pools.
#pragma once
#include <cuda_runtime.h>

#include "wi_common.cuh"
#include "wi_paged.h"
#include "wi_pipe.cuh"

namespace {

// --------------------------------------------------- norms, rotation, cache write
//
// A warp takes heads of one token in batches of eight: sixteen lanes hold one
// head row of 128 elements, eight each, as two groups of four.  Where the
// rotation pairs element i with i + R / 2, a lane's groups are four pairs
// (4l .. 4l+3 and R/2 further), so norm and rotation need no exchange but the
// sum of squares.  With the norm's weight w folded into the angle's cosine and
// sine once per token, a row costs
//   a' = (a / rms) (w_a cos) - (b / rms) (w_b sin), b' likewise,
// in packed fp32; the four sums of squares that a lane group has in flight are
// reduced together (each of sixteen lanes ends with a quarter of them).  The
// rows come through shared memory, kWrStages batches ahead; the first are
// asked for before the token's position and slot are known (the rows of a
// padding token exist too).  8192 tokens of 32 + 8 + 8 heads: 34.1 us (5.9
// TB/s; 35.1 and 34.7 with two and four stages); with the next batch in
// registers, which left no room for more warps, 38.1; with the operations one
// by one, a row to sixteen lanes, instruction issue bounds it (194 instructions
// for two rows, 48 us).
constexpr int kWrThreads = 128;
constexpr int kWrStages = 3;
constexpr int kWrBatch = 8 * WI_D * 2;  // bytes of a batch
constexpr int kWrPerSm = 16;    // warps per SM that a launch aims at (1531 tokens: 12.2, 8.6, 10.0 us at 8, 16, 24)

__device__ __forceinline__ uint64_t pair2(float a, float b) {
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
  return x;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(x));
  return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t unpack2(uint32_t w) { return pair2(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ uint32_t repack2(uint64_t x) {
  const float2 v = unpair(x);
  const __nv_bfloat162 w = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&w);
}
__device__ __forceinline__ uint64_t swap2(uint64_t x) {
  const float2 v = unpair(x);
  return pair2(v.y, v.x);
}

// A launch parameter by its generic address: as constant memory, which the compiler would read it as, it takes a turn for
// each of a warp's 32 addresses.
__device__ __forceinline__ void load_turns(const unsigned long long* p, unsigned long long (&x)[2]) {
  asm("ld.u64 %0, [%1];" : "=l"(x[0]) : "l"(p));
  asm("ld.u64 %0, [%1];" : "=l"(x[1]) : "l"(p + 1));
}
__device__ __forceinline__ unsigned load_axes(const unsigned char* p) {
  unsigned short x;
  asm("ld.u16 %0, [%1];" : "=h"(x) : "l"(p));
  return x;
}

// INTER: pairs (2i, 2i + 1).  FULL: the whole head is rotated (no lane holds elements that are only scaled).  AXES: a
// pair's position is that of its axis; a lane asks for those of its two pairs beside the token's first.
// A warp's unit of work: `parts` units per token, each with every parts-th batch; `mine`: its kWrStages batches of shared
// memory.
template <bool INTER, bool FULL, bool AXES>
__device__ __forceinline__ void write_rows(const WiPagedWrite& A, const WiRope& R, int Hq, int Hkv, int page, int n_slots,
                                           float eps, int parts, long long unit, unsigned char* mine, int* err) {
  const int lane = threadIdx.x & 31, l = lane & 15, row1 = lane >> 4;
  const long long tl = unit / parts;
  if (tl >= A.n_tokens) return;  // the whole warp
  const int t = (int)tl, part = (int)(unit - tl * parts);
  const int half = R.rotary >> 1, bq = (Hq + 7) >> 3, bk = (Hkv + 7) >> 3, batches = bq + 2 * bk;
  const bool turned = FULL || (INTER ? 8 * l < R.rotary : 4 * l < half);
  const int o0 = !INTER && turned ? 4 * l : 8 * l, o1 = !INTER && turned ? 4 * l + half : 8 * l + 4;
  // kWrStages batches of this warp are on their way or worked on; a row that does not exist is left as it is and
  // touches no other
  auto fetch = [&](int i, int stage) {
    if (i < batches) {
      const int kind = i < bq ? 0 : i < bq + bk ? 1 : 2;
      const int h0 = 8 * (kind == 0 ? i : kind == 1 ? i - bq : i - bq - bk) + row1;
      const bf16* from = (kind == 0   ? static_cast<const bf16*>(A.q) + (long long)t * A.q_stride
                          : kind == 1 ? static_cast<const bf16*>(A.k) + (long long)t * A.k_stride
                                      : static_cast<const bf16*>(A.v) + (long long)t * A.v_stride) +
                         h0 * WI_D + 8 * l;
      const int H = kind == 0 ? Hq : Hkv;
      const uint32_t to = smem_addr(mine) + stage * kWrBatch + row1 * (kWrBatch / 8) + 16 * l;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (h0 + 2 * k < H)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + k * (kWrBatch / 4)), "l"(from + 2 * k * WI_D)
                       : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < kWrStages - 1; ++s) fetch(part + s * parts, s);
  const int pos = A.positions[t];
  int at[2] = {0, 0};
  unsigned long long turn[2] = {0ull, 0ull};  // of this lane's two pairs
  if (turned) {
    load_turns(&R.turn[4 * l + 2 * row1], turn);
    if (AXES) {
      const unsigned both = load_axes(&R.axis[4 * l + 2 * row1]);
      at[0] = A.positions[(long long)(both & 0xffu) * A.n_tokens + t];
      at[1] = A.positions[(long long)(both >> 8) * A.n_tokens + t];
    }
  }
  int slot = A.slots ? A.slots[t] : t;
  if (pos < 0) {  // padding
    asm volatile("cp.async.wait_all;" ::: "memory");  // no copy outlives its warp
    return;
  }
  if (A.slots && slot >= n_slots) {
    if (lane == 0) atomicOr(err, WI_DEVERR_BAD_PAGE);
    slot = -1;
  }
  const int end = slot < 0 ? bq : batches;  // without a slot the query alone is wanted
  float cs[4], sn[4];
  {
    // the two lane groups need the same four angles: each computes two of them
    float c[2] = {1.f, 1.f}, s[2] = {0.f, 0.f};
    if (turned) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // the product's low 64 bits are the fraction of a turn; signed, it is the angle in [-1/2, 1/2) turns, rounded to
        // fp32 here (by at most 2^-26 of a turn, next to half turns)
        const long long a = (long long)(turn[i] * (unsigned long long)(AXES ? at[i] : pos));
        sincospif((float)(int)(a >> 32) * 4.656612873077393e-10f, &s[i], &c[i]);  // 2^-31: half turns
        c[i] *= R.scale;
        s[i] *= R.scale;
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float co = __shfl_xor_sync(0xffffffffu, c[i], 16), so = __shfl_xor_sync(0xffffffffu, s[i], 16);
      cs[i] = row1 ? co : c[i];
      sn[i] = row1 ? so : s[i];
      cs[2 + i] = row1 ? c[i] : co;
      sn[2 + i] = row1 ? s[i] : so;
    }
  }
  // elements between a token's kv heads in k_out / v_out, and its first
  const long long k_step = (A.slots ? page : 1) * (long long)WI_D;
  const long long k_at = (A.slots ? (long long)(slot / page) * Hkv * page + slot % page : (long long)slot * Hkv) * WI_D;
  uint64_t ca[2], cb[2], sa[2], sb[2];  // factors of a in a', of b in b', of a in b', of b in a'
  int have = -1;
  int stage = 0;
  for (int i = part; i < end; i += parts) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kWrStages - 2) : "memory");
    __syncwarp();  // the batch has come for every lane, and none reads the one before it any longer
    const int ahead = i + (kWrStages - 1) * parts;
    fetch(ahead < end ? ahead : batches, stage == 0 ? kWrStages - 1 : stage - 1);
    const unsigned char* const here = mine + stage * kWrBatch + row1 * (kWrBatch / 8);
    stage = stage + 1 == kWrStages ? 0 : stage + 1;
    const int kind = i < bq ? 0 : i < bq + bk ? 1 : 2;
    const int h0 = 8 * (kind == 0 ? i : kind == 1 ? i - bq : i - bq - bk) + row1;
    const int H = kind == 0 ? Hq : Hkv;
    bf16* to = kind == 0 ? static_cast<bf16*>(A.q_out) + ((long long)t * Hq + h0) * WI_D
                         : static_cast<bf16*>(kind == 1 ? A.k_out : A.v_out) + k_at + h0 * k_step;
    const long long step = 2 * (kind == 0 ? (long long)WI_D : k_step);
    const int pairs = (min(8, H - (h0 - row1)) + 1) >> 1;  // rows of the batch, two by two
    if (kind == 2) {  // a copy
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (h0 + 2 * k < H)
          *reinterpret_cast<uint4*>(to + k * step + 8 * l) =
              *reinterpret_cast<const uint4*>(here + k * (kWrBatch / 4) + 16 * l);
      continue;
    }
    uint2 ya[4], yb[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      ya[k] = *reinterpret_cast<const uint2*>(here + k * (kWrBatch / 4) + 2 * o0);
      yb[k] = *reinterpret_cast<const uint2*>(here + k * (kWrBatch / 4) + 2 * o1);
    }
    const bf16* w = static_cast<const bf16*>(kind == 0 ? A.q_weight : A.k_weight);
    if (kind != have) {
      have = kind;
      float wa[4] = {1.f, 1.f, 1.f, 1.f}, wb[4] = {1.f, 1.f, 1.f, 1.f};
      if (w) {
        load_bf16x4(w + o0, wa);
        load_bf16x4(w + o1, wb);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (INTER) {  // a = (x0, x1), (x2, x3): both groups hold whole pairs, turned with their own neighbour
          ca[k] = pair2(wa[2 * k] * cs[k], wa[2 * k + 1] * cs[k]);
          sa[k] = pair2(-wa[2 * k + 1] * sn[k], wa[2 * k] * sn[k]);
          cb[k] = pair2(wb[2 * k] * cs[2 + k], wb[2 * k + 1] * cs[2 + k]);
          sb[k] = pair2(-wb[2 * k + 1] * sn[2 + k], wb[2 * k] * sn[2 + k]);
        } else {
          ca[k] = pair2(wa[2 * k] * cs[2 * k], wa[2 * k + 1] * cs[2 * k + 1]);
          cb[k] = pair2(wb[2 * k] * cs[2 * k], wb[2 * k + 1] * cs[2 * k + 1]);
          sa[k] = pair2(wa[2 * k] * sn[2 * k], wa[2 * k + 1] * sn[2 * k + 1]);
          sb[k] = pair2(-wb[2 * k] * sn[2 * k], -wb[2 * k + 1] * sn[2 * k + 1]);
        }
      }
    }
    float inv[4] = {1.f, 1.f, 1.f, 1.f};
    if (w) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = 0.f;
        if (k >= pairs) continue;
        const uint64_t a0 = unpack2(ya[k].x), a1 = unpack2(ya[k].y), b0 = unpack2(yb[k].x), b1 = unpack2(yb[k].y);
        const float2 ss = unpair(fma2(a0, a0, fma2(a1, a1, fma2(b0, b0, mul2(b1, b1)))));
        v[k] = ss.x + ss.y;
      }
      const bool up8 = l & 8, up4 = l & 4;
      float s0 = up8 ? v[0] : v[2], s1 = up8 ? v[1] : v[3];
      float k0 = up8 ? v[2] : v[0], k1 = up8 ? v[3] : v[1];
      k0 += __shfl_xor_sync(0xffffffffu, s0, 8);
      k1 += __shfl_xor_sync(0xffffffffu, s1, 8);
      float r = (up4 ? k1 : k0) + __shfl_xor_sync(0xffffffffu, up4 ? k0 : k1, 4);
      r += __shfl_xor_sync(0xffffffffu, r, 2);
      r += __shfl_xor_sync(0xffffffffu, r, 1);
      r = rsqrtf(r * (1.f / WI_D) + eps);  // of the row that lanes 4k .. 4k + 3 summed
#pragma unroll
      for (int k = 0; k < 4; ++k) inv[k] = __shfl_sync(0xffffffffu, r, (lane & 16) + 4 * k);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k >= pairs) continue;
      uint64_t a[2] = {unpack2(ya[k].x), unpack2(ya[k].y)}, b[2] = {unpack2(yb[k].x), unpack2(yb[k].y)};
      if (w) {
        const uint64_t f = pair2(inv[k], inv[k]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          a[c] = mul2(a[c], f);
          b[c] = mul2(b[c], f);
        }
      }
      uint32_t ra[2], rb[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint64_t pa = INTER ? swap2(a[c]) : b[c], pb = INTER ? swap2(b[c]) : a[c];
        if (!FULL && !turned) pa = pb = 0;  // nothing of the partner, an infinite one included
        ra[c] = repack2(fma2(a[c], ca[c], mul2(pa, INTER ? sa[c] : sb[c])));
        rb[c] = repack2(fma2(b[c], cb[c], mul2(pb, INTER ? sb[c] : sa[c])));
      }
      ya[k] = make_uint2(ra[0], ra[1]);
      yb[k] = make_uint2(rb[0], rb[1]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (h0 + 2 * k < H) {
        *reinterpret_cast<uint2*>(to + k * step + o0) = ya[k];
        *reinterpret_cast<uint2*>(to + k * step + o1) = yb[k];
      }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace
