// wi_paged.cu -- the paged cache's tables, writes and gather.
#include <cuda_runtime.h>

#include "wi_common.cuh"
#include "wi_paged.h"
#include "wi_pipe.cuh"

namespace {

// ---------------------------------------------------------------- page tables
//
// Everything follows from two running sums over the requests, of the new
// tokens and of the new pages.  Every CTA computes both sums itself (a few
// thousand integers at most, from L2), so that one launch with no exchange
// between CTAs is all there is, and then fills its share of the tokens and of
// the fresh pages by binary search in the sums.  Latency: 1.8 us in a graph for
// a few requests, 4.1 us for 256 requests and 26K tokens, 5.1 us for 64
// requests and 154K tokens (1.3 MB).
constexpr int kTabThreads = 256;

struct TabReq {
  int q_start;   // first token
  int first;     // fresh pages of the requests before
  int ctx;       // positions before the step
};

__device__ __forceinline__ long long warp_scan64(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

__global__ void __launch_bounds__(kTabThreads) k_paged_tables(WiPagedTables A, int page, int n_pages, int max_pages,
                                                             int* err) {
  extern __shared__ TabReq req[];  // [batch + 1]
  constexpr int kWarps = kTabThreads / 32;
  __shared__ long long sum_t[kWarps], sum_p[kWarps];
  __shared__ int sum_bad[kWarps];
  const int tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  const int per = (A.batch + kTabThreads - 1) / kTabThreads;  // consecutive requests per thread
  const int b0 = min(tid * per, A.batch), b1 = min(b0 + per, A.batch);
  const long long most = (long long)max_pages * page;  // < 2^31
  auto pages_of = [&](long long n) { return (int)(((unsigned)n + (unsigned)page - 1u) / (unsigned)page); };
  const int free_now = *A.n_free;
  long long tokens = 0, pages = 0;
  int bad = 0;
  for (int b = b0; b < b1; ++b) {
    const long long c = A.ctx_len[b], n = A.new_len[b];
    if (c < 0 || n < 0 || c + n > most) {
      bad = 1;
    } else {
      tokens += n;
      pages += pages_of(c + n) - pages_of(c);
    }
  }
  // exclusive sums over the block; 64 bits, since lengths that are in range each may add up to more
  const int lane = tid & 31, warp = tid >> 5;
  const long long it = warp_scan64(tokens), ip = warp_scan64(pages);
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 31) {
    sum_t[warp] = it;
    sum_p[warp] = ip;
    sum_bad[warp] = bad;
  }
  __syncthreads();
  long long at = it - tokens, first = ip - pages, all_tokens = 0, all_pages = 0;
  bad = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) {
      at += all_tokens;
      first += all_pages;
    }
    all_tokens += sum_t[w];
    all_pages += sum_p[w];
    bad |= sum_bad[w];
  }
  int wrong = bad || all_tokens > A.n_tokens || free_now < 0 || free_now > A.free_cap
                  ? WI_DEVERR_BAD_LENGTH
                  : 0;
  if (all_pages > free_now) wrong |= WI_DEVERR_NO_PAGES;
  if (wrong) all_tokens = all_pages = 0;  // the step is refused as a whole: no token, no page
  const bool lead = blockIdx.x == 0;
  for (int b = b0; b < b1; ++b) {
    const long long c = A.ctx_len[b], n = wrong ? 0 : A.new_len[b];
    const int ctx = c < 0 || c > most ? 0 : (int)c;
    req[b] = {wrong ? 0 : (int)at, wrong ? 0 : (int)first, ctx};
    if (lead) {
      A.kv_len[b] = (int)(ctx + n);
      A.q_start[b] = wrong ? 0 : (int)at;
    }
    at += n;
    first += pages_of(ctx + n) - pages_of(ctx);
  }
  if (tid == 0) {
    req[A.batch] = {(int)all_tokens, (int)all_pages, 0};
    if (lead) {
      A.q_start[A.batch] = (int)all_tokens;
      *A.n_free_out = (int)(free_now - all_pages);
      if (wrong) atomicOr(err, wrong);
    }
  }
  __syncthreads();
  const int step = gridDim.x * kTabThreads, me = blockIdx.x * kTabThreads + tid;
  int flags = 0;
  for (int t = me; t < A.n_tokens; t += step) {
    int slot = -1, pos = -1;
    if (t < all_tokens) {
      int lo = 0, hi = A.batch - 1;  // the last request that starts at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (req[mid].q_start <= t) lo = mid; else hi = mid - 1;
      }
      pos = req[lo].ctx + (t - req[lo].q_start);
      const int held = pages_of(req[lo].ctx), j = pos / page;
      const int pg = j < held ? A.block_table[(long long)lo * max_pages + j]
                              : A.free_pages[free_now - 1 - (req[lo].first + j - held)];
      if (pg < 0 || pg >= n_pages) flags |= WI_DEVERR_BAD_PAGE;
      else slot = pg * page + (pos - j * page);
    }
    A.slots[t] = slot;
    A.positions[t] = pos;
  }
  for (int k = me; k < all_pages; k += step) {
    int lo = 0, hi = A.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (req[mid].first <= k) lo = mid; else hi = mid - 1;
    }
    const int j = pages_of(req[lo].ctx) + (k - req[lo].first);
    const int pg = A.free_pages[free_now - 1 - k];
    if (pg < 0 || pg >= n_pages) flags |= WI_DEVERR_BAD_PAGE;
    A.block_table[(long long)lo * max_pages + j] = pg;
  }
  if (flags) atomicOr(err, flags);
}

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

// INTER: pairs (2i, 2i + 1).  FULL: the whole head is rotated (no lane holds elements that are only scaled).
template <bool INTER, bool FULL>
__global__ void __launch_bounds__(kWrThreads, 6) k_paged_write(const __grid_constant__ WiPagedWrite A,
                                                              const __grid_constant__ WiRope R, int Hq, int Hkv, int page,
                                                              int n_slots, float eps, int parts, int* err) {
  const int lane = threadIdx.x & 31, l = lane & 15, row1 = lane >> 4;
  pdl_trigger();
  pdl_wait();
  const long long unit = (long long)blockIdx.x * (kWrThreads / 32) + (threadIdx.x >> 5);
  const long long tl = unit / parts;
  if (tl >= A.n_tokens) return;  // the whole warp
  const int t = (int)tl, part = (int)(unit - tl * parts);
  const int half = R.rotary >> 1, bq = (Hq + 7) >> 3, bk = (Hkv + 7) >> 3, batches = bq + 2 * bk;
  const bool turned = FULL || (INTER ? 8 * l < R.rotary : 4 * l < half);
  const int o0 = !INTER && turned ? 4 * l : 8 * l, o1 = !INTER && turned ? 4 * l + half : 8 * l + 4;
  // kWrStages batches of this warp are on their way or worked on; a row that does not exist is left as it is and
  // touches no other
  __shared__ __align__(16) unsigned char rows[kWrThreads / 32][kWrStages][kWrBatch];
  unsigned char* const mine = rows[threadIdx.x >> 5][0];
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
        const long long a = (long long)(R.turn[4 * l + 2 * row1 + i] * (unsigned long long)pos);
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

// ---------------------------------------------------------------- gather
//
// A copy: sixteen lanes move one 256-byte row with 16-byte loads, and each
// takes kGaRows rows of K and of V at once.  Rows are numbered through over
// all (request, layer, kv head) units, so that one row per unit fills the
// CTAs as well as long units do.  A 131K prompt of 8 kv heads in 163 us: 6.6
// TB/s, 0.97 of the measured copy rate.
constexpr int kGaThreads = 256;
constexpr int kGaRows = 4;

// a / b for a >= 0, b > 0; 64-bit division only where 32 bits do not do.
__device__ __forceinline__ long long quot(long long a, int b) {
  return (a >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

__global__ void __launch_bounds__(kGaThreads) k_paged_gather(WiPagedGather A, long long rows, int Hkv, int page,
                                                            int n_pages, int max_pages, int* err) {
  constexpr int kStep = kGaThreads / 16;
  pdl_trigger();
  pdl_wait();
  const int l = threadIdx.x & 15;
  const int most = max_pages * page, n = (int)A.n;
  const long long r0 = (long long)blockIdx.x * (kStep * kGaRows);
  const long long u0 = quot(r0, n);
  const unsigned i0 = (unsigned)(r0 - u0 * n) + (threadIdx.x >> 4);
  long long cur = -1, pool = 0;  // the unit of the last row, and where its layer's pool starts
  int b = 0, h = 0, len = 0, flags = 0;
  uint4 kr[kGaRows], vr[kGaRows];
#pragma unroll
  for (int k = 0; k < kGaRows; ++k) {
    const long long r = r0 + (threadIdx.x >> 4) + k * kStep;
    kr[k] = vr[k] = make_uint4(0u, 0u, 0u, 0u);
    if (r >= rows) continue;
    unsigned i = i0 + k * kStep;
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
      pool = (bl - (long long)b * A.layers) * n_pages * (long long)Hkv * page;
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
        const long long src = (pool + ((long long)pg * Hkv + h) * page + (p - j * page)) * 16 + l;
        kr[k] = __ldcg(static_cast<const uint4*>(A.k_pages) + src);
        vr[k] = __ldcg(static_cast<const uint4*>(A.v_pages) + src);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kGaRows; ++k) {
    const long long r = r0 + (threadIdx.x >> 4) + k * kStep;
    if (r < rows) {
      static_cast<uint4*>(A.k_out)[r * 16 + l] = kr[k];
      static_cast<uint4*>(A.v_out)[r * 16 + l] = vr[k];
    }
  }
  if (flags && l == 0) atomicOr(err, flags);
}

}  // namespace

cudaError_t wi_launch_paged_tables(const WiPagedGeom& g, const WiPagedTables& a, int sms, int* err, cudaStream_t st) {
  const size_t smem = (size_t)(a.batch + 1) * sizeof(TabReq);
  static int smem_set[kWiSmemDevices] = {};
  if (smem > 40 * 1024) {
    const cudaError_t e = wi_ensure_smem(k_paged_tables, smem, smem_set);
    if (e != cudaSuccess) return e;
  }
  const long long want = ((long long)a.n_tokens + kTabThreads - 1) / kTabThreads;
  const int grid = want < 1 ? 1 : want > sms ? sms : (int)want;
  return wi_launch_chained(k_paged_tables, dim3((unsigned)grid), kTabThreads, smem, st, a, g.page, g.n_pages,
                           g.max_pages, err);
}

cudaError_t wi_launch_paged_write(const WiPagedGeom& g, const WiPagedWrite& a, int sms, int* err, cudaStream_t st) {
  // warps that share a token's batches: enough to fill the machine, no more than there are batches (each computes
  // the token's angles again)
  const int batches = (g.Hq + 7) / 8 + 2 * ((g.Hkv + 7) / 8);
  long long parts = ((long long)kWrPerSm * sms + a.n_tokens - 1) / a.n_tokens;
  if (parts > batches) parts = batches;
  const long long grid = (parts * a.n_tokens + kWrThreads / 32 - 1) / (kWrThreads / 32);
  const bool full = g.rope.rotary == WI_D;
  auto* kernel = g.rope.interleaved ? (full ? k_paged_write<true, true> : k_paged_write<true, false>)
                                    : (full ? k_paged_write<false, true> : k_paged_write<false, false>);
  return wi_launch_chained(kernel, dim3((unsigned)grid), kWrThreads, 0, st, a, g.rope, g.Hq, g.Hkv, g.page,
                           g.n_pages * g.page, g.eps, (int)parts, err);
}

cudaError_t wi_launch_paged_gather(const WiPagedGeom& g, const WiPagedGather& a, int* err, cudaStream_t st) {
  const int per = kGaThreads / 16 * kGaRows;
  const long long rows = (long long)a.batch * a.layers * g.Hkv * a.n, grid = (rows + per - 1) / per;
  if (grid > 2147483647LL) return cudaErrorInvalidConfiguration;
  return wi_launch_chained(k_paged_gather, dim3((unsigned)grid), kGaThreads, 0, st, a, rows, g.Hkv, g.page, g.n_pages,
                           g.max_pages, err);
}
