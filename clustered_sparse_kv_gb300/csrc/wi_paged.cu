// wi_paged.cu -- the paged cache's tables, writes and gather.
#include <cuda_runtime.h>

#include "wi_common.cuh"
#include "wi_paged.h"

namespace {

// ---------------------------------------------------------------- page tables
//
// Everything follows from two running sums over the requests, of the new
// tokens and of the new pages.  Every CTA computes both sums itself (a few
// thousand integers at most, from L2), so that one launch with no exchange
// between CTAs is all there is, and then fills its share of the tokens and of
// the fresh pages by binary search in the sums.
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

// Exclusive sums over the block of two values; 64 bits, since lengths that are in range each may add up to more.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long* tmp, long long* tot_a,
                                            long long* tot_b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int nw = kTabThreads / 32;
  const long long ia = warp_scan64(a), ib = warp_scan64(b);
  __syncthreads();
  if (lane == 31) {
    tmp[warp] = ia;
    tmp[nw + warp] = ib;
  }
  __syncthreads();
  long long ba = 0, bb = 0, ta = 0, tb = 0;
#pragma unroll
  for (int w = 0; w < nw; ++w) {
    if (w == warp) {
      ba = ta;
      bb = tb;
    }
    ta += tmp[w];
    tb += tmp[nw + w];
  }
  a = ba + ia - a;
  b = bb + ib - b;
  *tot_a = ta;
  *tot_b = tb;
}

__global__ void __launch_bounds__(kTabThreads) k_paged_tables(WiPagedTables A, int page, int n_pages, int max_pages,
                                                             int* err) {
  extern __shared__ TabReq req[];  // [batch + 1]
  __shared__ long long tmp[2 * (kTabThreads / 32)];
  const int tid = threadIdx.x;
  const int per = (A.batch + kTabThreads - 1) / kTabThreads;  // consecutive requests per thread
  const int b0 = min(tid * per, A.batch), b1 = min(b0 + per, A.batch);
  const long long most = (long long)max_pages * page;
  long long tokens = 0, pages = 0;
  int bad = 0;
  for (int b = b0; b < b1; ++b) {
    const long long c = A.ctx_len[b], n = A.new_len[b];
    if (c < 0 || n < 0 || c + n > most) {
      bad = 1;
    } else {
      tokens += n;
      pages += (c + n + page - 1) / page - (c + page - 1) / page;
    }
  }
  long long all_tokens, all_pages;
  long long at = tokens, first = pages;
  block_scan2(at, first, tmp, &all_tokens, &all_pages);
  const int free_now = *A.n_free;
  int wrong = __syncthreads_or(bad) || all_tokens > A.n_tokens || free_now < 0 || free_now > A.free_cap
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
    first += (ctx + n + page - 1) / page - (ctx + page - 1) / page;
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
      const int held = (int)(((long long)req[lo].ctx + page - 1) / page), j = pos / page;
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
    const int j = (int)(((long long)req[lo].ctx + page - 1) / page) + (k - req[lo].first);
    const int pg = A.free_pages[free_now - 1 - k];
    if (pg < 0 || pg >= n_pages) flags |= WI_DEVERR_BAD_PAGE;
    A.block_table[(long long)lo * max_pages + j] = pg;
  }
  if (flags) atomicOr(err, flags);
}

// --------------------------------------------------- norms, rotation, cache write
//
// Sixteen lanes hold one head row of 128 elements, eight each, as two groups
// of four: where the rotation pairs element i with i + R / 2, a lane's groups
// are four pairs (4l .. 4l+3 and R/2 further), so that norm and rotation need
// no exchange but the sum of squares.  The lane's four angles are computed
// once for all the rows that it takes from one token.
constexpr int kWrThreads = 256;
constexpr int kWrRows = 4;  // rows in flight per 16 lanes

struct Lane8 {
  uint2 a, b;
};

// Offsets of a lane's two groups inside a head row.
__device__ __forceinline__ void lane_groups(int l, const WiRope& r, int& o0, int& o1) {
  const int half = r.rotary >> 1;
  if (!r.interleaved && 4 * l < half) {
    o0 = 4 * l;
    o1 = 4 * l + half;
  } else {
    o0 = 8 * l;
    o1 = 8 * l + 4;
  }
}

__device__ __forceinline__ uint2 pack4(const float (&x)[4]) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]), hi = __floats2bfloat162_rn(x[2], x[3]);
  uint2 w;
  w.x = *reinterpret_cast<const uint32_t*>(&lo);
  w.y = *reinterpret_cast<const uint32_t*>(&hi);
  return w;
}

__global__ void __launch_bounds__(kWrThreads) k_paged_write(const __grid_constant__ WiPagedWrite A,
                                                           const __grid_constant__ WiRope R, int Hq, int Hkv, int page,
                                                           int n_slots, float eps, int parts, int* err) {
  const int l = threadIdx.x & 15;
  const long long unit = (long long)blockIdx.x * (kWrThreads / 16) + (threadIdx.x >> 4);
  const int t = (int)(unit / parts), part = (int)(unit % parts);
  // whole warps stay together for the shuffles: lanes without a token run along with nothing to do
  const bool on = t < A.n_tokens;
  const int pos = on ? A.positions[t] : -1;
  int slot = -1;
  if (pos >= 0) {
    slot = A.slots ? A.slots[t] : t;
    if (A.slots && slot >= n_slots) {
      if (l == 0) atomicOr(err, WI_DEVERR_BAD_PAGE);
      slot = -1;
    }
  }
  int o0, o1;
  lane_groups(l, R, o0, o1);
  const bool turned = R.interleaved ? 8 * l < R.rotary : 4 * l < (R.rotary >> 1);
  float cs[4], sn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
    if (turned && pos >= 0) {
      // the product's low 64 bits are the fraction of a turn; signed, it is the angle in (-1/2, 1/2] turns
      const long long a = (long long)(R.turn[4 * l + i] * (unsigned long long)pos);
      sincospif((float)(int)(a >> 32) * 4.656612873077393e-10f, &sn[i], &cs[i]);  // 2^-31: half turns
      cs[i] *= R.scale;
      sn[i] *= R.scale;
    }
  }
  const long long k_row = A.slots ? (long long)(slot / page) * Hkv * page + slot % page : (long long)slot * Hkv;
  const int k_step = A.slots ? page : 1;  // rows between a token's kv heads
  const int rows = Hq + 2 * Hkv;
  const int r0 = (int)((long long)rows * part / parts), r1 = (int)((long long)rows * (part + 1) / parts);
  const int most = (rows + parts - 1) / parts;
  for (int base = 0; base < most; base += kWrRows) {
    Lane8 x[kWrRows];
    bf16* to[kWrRows];
#pragma unroll
    for (int i = 0; i < kWrRows; ++i) {
      const int r = r0 + base + i;
      const bf16* from = nullptr;
      to[i] = nullptr;
      if (r < r1 && pos >= 0) {
        if (r < Hq) {
          from = static_cast<const bf16*>(A.q) + (long long)t * A.q_stride + (long long)r * WI_D;
          to[i] = static_cast<bf16*>(A.q_out) + ((long long)t * Hq + r) * WI_D;
        } else if (slot >= 0) {
          const int h = r < Hq + Hkv ? r - Hq : r - Hq - Hkv;
          const long long row = (k_row + (long long)h * k_step) * WI_D;
          if (r < Hq + Hkv) {
            from = static_cast<const bf16*>(A.k) + (long long)t * A.k_stride + (long long)h * WI_D;
            to[i] = static_cast<bf16*>(A.k_out) + row;
          } else {
            from = static_cast<const bf16*>(A.v) + (long long)t * A.v_stride + (long long)h * WI_D;
            to[i] = static_cast<bf16*>(A.v_out) + row;
          }
        }
      }
      x[i].a = x[i].b = make_uint2(0u, 0u);
      if (to[i]) {
        x[i].a = *reinterpret_cast<const uint2*>(from + o0);
        x[i].b = *reinterpret_cast<const uint2*>(from + o1);
      }
    }
#pragma unroll
    for (int i = 0; i < kWrRows; ++i) {
      const int r = r0 + base + i;
      if (r < Hq + Hkv) {
        float a[4], b[4];
        unpack_bf16x4(x[i].a, a);
        unpack_bf16x4(x[i].b, b);
        const bf16* w = static_cast<const bf16*>(r < Hq ? A.q_weight : A.k_weight);
        if (w) {
          float ss = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) ss += a[j] * a[j] + b[j] * b[j];
          // both halves of a warp may hold rows of different kinds: each sums over its own sixteen lanes
          const unsigned mask = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
          const float inv = rsqrtf(ss * (1.f / WI_D) + eps);
          float wa[4], wb[4];
          load_bf16x4(w + o0, wa);
          load_bf16x4(w + o1, wb);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            a[j] = a[j] * inv * wa[j];
            b[j] = b[j] * inv * wb[j];
          }
        }
        if (turned) {
          if (R.interleaved) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float a0 = a[2 * j], a1 = a[2 * j + 1], b0 = b[2 * j], b1 = b[2 * j + 1];
              a[2 * j] = a0 * cs[j] - a1 * sn[j];
              a[2 * j + 1] = a1 * cs[j] + a0 * sn[j];
              b[2 * j] = b0 * cs[2 + j] - b1 * sn[2 + j];
              b[2 * j + 1] = b1 * cs[2 + j] + b0 * sn[2 + j];
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float p = a[j], s = b[j];
              a[j] = p * cs[j] - s * sn[j];
              b[j] = s * cs[j] + p * sn[j];
            }
          }
        }
        x[i].a = pack4(a);
        x[i].b = pack4(b);
      }
      if (to[i]) {
        *reinterpret_cast<uint2*>(to[i] + o0) = x[i].a;
        *reinterpret_cast<uint2*>(to[i] + o1) = x[i].b;
      }
    }
  }
}

// ---------------------------------------------------------------- gather
//
// A copy: sixteen lanes move one 256-byte row with 16-byte loads, and each
// takes kGaRows rows of K and of V at once.  Rows are numbered through over
// all (request, layer, kv head) units, so that one row per unit fills the
// CTAs as well as long units do.
constexpr int kGaThreads = 256;
constexpr int kGaRows = 4;

__global__ void __launch_bounds__(kGaThreads) k_paged_gather(WiPagedGather A, long long rows, int Hkv, int page,
                                                            int n_pages, int max_pages, int* err) {
  constexpr int kStep = kGaThreads / 16;
  const int l = threadIdx.x & 15;
  const int most = max_pages * page, n = (int)A.n;
  const long long r0 = (long long)blockIdx.x * (kStep * kGaRows);
  const long long u0 = r0 / n;
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
      h = (int)(u % Hkv);
      const long long bl = u / Hkv;
      b = (int)(bl / A.layers);
      pool = (bl % A.layers) * n_pages * (long long)Hkv * page;
      len = A.kv_len[b];
      if (len < 0 || len > most) {
        flags |= WI_DEVERR_BAD_LENGTH;
        len = 0;
      }
    }
    const int p = (int)A.pos0 + (int)i;
    if (p < len) {
      const int j = p / page, pg = A.block_table[(long long)b * max_pages + j];
      if (pg < 0 || pg >= n_pages) {
        flags |= WI_DEVERR_BAD_PAGE;
      } else {
        const long long src = (pool + ((long long)pg * Hkv + h) * page + (p - j * page)) * 16 + l;
        kr[k] = __ldg(static_cast<const uint4*>(A.k_pages) + src);
        vr[k] = __ldg(static_cast<const uint4*>(A.v_pages) + src);
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
  k_paged_tables<<<grid, kTabThreads, smem, st>>>(a, g.page, g.n_pages, g.max_pages, err);
  return cudaGetLastError();
}

cudaError_t wi_launch_paged_write(const WiPagedGeom& g, const WiPagedWrite& a, int sms, int* err, cudaStream_t st) {
  // rows per sixteen lanes: as many as leave eight warps per SM, so that few tokens spread over the
  // machine and many share each token's angles among all of its rows
  const int rows = g.Hq + 2 * g.Hkv;
  const long long groups = 16LL * sms;
  long long parts = (groups + a.n_tokens - 1) / a.n_tokens;
  const int widest = (rows + kWrRows - 1) / kWrRows;
  if (parts > widest) parts = widest;
  const long long units = parts * a.n_tokens;
  const long long grid = (units + kWrThreads / 16 - 1) / (kWrThreads / 16);
  k_paged_write<<<(unsigned)grid, kWrThreads, 0, st>>>(a, g.rope, g.Hq, g.Hkv, g.page, g.n_pages * g.page, g.eps,
                                                      (int)parts, err);
  return cudaGetLastError();
}

cudaError_t wi_launch_paged_gather(const WiPagedGeom& g, const WiPagedGather& a, int* err, cudaStream_t st) {
  const int per = kGaThreads / 16 * kGaRows;
  const long long rows = (long long)a.batch * a.layers * g.Hkv * a.n, grid = (rows + per - 1) / per;
  if (grid > 2147483647LL) return cudaErrorInvalidConfiguration;
  k_paged_gather<<<(unsigned)grid, kGaThreads, 0, st>>>(a, rows, g.Hkv, g.page, g.n_pages, g.max_pages, err);
  return cudaGetLastError();
}
