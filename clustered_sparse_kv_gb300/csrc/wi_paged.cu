// wi_paged.cu -- the paged cache's tables, writes and gather.
#include <cuda_runtime.h>

#include "wi_common.cuh"
#include "wi_paged.h"
#include "wi_paged_write.cuh"
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

template <bool INTER, bool FULL, bool AXES>
__global__ void __launch_bounds__(kWrThreads, 6) k_paged_write(const __grid_constant__ WiPagedWrite A,
                                                              const __grid_constant__ WiRope R, int Hq, int Hkv, int page,
                                                              int n_slots, float eps, int parts, int* err) {
  __shared__ __align__(16) unsigned char rows[kWrThreads / 32][kWrStages * kWrBatch];
  pdl_trigger();
  pdl_wait();
  write_rows<INTER, FULL, AXES>(A, R, Hq, Hkv, page, n_slots, eps, parts,
                                (long long)blockIdx.x * (kWrThreads / 32) + (threadIdx.x >> 5), rows[threadIdx.x >> 5], err);
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
  auto* kernel = g.rope.axes > 1
                     ? (g.rope.interleaved ? (full ? k_paged_write<true, true, true> : k_paged_write<true, false, true>)
                                           : (full ? k_paged_write<false, true, true> : k_paged_write<false, false, true>))
                     : (g.rope.interleaved ? (full ? k_paged_write<true, true, false> : k_paged_write<true, false, false>)
                                           : (full ? k_paged_write<false, true, false> : k_paged_write<false, false, false>));
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
