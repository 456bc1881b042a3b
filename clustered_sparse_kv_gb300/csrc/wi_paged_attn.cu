// wi_paged_attn.cu -- attention of new tokens over the paged cache.
#include <cuda_runtime.h>

#include "wi_common.cuh"
#include "wi_paged.h"

namespace {

constexpr int kWarps = 8;

// The plain form on the CUDA cores: a warp per (token, query head), one pass over its keys with the running
// maximum and sum of the softmax; a lane holds four of the 128 elements.
__global__ void __launch_bounds__(kWarps * 32) k_paged_attention(WiPagedAttn A, int Hq, int Hkv, int page, int n_pages,
                                                                int max_pages, int* err) {
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < A.batch; b += kWarps * 32)
      if (A.q_start[b] < 0 || A.q_start[b + 1] < A.q_start[b] || A.q_start[b + 1] > A.n_tokens)
        atomicOr(err, WI_DEVERR_BAD_LENGTH);
  const long long row = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = (int)(row / Hq), h = (int)(row % Hq);
  if (t >= A.n_tokens) return;
  int lo = 0, hi = A.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (A.q_start[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int s0 = A.q_start[lo], s1 = A.q_start[lo + 1], kv = A.kv_len[lo];
  if (t < s0 || t >= s1) return;  // behind the last request
  if (kv < 0 || (long long)kv > (long long)max_pages * page) {
    if (lane == 0) atomicOr(err, WI_DEVERR_BAD_LENGTH);
    return;
  }
  const int last = kv - (s1 - s0) + (t - s0);
  const int kh = h / (Hq / Hkv);
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f};
  load_bf16x4(static_cast<const bf16*>(A.q) + row * WI_D + 4 * lane, q);
  float m = -INFINITY, z = 0.f;
  for (int p = 0; p <= last; ++p) {
    const int pg = A.block_table[(long long)lo * max_pages + p / page];
    if (pg < 0 || pg >= n_pages) {
      if (lane == 0) atomicOr(err, WI_DEVERR_BAD_PAGE);
      continue;
    }
    const long long at = (((long long)pg * Hkv + kh) * page + p % page) * WI_D + 4 * lane;
    float k[4], v[4];
    load_bf16x4(static_cast<const bf16*>(A.k_pages) + at, k);
    load_bf16x4(static_cast<const bf16*>(A.v_pages) + at, v);
    const float s = warp_sum(q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3]) * 0.08838834764831845f;
    const float top = fmaxf(m, s), keep = expf(m - top), w = expf(s - top);
    m = top;
    z = z * keep + w;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = o[i] * keep + w * v[i];
  }
  const float inv = z > 0.f ? 1.f / z : 0.f;
  const __nv_bfloat162 a = __floats2bfloat162_rn(o[0] * inv, o[1] * inv), b = __floats2bfloat162_rn(o[2] * inv, o[3] * inv);
  uint2 w;
  w.x = *reinterpret_cast<const uint32_t*>(&a);
  w.y = *reinterpret_cast<const uint32_t*>(&b);
  *reinterpret_cast<uint2*>(static_cast<bf16*>(A.out) + row * WI_D + 4 * lane) = w;
  if (A.lse && lane == 0) A.lse[row] = z > 0.f ? m + logf(z) : -INFINITY;
}

}  // namespace

cudaError_t wi_launch_paged_attention(const WiPagedGeom& g, const WiPagedAttn& a, int sms, int* err, cudaStream_t st) {
  (void)sms;
  const long long rows = (long long)a.n_tokens * g.Hq;
  k_paged_attention<<<(unsigned)((rows + kWarps - 1) / kWarps), kWarps * 32, 0, st>>>(a, g.Hq, g.Hkv, g.page, g.n_pages,
                                                                                   g.max_pages, err);
  return cudaGetLastError();
}
