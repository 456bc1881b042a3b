// wi_paged8_attn.cu -- attention of new tokens over the paged cache in 8 bits.
//
// out = softmax(q K^T / sqrt(128)) V over the positions a token sees, K and V
// the pools' values times their group's scale.  A CTA takes one token and one
// kv head: its warps take every fourth run of 32 positions, a lane a key, for
// the scores of the head's queries, and then a lane four columns of the values.
#include <cuda_runtime.h>

#include "wi_common.cuh"
#include "wi_e4m3.cuh"
#include "wi_internal.h"
#include "wi_paged.h"
#include "wi_paged8.h"
#include "wi_pipe.cuh"

namespace {

constexpr int kWarps = 4;
constexpr int kMaxG = 8;
constexpr float kScaleLog2 = 0.08838834764831845f * 1.4426950408889634f;  // log2(e) / sqrt(128)
constexpr float kLn2 = 0.6931471805599453f;

__global__ void __launch_bounds__(32 * kWarps) k_paged_attention8(WiPagedAttn A, WiPagedScales S, int Hq, int Hkv, int G,
                                                                  int page, int n_pages, int max_pages, int* err) {
  __shared__ float q[kMaxG][WI_D];
  __shared__ float part[kWarps][kMaxG][WI_D + 2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  pdl_wait();
  const int t = blockIdx.x / Hkv, kh = blockIdx.x - t * Hkv;
  int b = 0, s0 = 0, n = 0, kv = 0;
  bool found = false;
  for (; b < A.batch; ++b) {
    s0 = A.q_start[b];
    const int s1 = A.q_start[b + 1];
    if (s1 < s0) {
      if (blockIdx.x == 0 && tid == 0) atomicOr(err, WI_DEVERR_BAD_LENGTH);
      break;
    }
    kv = A.kv_len[b];
    const bool ok = s0 >= 0 && s1 <= A.n_tokens && kv >= 0 && (long long)kv <= (long long)max_pages * page;
    if (!ok && blockIdx.x == 0 && tid == 0) atomicOr(err, WI_DEVERR_BAD_LENGTH);
    if (t >= s0 && t < s1 && !found) {
      if (!ok) return;
      n = s1 - s0;
      found = true;
      if (blockIdx.x != 0) break;
    }
    if (found) continue;
  }
  if (!found) return;
  // (block 0 went on to look at every request: its own again)
  if (blockIdx.x == 0) {
    for (b = 0; !(A.q_start[b] <= t && t < A.q_start[b + 1]); ++b) {
    }
    s0 = A.q_start[b];
    n = A.q_start[b + 1] - s0;
    kv = A.kv_len[b];
  }
  const int end = (int)((long long)kv - n + (t - s0)) + 1;  // positions that the token sees: 0 or less, none
  for (int i = tid; i < G * WI_D; i += 32 * kWarps)
    q[i / WI_D][i % WI_D] = __bfloat162float(static_cast<const bf16*>(A.q)[((long long)t * Hq + kh * G) * WI_D + i]) * kScaleLog2;
  __syncthreads();
  float m[kMaxG], z[kMaxG], acc[kMaxG][4];
#pragma unroll
  for (int g = 0; g < kMaxG; ++g) {
    m[g] = -INFINITY;
    z[g] = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[g][c] = 0.f;
  }
  for (int p0 = warp * 32; p0 < end; p0 += 32 * kWarps) {
    const int p = p0 + lane;
    long long row = -1;
    float x[kMaxG];
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) x[g] = 0.f;
    float vscale = 0.f;
    if (p < end) {
      const int j = p / page;
      int pg = A.block_table[(long long)b * max_pages + j];
      if (pg < 0 || pg >= n_pages) {
        atomicOr(err, WI_DEVERR_BAD_PAGE);
        pg = 0;
      }
      const long long head = (long long)pg * Hkv + kh;
      row = head * page + (p - j * page);
      const long long group = head * (page / kGroup) + (p - j * page) / kGroup;
      const float kscale = pow2(scale_exponent(S.k[group]));
      vscale = pow2(scale_exponent(S.v[group]));
      const uint4* k = static_cast<const uint4*>(A.k_pages) + row * 8;
      for (int c = 0; c < 8; ++c) {
        const uint4 w = k[c];
        const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 v = e4m3x2_to_f32x2(e[i >> 1] >> (16 * (i & 1)) & 0xffffu);
          const int d = c * 16 + 2 * i;
          for (int g = 0; g < G; ++g) x[g] += q[g][d] * v.x + q[g][d + 1] * v.y;
        }
      }
#pragma unroll
      for (int g = 0; g < kMaxG; ++g) x[g] *= kscale;
    }
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) {
      if (p >= end) x[g] = -INFINITY;
      const float top = fmaxf(m[g], warp_max(x[g])), ref = top == -INFINITY ? 0.f : top;
      const float f = exp2f(m[g] - ref);
      m[g] = top;
      x[g] = exp2f(x[g] - ref);
      z[g] = z[g] * f + warp_sum(x[g]);
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[g][c] *= f;
    }
    for (int i = 0; i < 32 && p0 + i < end; ++i) {
      const long long r = __shfl_sync(0xffffffffu, row, i);
      const float f = __shfl_sync(0xffffffffu, vscale, i);
      const uint32_t w = static_cast<const uint32_t*>(A.v_pages)[r * 32 + lane];
      const float2 a = e4m3x2_to_f32x2(w & 0xffffu), c = e4m3x2_to_f32x2(w >> 16);
      const float v[4] = {a.x * f, a.y * f, c.x * f, c.y * f};
#pragma unroll
      for (int g = 0; g < kMaxG; ++g) {
        const float y = __shfl_sync(0xffffffffu, x[g], i);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[g][k] += y * v[k];
      }
    }
  }
#pragma unroll
  for (int g = 0; g < kMaxG; ++g) {
    if (g >= G) break;
#pragma unroll
    for (int c = 0; c < 4; ++c) part[warp][g][4 * lane + c] = acc[g][c];
    part[warp][g][WI_D] = m[g];
    part[warp][g][WI_D + 1] = z[g];
  }
  __syncthreads();
  for (int g = 0; g < G; ++g) {
    float top = -INFINITY, sum = 0.f, o = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part[w][g][WI_D]);
    const float ref = top == -INFINITY ? 0.f : top;
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2f(part[w][g][WI_D] - ref);
      sum += f * part[w][g][WI_D + 1];
      o += f * part[w][g][tid];
    }
    const long long at = (long long)t * Hq + kh * G + g;
    static_cast<bf16*>(A.out)[at * WI_D + tid] = __float2bfloat16_rn(sum == 0.f ? 0.f : o / sum);
    if (A.lse && tid == 0) A.lse[at] = sum == 0.f ? -INFINITY : top * kLn2 + logf(sum);
  }
}

}  // namespace

cudaError_t wi_launch_paged_attention8(const WiPagedGeom& g, const WiPagedAttn& a, const WiPagedScales& s, int sms,
                                       void* scratch, int* err, cudaStream_t st) {
  if (wi_paged_few(g, a)) return wi_launch_paged_few(g, a, s, sms, scratch, err, st);
  return wi_launch_chained(k_paged_attention8, dim3((unsigned)(a.n_tokens * (long long)g.Hkv)), 32 * kWarps, 0, st, a, s,
                           g.Hq, g.Hkv, g.G, g.page, g.n_pages, g.max_pages, err);
}
