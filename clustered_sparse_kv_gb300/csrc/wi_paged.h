// wi_paged.h -- host-side declarations shared by the paged-cache sources.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "wave_index.h"

// Launch that may be scheduled while the kernel before it in the stream drains (the kernel waits with pdl_wait
// before it reads or writes anything that another one touches).
template <typename... K, typename... A>
inline cudaError_t wi_launch_chained(void (*kernel)(K...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                                     const A&... args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3((unsigned)threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  lc.attrs = at;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, args...);
}

constexpr int kPagedMaxBatch = 4096;
constexpr int kPagedMaxTokens = 1 << 24;  // of a step

// Rotation of a head's pairs: the angle of pair i at position p is p * turn[i] / 2^64 turns, so the whole
// turns drop out of a 64-bit product, and a far position's angle is as good as a near one's: known to 2^-31 of a turn, then
// rounded to fp32.
struct WiRope {
  unsigned long long turn[64];
  float scale;       // on cosine and sine
  int rotary;        // rotated elements, a multiple of 8
  int interleaved;
};

// Geometry of a paged cache, derived from wi_paged_config.
struct WiPagedGeom {
  int Hq, Hkv, G;    // query heads, kv heads, query heads per kv head
  int page;          // positions per page
  int n_pages;
  int max_batch, max_pages;
  float eps;
  WiRope rope;
};

struct WiPagedTables {
  const int32_t* ctx_len;
  const int32_t* new_len;
  const int32_t* free_pages;
  const int32_t* n_free;
  int32_t* block_table;
  int32_t* kv_len;
  int32_t* q_start;
  int32_t* slots;
  int32_t* positions;
  int32_t* n_free_out;
  int batch, free_cap, n_tokens;
};
cudaError_t wi_launch_paged_tables(const WiPagedGeom& g, const WiPagedTables& a, int sms, int* err, cudaStream_t st);

struct WiPagedWrite {
  const void* q;
  const void* k;
  const void* v;
  long long q_stride, k_stride, v_stride;
  const void* q_weight;
  const void* k_weight;
  const int32_t* positions;
  const int32_t* slots;  // null: k_out / v_out are [n_tokens][Hkv][128]
  void* q_out;
  void* k_out;
  void* v_out;
  int n_tokens;
};
cudaError_t wi_launch_paged_write(const WiPagedGeom& g, const WiPagedWrite& a, int sms, int* err, cudaStream_t st);

struct WiPagedGather {
  const void* k_pages;
  const void* v_pages;
  const int32_t* block_table;
  const int32_t* kv_len;
  void* k_out;
  void* v_out;
  int batch, layers;
  long long pos0, n;
};
cudaError_t wi_launch_paged_gather(const WiPagedGeom& g, const WiPagedGather& a, int* err, cudaStream_t st);

struct WiPagedAttn {
  const void* q;
  const void* k_pages;
  const void* v_pages;
  const int32_t* block_table;
  const int32_t* q_start;
  const int32_t* kv_len;
  void* out;
  float* lse;
  int batch, n_tokens;
};
constexpr int kPagedMaxSms = 1024;
constexpr size_t kPagedTicketBytes = kPagedMaxSms * 4;  // at the start of the scratch, zero between calls
// Scratch of the attention, part of the handle: tickets, two partial results per CTA (of an item that the CTA before began,
// and of one that the CTA after goes on with) and what the merge needs to know of the latter.
size_t wi_paged_attention_scratch(int sms);
cudaError_t wi_launch_paged_attention(const WiPagedGeom& g, const WiPagedAttn& a, int sms, void* scratch, int* err,
                                      cudaStream_t st);
