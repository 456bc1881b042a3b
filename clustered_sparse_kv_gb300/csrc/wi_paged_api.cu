// wi_paged_api.cu -- the paged cache's part of the C ABI (include/wave_index.h): argument checks, the
// handle and its scratch.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "wi_common.cuh"
#include "wi_internal.h"
#include "wi_paged.h"

struct wi_paged {
  WiPagedGeom g{};
  int device = 0;
  int sms = 0;
  int* err = nullptr;
  void* scratch = nullptr;  // the attention's
};

namespace {

int fail(int code, const char* fmt, ...) {
  char buf[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  wi_set_error(buf);
  return code;
}

#define WI_CUDA(call)                                                       \
  do {                                                                      \
    cudaError_t e_ = (call);                                                \
    if (e_ != cudaSuccess) {                                                \
      cudaGetLastError();                                                   \
      return fail(WI_ECUDA, "%s: %s", #call, cudaGetErrorString(e_));      \
    }                                                                       \
  } while (0)

bool misaligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// Bytes of device memory that an argument covers.
struct Span {
  const void* at;
  long long bytes;
};

bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return a.at && b.at && a.bytes > 0 && b.bytes > 0 && x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

// Whether an output shares memory with an input or with another output.
template <int N, int M>
bool clash(const Span (&outs)[N], const Span (&ins)[M]) {
  for (int o = 0; o < N; ++o) {
    for (int i = 0; i < M; ++i)
      if (overlap(outs[o], ins[i])) return true;
    for (int q = 0; q < o; ++q)
      if (overlap(outs[o], outs[q])) return true;
  }
  return false;
}

long long pool_bytes(const WiPagedGeom& g) { return (long long)g.n_pages * g.Hkv * g.page * WI_D * 2; }
// ... of 8-bit pools, and of their scales
long long pool8_bytes(const WiPagedGeom& g) { return (long long)g.n_pages * g.Hkv * g.page * WI_D; }
long long scale_bytes(const WiPagedGeom& g) { return (long long)g.n_pages * g.Hkv * (g.page / kGroup); }

// What every call checks first: the handle, and that its device is the current one.
int enter(const wi_paged* pc) {
  wi_set_error("");
  if (!pc) return fail(WI_EINVAL, "paged cache handle is NULL");
  int dev = 0;
  WI_CUDA(cudaGetDevice(&dev));
  if (dev != pc->device) return fail(WI_EINVAL, "the handle belongs to device %d, device %d is current", pc->device, dev);
  return WI_OK;
}

// A call's status.  A launch that fails leaves its error for the next call that asks for the last one: it is taken away.
int launched(const char* what, cudaError_t e) {
  if (e == cudaSuccess) return WI_OK;
  cudaGetLastError();
  return fail(WI_ECUDA, "paged %s launch: %s", what, cudaGetErrorString(e));
}

int bad_batch(const wi_paged* pc, int batch) {
  return fail(WI_EINVAL, "batch (%d) must be in [1, %d]", batch, pc->g.max_batch);
}

// The fraction of a turn that x radians are, in 2^-64 turns: x / 2 pi in two doubles (one alone is off by up to 2^-55 of a
// turn, which a position of 2^31 makes 2^-24), each without its whole turns, which are no rotation.
unsigned long long turn_of(double x) {
  constexpr double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;  // 1 / 2 pi
  const double a = x * hi, b = std::fma(x, lo, std::fma(x, hi, -a));
  auto fraction = [](double v) {
    v -= std::rint(v);  // exact
    const unsigned long long m = (unsigned long long)std::ldexp(std::fabs(v), 64);  // 2^63 at most
    return v < 0 ? 0ull - m : m;
  };
  return fraction(a) + fraction(b);
}

int geom_from_config(const wi_paged_config* c, WiPagedGeom* g) {
  if (!c) return fail(WI_EINVAL, "config is NULL");
  if (c->n_q_heads < 1 || c->n_kv_heads < 1 || c->n_q_heads % c->n_kv_heads)
    return fail(WI_EINVAL, "n_q_heads (%d) must be a positive multiple of n_kv_heads (%d)", c->n_q_heads, c->n_kv_heads);
  if (c->head_dim != WI_D) return fail(WI_EINVAL, "head_dim must be 128 (got %d)", c->head_dim);
  if (c->page_size < 16 || c->page_size % 16)
    return fail(WI_EINVAL, "page_size must be a positive multiple of 16 (got %d)", c->page_size);
  if (c->n_pages < 1 || c->max_batch < 1 || c->max_pages < 1)
    return fail(WI_EINVAL, "n_pages, max_batch and max_pages must be >= 1");
  if (c->rotary_dim < 0 || c->rotary_dim > WI_D || c->rotary_dim % 8)
    return fail(WI_EINVAL, "rotary_dim must be a multiple of 8 in [0, 128] (got %d)", c->rotary_dim);
  if (c->interleaved != 0 && c->interleaved != 1) return fail(WI_EINVAL, "interleaved must be 0 or 1");
  if (c->reserved[0] || c->reserved[1] || c->reserved[2]) return fail(WI_EINVAL, "reserved fields must be zero");
  if (!(c->eps > 0.0) || !((float)c->eps > 0.f) || !std::isfinite((float)c->eps))
    return fail(WI_EINVAL, "eps must be a positive fp32 number");
  if (!std::isfinite((float)c->rope_scale)) return fail(WI_EINVAL, "rope_scale must be finite");
  if (c->rotary_dim > 0 && !c->inv_freq) return fail(WI_EINVAL, "inv_freq is NULL with rotary_dim > 0");
  if (c->n_q_heads / c->n_kv_heads > 8)
    return fail(WI_EUNSUPPORTED, "query heads per kv head must be <= 8 (got %d)", c->n_q_heads / c->n_kv_heads);
  if (c->n_q_heads > 1024) return fail(WI_EUNSUPPORTED, "n_q_heads must be <= 1024 (got %d)", c->n_q_heads);
  if (c->max_batch > kPagedMaxBatch)
    return fail(WI_EUNSUPPORTED, "max_batch must be <= %d (got %d)", kPagedMaxBatch, c->max_batch);
  // row numbers of a pool and positions of a request are 32-bit
  if ((double)c->n_pages * c->n_kv_heads * c->page_size >= 2147483648.0)
    return fail(WI_EUNSUPPORTED, "n_pages * n_kv_heads * page_size must be < 2^31");
  if ((double)c->max_pages * c->page_size >= 2147483648.0)
    return fail(WI_EUNSUPPORTED, "max_pages * page_size must be < 2^31");
  g->Hq = c->n_q_heads;
  g->Hkv = c->n_kv_heads;
  g->G = c->n_q_heads / c->n_kv_heads;
  g->page = c->page_size;
  g->n_pages = c->n_pages;
  g->max_batch = c->max_batch;
  g->max_pages = c->max_pages;
  g->eps = (float)c->eps;
  g->rope.scale = (float)c->rope_scale;
  g->rope.rotary = c->rotary_dim;
  g->rope.interleaved = c->interleaved;
  g->rope.axes = 1;
  for (int i = 0; i < c->rotary_dim / 2; ++i) {
    if (!std::isfinite(c->inv_freq[i])) return fail(WI_EINVAL, "inv_freq[%d] is not finite", i);
    g->rope.turn[i] = turn_of(c->inv_freq[i]);
  }
  return WI_OK;
}

// Zeros, there when the call returns: a memset is queued on the default stream, which the streams of later calls need
// not wait for.
cudaError_t clear(void* p, size_t bytes) {
  const cudaError_t e = cudaMemset(p, 0, bytes);
  return e != cudaSuccess ? e : cudaStreamSynchronize(cudaStreamLegacy);
}

void destroy(wi_paged* pc) {
  if (pc->err) cudaFree(pc->err);
  if (pc->scratch) cudaFree(pc->scratch);
  delete pc;
}

int create_impl(const wi_paged_config* cfg, wi_paged** out) {
  wi_set_error("");
  if (!out) return fail(WI_EINVAL, "out is NULL");
  *out = nullptr;
  WiPagedGeom g{};
  const int rc = geom_from_config(cfg, &g);
  if (rc != WI_OK) return rc;
  int dev = 0, sms = 0;
  WI_CUDA(cudaGetDevice(&dev));
  WI_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  wi_paged* pc = new wi_paged;
  pc->g = g;
  pc->device = dev;
  pc->sms = sms;
  if (cudaMalloc(reinterpret_cast<void**>(&pc->err), 4) != cudaSuccess ||
      cudaMalloc(&pc->scratch, wi_paged_attention_scratch(sms)) != cudaSuccess ||
      clear(pc->err, 4) != cudaSuccess || clear(pc->scratch, kPagedTicketBytes) != cudaSuccess) {
    cudaGetLastError();
    destroy(pc);
    return fail(WI_ENOMEM, "device allocation failed");
  }
  *out = pc;
  return WI_OK;
}

}  // namespace

extern "C" {

int wi_paged_create(const wi_paged_config* cfg, wi_paged** out) {
  try {
    return create_impl(cfg, out);
  } catch (...) {
    if (out) *out = nullptr;
    return fail(WI_ENOMEM, "host allocation failed");
  }
}

int wi_paged_check(wi_paged* pc) {
  const int rc = enter(pc);
  if (rc != WI_OK) return rc;
  WI_CUDA(cudaDeviceSynchronize());
  int herr = 0;
  WI_CUDA(cudaMemcpy(&herr, pc->err, 4, cudaMemcpyDeviceToHost));
  if (!herr) return WI_OK;
  WI_CUDA(clear(pc->err, 4));
  if (herr & WI_DEVERR_MBAR_TIMEOUT) WI_CUDA(clear(pc->scratch, kPagedTicketBytes));  // tickets left behind
  return fail(WI_EDEVICE, "paged cache (flags 0x%x):%s%s%s%s", herr,
              herr & WI_DEVERR_BAD_PAGE ? " a page or slot outside the pool;" : "",
              herr & WI_DEVERR_BAD_LENGTH ? " a length or offset out of range;" : "",
              herr & WI_DEVERR_NO_PAGES ? " more pages needed than are free;" : "",
              herr & WI_DEVERR_MBAR_TIMEOUT ? " a wait timed out;" : "");
}

int wi_paged_axes(wi_paged* pc, int n_axes, const int32_t* axis) {
  wi_set_error("");
  if (!pc) return fail(WI_EINVAL, "paged cache handle is NULL");
  WiRope& r = pc->g.rope;
  if (n_axes < 1 || n_axes > kPagedMaxAxes) return fail(WI_EINVAL, "n_axes (%d) must be in [1, %d]", n_axes, kPagedMaxAxes);
  if (n_axes > 1 && !axis && r.rotary > 0) return fail(WI_EINVAL, "axis is NULL");
  for (int i = 0; n_axes > 1 && i < r.rotary / 2; ++i)
    if (axis[i] < 0 || axis[i] >= n_axes)
      return fail(WI_EINVAL, "axis[%d] (%d) must be in [0, %d)", i, axis[i], n_axes);
  for (int i = 0; i < r.rotary / 2; ++i) r.axis[i] = n_axes > 1 ? (unsigned char)axis[i] : 0;
  r.axes = n_axes;
  return WI_OK;
}

void wi_paged_free(wi_paged* pc) {
  if (!pc) return;
  int dev = -1;
  const bool other = cudaGetDevice(&dev) == cudaSuccess && dev != pc->device && cudaSetDevice(pc->device) == cudaSuccess;
  cudaDeviceSynchronize();
  destroy(pc);
  if (other) cudaSetDevice(dev);
}

int wi_paged_tables(wi_paged* pc, int batch, const int32_t* ctx_len, const int32_t* new_len,
                    const int32_t* free_pages, const int32_t* n_free, int free_cap, int32_t* block_table,
                    int32_t* kv_len, int32_t* q_start, int32_t* slots, int32_t* positions, int n_tokens,
                    int32_t* n_free_out, void* stream) {
  const int rc = enter(pc);
  if (rc != WI_OK) return rc;
  if (batch < 1 || batch > pc->g.max_batch) return bad_batch(pc, batch);
  if (n_tokens < 0 || free_cap < 0) return fail(WI_EINVAL, "n_tokens and free_cap must be >= 0");
  if (n_tokens > kPagedMaxTokens) return fail(WI_EUNSUPPORTED, "n_tokens must be <= %d (got %d)", kPagedMaxTokens, n_tokens);
  if (!ctx_len || !new_len || !n_free || !block_table || !kv_len || !q_start || !n_free_out ||
      (free_cap > 0 && !free_pages) || (n_tokens > 0 && (!slots || !positions)))
    return fail(WI_EINVAL, "a table pointer is NULL");
  const long long B = batch;
  const Span in[4] = {{ctx_len, 4 * B}, {new_len, 4 * B}, {free_pages, 4LL * free_cap}, {n_free, 4}};
  const Span outs[6] = {{block_table, 4 * B * pc->g.max_pages}, {kv_len, 4 * B}, {q_start, 4 * (B + 1)},
                        {slots, 4LL * n_tokens}, {positions, 4LL * n_tokens}, {n_free_out, 4}};
  for (const Span& x : in)
    if (misaligned(x.at, 4)) return fail(WI_EINVAL, "the tables must be 4-byte aligned");
  for (const Span& x : outs)
    if (misaligned(x.at, 4)) return fail(WI_EINVAL, "the tables must be 4-byte aligned");
  if (clash(outs, in)) return fail(WI_EINVAL, "an output shares memory with an input or another output");
  const WiPagedTables a = {ctx_len, new_len, free_pages, n_free,    block_table, kv_len,  q_start,
                           slots,   positions, n_free_out, batch, free_cap,    n_tokens};
  return launched("tables", wi_launch_paged_tables(pc->g, a, pc->sms, pc->err, static_cast<cudaStream_t>(stream)));
}

// The write's checks: into bf16 pools or rows, or with scales into 8-bit pools.
static int write_any(wi_paged* pc, int n_tokens, const void* q, long long q_stride, const void* k, long long k_stride,
                     const void* v, long long v_stride, const void* q_weight, const void* k_weight,
                     const int32_t* positions, const int32_t* slots, void* q_out, void* k_pages, void* v_pages,
                     const WiPagedScales* scales, void* stream) {
  const int rc = enter(pc);
  if (rc != WI_OK) return rc;
  const WiPagedGeom& g = pc->g;
  if (n_tokens < 0) return fail(WI_EINVAL, "n_tokens must be >= 0");
  if (n_tokens == 0) return WI_OK;
  if (n_tokens > kPagedMaxTokens) return fail(WI_EUNSUPPORTED, "n_tokens must be <= %d (got %d)", kPagedMaxTokens, n_tokens);
  if (!q || !k || !v || !positions || !q_out || !k_pages || !v_pages)
    return fail(WI_EINVAL, "q, k, v, positions, q_out, k_pages and v_pages must be non-NULL");
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(q_weight, 16) ||
      misaligned(k_weight, 16) || misaligned(q_out, 16) || misaligned(k_pages, 16) || misaligned(v_pages, 16))
    return fail(WI_EINVAL, "q, k, v, the weights, q_out and the pools must be 16-byte aligned");
  if (misaligned(positions, 4) || misaligned(slots, 4)) return fail(WI_EINVAL, "positions and slots must be 4-byte aligned");
  const long long qw = (long long)g.Hq * WI_D, kw = (long long)g.Hkv * WI_D;
  if (n_tokens > 1 && (q_stride < qw || k_stride < kw || v_stride < kw || q_stride % 8 || k_stride % 8 || v_stride % 8))
    return fail(WI_EINVAL, "token strides must be multiples of 8 and at least a token's heads");
  if (scales && (!slots || !scales->k || !scales->v)) return fail(WI_EINVAL, "slots, k_scales and v_scales must be non-NULL");
  const long long n1 = n_tokens - 1, kb = scales ? pool8_bytes(g) : slots ? pool_bytes(g) : 2 * kw * n_tokens;
  const long long sb = scales ? scale_bytes(g) : 0;
  const bool in_place = q_out == q && (n_tokens == 1 || q_stride == qw);
  const Span in[7] = {{in_place ? nullptr : q, 2 * (n1 * q_stride + qw)}, {k, 2 * (n1 * k_stride + kw)},
                      {v, 2 * (n1 * v_stride + kw)}, {q_weight, 2 * WI_D}, {k_weight, 2 * WI_D},
                      {positions, 4LL * g.rope.axes * n_tokens}, {slots, 4LL * n_tokens}};
  const Span outs[5] = {{q_out, 2 * qw * n_tokens}, {k_pages, kb}, {v_pages, kb}, {scales ? scales->k : nullptr, sb},
                        {scales ? scales->v : nullptr, sb}};
  if (clash(outs, in))
    return fail(WI_EINVAL, "an output shares memory with an input or another output (q_out may be q itself where q's "
                           "tokens are contiguous)");
  const WiPagedWrite a = {q,     k,     v,       q_stride, k_stride, v_stride, q_weight, k_weight, positions,
                          slots, q_out, k_pages, v_pages,  n_tokens};
  if (scales)
    return launched("write8", wi_launch_paged_write8(g, a, *scales, pc->sms, pc->err, static_cast<cudaStream_t>(stream)));
  return launched("write", wi_launch_paged_write(g, a, pc->sms, pc->err, static_cast<cudaStream_t>(stream)));
}

int wi_paged_write(wi_paged* pc, int n_tokens, const void* q, long long q_stride, const void* k, long long k_stride,
                   const void* v, long long v_stride, const void* q_weight, const void* k_weight,
                   const int32_t* positions, const int32_t* slots, void* q_out, void* k_pages, void* v_pages,
                   void* stream) {
  return write_any(pc, n_tokens, q, q_stride, k, k_stride, v, v_stride, q_weight, k_weight, positions, slots, q_out,
                   k_pages, v_pages, nullptr, stream);
}

int wi_paged_write8(wi_paged* pc, int n_tokens, const void* q, long long q_stride, const void* k, long long k_stride,
                    const void* v, long long v_stride, const void* q_weight, const void* k_weight,
                    const int32_t* positions, const int32_t* slots, void* q_out, void* k_pages, void* v_pages,
                    void* k_scales, void* v_scales, void* stream) {
  const WiPagedScales s = {static_cast<unsigned char*>(k_scales), static_cast<unsigned char*>(v_scales)};
  return write_any(pc, n_tokens, q, q_stride, k, k_stride, v, v_stride, q_weight, k_weight, positions, slots, q_out,
                   k_pages, v_pages, &s, stream);
}

static int attention_any(wi_paged* pc, int batch, int n_tokens, const void* q, const void* k_pages, const void* v_pages,
                         const WiPagedScales* scales, const int32_t* block_table, const int32_t* q_start,
                         const int32_t* kv_len, void* out, float* lse, void* stream) {
  const int rc = enter(pc);
  if (rc != WI_OK) return rc;
  if (batch < 1 || batch > pc->g.max_batch) return bad_batch(pc, batch);
  if (n_tokens < 0) return fail(WI_EINVAL, "n_tokens must be >= 0");
  if (n_tokens == 0) return WI_OK;
  if (n_tokens > kPagedMaxTokens) return fail(WI_EUNSUPPORTED, "n_tokens must be <= %d (got %d)", kPagedMaxTokens, n_tokens);
  if (!q || !k_pages || !v_pages || !block_table || !q_start || !kv_len || !out)
    return fail(WI_EINVAL, "q, the pools, block_table, q_start, kv_len and out must be non-NULL");
  if (misaligned(q, 16) || misaligned(k_pages, 16) || misaligned(v_pages, 16) || misaligned(out, 16))
    return fail(WI_EINVAL, "q, the pools and out must be 16-byte aligned");
  if (misaligned(block_table, 4) || misaligned(q_start, 4) || misaligned(kv_len, 4) || misaligned(lse, 4))
    return fail(WI_EINVAL, "the tables and lse must be 4-byte aligned");
  const WiPagedGeom& g = pc->g;
  if (scales && (!scales->k || !scales->v)) return fail(WI_EINVAL, "k_scales and v_scales must be non-NULL");
  const long long qb = 2LL * n_tokens * g.Hq * WI_D;
  const long long kb = scales ? pool8_bytes(g) : pool_bytes(g), sb = scales ? scale_bytes(g) : 0;
  const Span in[8] = {{q, qb}, {k_pages, kb}, {v_pages, kb}, {block_table, 4LL * batch * g.max_pages},
                      {q_start, 4LL * (batch + 1)}, {kv_len, 4LL * batch}, {scales ? scales->k : nullptr, sb},
                      {scales ? scales->v : nullptr, sb}};
  const Span outs[2] = {{out, qb}, {lse, 4LL * n_tokens * g.Hq}};
  if (clash(outs, in)) return fail(WI_EINVAL, "out or lse shares memory with an input or with the other");
  const WiPagedAttn a = {q, k_pages, v_pages, block_table, q_start, kv_len, out, lse, batch, n_tokens};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (scales)
    return launched("attention8", wi_launch_paged_attention8(g, a, *scales, pc->sms, pc->scratch, pc->err, st));
  return launched("attention", wi_launch_paged_attention(g, a, pc->sms, pc->scratch, pc->err, st));
}

int wi_paged_attention(wi_paged* pc, int batch, int n_tokens, const void* q, const void* k_pages,
                       const void* v_pages, const int32_t* block_table, const int32_t* q_start,
                       const int32_t* kv_len, void* out, float* lse, void* stream) {
  return attention_any(pc, batch, n_tokens, q, k_pages, v_pages, nullptr, block_table, q_start, kv_len, out, lse, stream);
}

int wi_paged_attention8(wi_paged* pc, int batch, int n_tokens, const void* q, const void* k_pages,
                        const void* v_pages, const void* k_scales, const void* v_scales, const int32_t* block_table,
                        const int32_t* q_start, const int32_t* kv_len, void* out, float* lse, void* stream) {
  const WiPagedScales s = {static_cast<unsigned char*>(const_cast<void*>(k_scales)),
                           static_cast<unsigned char*>(const_cast<void*>(v_scales))};
  return attention_any(pc, batch, n_tokens, q, k_pages, v_pages, &s, block_table, q_start, kv_len, out, lse, stream);
}

static int gather_any(wi_paged* pc, int batch, int layers, const void* k_pages, const void* v_pages,
                      const WiPagedScales* scales, const int32_t* block_table, const int32_t* kv_len, long long pos0,
                      long long n, void* k_out, void* v_out, void* stream) {
  const int rc = enter(pc);
  if (rc != WI_OK) return rc;
  const WiPagedGeom& g = pc->g;
  if (batch < 1 || batch > g.max_batch) return bad_batch(pc, batch);
  if (layers < 1 || layers > 65536) return fail(WI_EINVAL, "layers (%d) must be in [1, 65536]", layers);
  const long long most = (long long)g.max_pages * g.page;
  if (pos0 < 0 || n < 0 || pos0 > most || n > most - pos0)
    return fail(WI_EINVAL, "positions [pos0, pos0 + n) must lie in [0, max_pages * page_size = %lld)", most);
  if (n == 0) return WI_OK;
  const int rows_log2 = scales ? 36 : 37;  // 32 or 64 rows a block, 2^31 blocks
  if ((double)batch * layers * g.Hkv * (double)n >= std::ldexp(1.0, rows_log2))
    return fail(WI_EUNSUPPORTED, "batch * layers * n_kv_heads * n must be < 2^%d", rows_log2);
  if (!k_pages || !v_pages || !block_table || !kv_len || !k_out || !v_out)
    return fail(WI_EINVAL, "the pools, block_table, kv_len, k_out and v_out must be non-NULL");
  if (misaligned(k_pages, 16) || misaligned(v_pages, 16) || misaligned(k_out, 16) || misaligned(v_out, 16))
    return fail(WI_EINVAL, "the pools, k_out and v_out must be 16-byte aligned");
  if (misaligned(block_table, 4) || misaligned(kv_len, 4)) return fail(WI_EINVAL, "the tables must be 4-byte aligned");
  if (scales && (!scales->k || !scales->v)) return fail(WI_EINVAL, "k_scales and v_scales must be non-NULL");
  const long long ob = 2LL * batch * layers * g.Hkv * n * WI_D;
  const long long kb = layers * (scales ? pool8_bytes(g) : pool_bytes(g)), sb = scales ? layers * scale_bytes(g) : 0;
  const Span in[6] = {{k_pages, kb}, {v_pages, kb}, {block_table, 4LL * batch * g.max_pages}, {kv_len, 4LL * batch},
                      {scales ? scales->k : nullptr, sb}, {scales ? scales->v : nullptr, sb}};
  const Span outs[2] = {{k_out, ob}, {v_out, ob}};
  if (clash(outs, in)) return fail(WI_EINVAL, "k_out or v_out shares memory with an input or with the other");
  const WiPagedGather a = {k_pages, v_pages, block_table, kv_len, k_out, v_out, batch, layers, pos0, n};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (scales) return launched("gather8", wi_launch_paged_gather8(g, a, *scales, pc->sms, pc->err, st));
  return launched("gather", wi_launch_paged_gather(g, a, pc->err, st));
}

int wi_paged_gather(wi_paged* pc, int batch, int layers, const void* k_pages, const void* v_pages,
                    const int32_t* block_table, const int32_t* kv_len, long long pos0, long long n, void* k_out,
                    void* v_out, void* stream) {
  return gather_any(pc, batch, layers, k_pages, v_pages, nullptr, block_table, kv_len, pos0, n, k_out, v_out, stream);
}

int wi_paged_gather8(wi_paged* pc, int batch, int layers, const void* k_pages, const void* v_pages,
                     const void* k_scales, const void* v_scales, const int32_t* block_table, const int32_t* kv_len,
                     long long pos0, long long n, void* k_out, void* v_out, void* stream) {
  const WiPagedScales s = {static_cast<unsigned char*>(const_cast<void*>(k_scales)),
                           static_cast<unsigned char*>(const_cast<void*>(v_scales))};
  return gather_any(pc, batch, layers, k_pages, v_pages, &s, block_table, kv_len, pos0, n, k_out, v_out, stream);
}

}  // extern "C"
