// wi_paged8_attn.cu -- attention of new tokens over the paged cache in 8 bits, on tiles of 128 rows.
//
// out = softmax(q K^T / sqrt(128)) V over the positions a token sees, K and V
// the pools' values times their group's scale.  Rows, items, runs and the two
// softmax chains are those of the bf16 attention (wi_paged_attn.cu); what
// differs is how the operands reach the tensor cores.
//
// S = Q K^T in e4m3: keys as they lie in the cache, queries as two e4m3 pieces, a
// first one of four significant bits and the rest of four, which a bf16 query is
// exactly (over the row's largest element; what is below 2^-17 of that may be
// lost).  Two products of half the time each, so S costs what it does in bf16, and
// no key is ever widened.  A column's scale is its group's: a score is
// S 2^(e_row + e_group), one multiplier per sixteen columns.
//
// O += P V in f16: e4m3 pieces of P would lose what weighs less than 2^-18 of the
// row's largest, which a sink of attention makes most of the row, and three of
// them would cost more than bf16 does.  So two warps widen a block's values (a
// conversion of two values an instruction, exact) on their way from the copy's
// stage to the product's, once for both chains.  The value's scale goes into
// the weight, p' = 2^(score + e - m), and out of the row's sum, l += p' 2^-e.
//
// Warps of a CTA (384 threads):
//   0-3, 4-7  softmax, one thread per row of chain 0 / chain 1; they also cut the
//             queries of their tile into pieces
//   8         TMA: key and value blocks, box by box, and their groups' scales
//   9         issues tcgen05.mma
//   10-11     widen the values, and clean what not every row sees
// A chain's weights of a block come in two halves of 64 positions, so that the
// first half's product with the values runs while the second half's weights are
// worked out; O then waits for half a product and the next scores.
//
// What bounds it, 32 query and 8 kv heads on one GB300: the chain of scores,
// weights and product of either tile between two of its turns on the tensor
// cores, which are active 57% of the time (2048 tokens behind 14K positions 392
// us, 1300 TFLOP/s; behind 129K 3.1 - 3.2 ms; 8192 fresh tokens 457 us).  Of 3050
// cycles a block takes, a chain spends 1600 on weights (2 x 670 where the other
// chain does not want the special function units too) and 1400 waiting: 770 for the
// tensor cores, the rest for barriers.  Shared memory, at 128 bytes a cycle, is in
// use for 2180 of them: operands 1540, copies and widening 640.  (The second half's
// weights through it, to let the next scores in beside them: 420 us for 403.)
// A segment's start and end cost 10000 cycles
// (queries cut into pieces 4000 of them, outputs stored row by row 4500).
// The way here, 2048 tokens behind 14K unless said: two warps widening a word at a
// time 498 us, all loads in front of the stores 455; scales read ahead of the
// scores 456 (behind 129K 3.41 ms, 3.74 before); blocks that need no mask and no new
// reference in code of their own 424; queries by TMA, cut by a short loop 406; what a
// product needs made ready in front of the wait for its weights 396 (403).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>

#include "wi_common.cuh"
#include "wi_e4m3.cuh"
#include "wi_internal.h"
#include "wi_paged.h"
#include "wi_paged8.h"
#include "wi_paged_merge.cuh"
#include "wi_paged_walk.cuh"
#include "wi_pipe.cuh"
#include "wi_tc.cuh"

namespace {

constexpr int kKStages = 3, kVStages = 2, kWStages = 2, kScaleSlots = 8;
constexpr int kBlockBytes = kRows * WI_D;       // a block of keys or values in 8 bits, a piece of a tile's queries
constexpr int kWideBytes = kRows * WI_D * 2;    // a block of values in f16: [group of 8 rows][half of 64 columns][8][128 B]
constexpr int kSoftWarps = 8;
constexpr int kThreads = 32 * (kSoftWarps + 4);
constexpr int kWideWarps = 2;
constexpr int kGroups = kRows / kGroup;         // of a block
constexpr int kHalf = kRows / 2;                // positions of a step: the first half's product runs while the second half's weights are worked out
constexpr float kScaleLog2 = 0.08838834764831845f * 1.4426950408889634f;  // log2(e) / sqrt(128)
constexpr int kLead = 4;                        // units in front of an item's blocks, for what its start and end cost
// What the largest item may have above an equal run, where each item is a run (sixteen requests' four tokens over 2000 positions
// 37.8 us whole, 46.1 cut; eight requests' sixteen over 500 - 1500 25.3 cut, 28.1 with a slack of sixteen).
constexpr int kSlack = 8;
constexpr int kWhole = 4;                       // blocks up to which one request's items of few rows are not cut
// Blocks that one segment has at most: the tensor cores' additions cut bits off, so longer sums are added up in fp32.  Sums of
// numbers of one sign come out too small by 3e-4 of themselves after 1024 blocks, by 7e-4 after 2048 and more (with 512 at most
// 1.6e-4, and 2048 tokens behind 129K 3170 us for 3120; with 256 6e-5 and 3240).
constexpr int kLongest = 2048;
// A reference makes the row's largest weight 2^4 (for values' scales of 2^-64 or more): f16 holds a weight to 2^-11 of itself
// down to 2^-18 of that, and to 2^-29 of it below.  A row takes a new one when half a block's weights add up to more than f16
// takes, or its sum (through values of a tiny scale) to more than kFarMost.  A larger first weight would hold more and leave
// less room above it, and new references cost time: seven mixed requests 173 us, with 2^5 178, with 2^6 183, with 2^8 201.
constexpr float kTop = 4.f, kAgain = 60000.f, kFar = 64.f + kTop, kFarMost = 0x1p90f;

template <bool LONG>
using Walk = WalkOver<kLead, 2, LONG ? kLongest : 0>;

struct Smem {
  uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages], w_full[kWStages], w_empty[kWStages];
  uint64_t scale_full[kScaleSlots];
  uint64_t q_raw, q_empty, q_full;  // the queries as they are have come; nobody reads their pieces any more; the pieces are there
  // Of a chain: a block's scores are there; the weights of half of it are; the first half's product is done.
  uint64_t s_full[2], p_ready[2][2], pv_done[2];
  uint64_t o_full[2], drained;
  uint32_t tmem_base;
  int last;                 // this CTA merges the item that it just added to
  int poison[8];            // segment number + 1 of the last segment (modulo 8) with a NaN value
  long long scan[2 * (kThreads / 32)];
  Run run;
  Req reqs[2][kSoftWarps];  // of the softmax warps' segments, this one's and the next one's in turn
  // of a block's groups: 2^e of the keys, e of the values, 2^-e of the values.  A slot is written again eight blocks on,
  // behind the scores of the block three before that, which come behind the weights of this one.
  struct Slot {
    float k[kGroups];
    float2 e[kGroups];  // (the same number twice)
    float back[kGroups];
  };
  alignas(16) Slot scale[kScaleSlots];
  float q_scale[2][kRows];
  float xch[2][2][kRows];   // maximum and sum of a row, from chain to chain: [chain][m, l]
  alignas(1024) unsigned char q[2][2][kBlockBytes];   // [tile][piece]; before that [tile][half of 64 columns] in bf16
  unsigned char k[kKStages][kBlockBytes];
  unsigned char v[kVStages][kBlockBytes];
  unsigned char w[kWStages][kWideBytes];
};
static_assert(offsetof(Smem, q) % 1024 == 0, "tiles must start 1024-byte aligned");
static_assert(sizeof(Smem) <= 232448, "shared memory");

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 w = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&w);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 w = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&w);
}

__device__ __forceinline__ void soft_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftWarps * 32) : "memory"); }

// Scores behind column `seen` of 64 are not seen.
__device__ __forceinline__ void mask_scores(uint32_t (&s)[2][32], int seen) {
#pragma unroll
  for (int i = 0; i < 64; ++i)
    if (i > seen) s[i >> 5][i & 31] = 0xFF800000u;  // -infinity
}

// The scales of two of a block's groups as the weights take them, asked for one step ahead of their use: of the keys, the
// values' exponents twice, for packed arithmetic, and the inverse of the values'.
struct Scales {
  ulonglong2 e;
  float2 k, back;
  __device__ __forceinline__ void load(const Smem::Slot& from, int g0) {
    k = *reinterpret_cast<const float2*>(&from.k[g0]);
    e = *reinterpret_cast<const ulonglong2*>(&from.e[g0]);
    back = *reinterpret_cast<const float2*>(&from.back[g0]);
  }
};

// What a group's scores are multiplied by: its keys' scale times the row's factor, which may leave fp32 together (a row of
// zeros over a group of zeros).  No less than the smallest normal number: a score that small is nothing, but 0 would make NaN of
// the scores that stand at minus infinity.  A row's factor that is no number stays none.
__device__ __forceinline__ float factor_of(float k_scale, float q_scale) {
  float f;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(f) : "f"(k_scale * q_scale), "f"(0x1p-126f));
  return f;
}

// The reference that 64 scores ask for: the largest score + e less kTop, and the largest score less kFar.
__device__ __forceinline__ float top_of(const uint32_t (&s)[2][32], const Smem::Slot& x8, int g0, float q_scale) {
  float best = -INFINITY;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const uint32_t* x = s[g >> 1] + (g & 1) * 16;
    float t = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
#pragma unroll
    for (int i = 2; i < 16; i += 2) t = max3(t, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
    t *= factor_of(x8.k[g0 + g], q_scale);
    best = max3(best, t + (x8.e[g0 + g].x - kTop), t - kFar);
  }
  return best;
}

// 32 scores, two groups of columns, to weights 2^(score + e - ref): added to `sum`, and over the values' scale to `low`, and
// as f16 to 16 columns of P.
__device__ __forceinline__ void weights(const uint32_t (&s)[32], uint32_t tp, const Scales& x8, float q_scale, uint64_t ref2,
                                        float& sum, float& low) {
  uint32_t p[16];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const float f = factor_of(g ? x8.k.y : x8.k.x, q_scale);
    const uint64_t f2 = pair(f, f), e2 = add2(g ? x8.e.y : x8.e.x, ref2);
    uint64_t z[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t x = fma2(pair(s[16 * g + 2 * i], s[16 * g + 2 * i + 1]), f2, e2);
      const float a = ex2(lo_of(x)), b = ex2(hi_of(x));
      z[i & 1] = i < 2 ? pair(a, b) : add2(z[i & 1], pair(a, b));
      p[8 * g + i] = pack_f16(a, b);
    }
    const uint64_t z2 = add2(z[0], z[1]);
    const float zs = lo_of(z2) + hi_of(z2);
    sum += zs;
    low += zs * (g ? x8.back.y : x8.back.x);
  }
  tmem_st16_nowait(tp, p);
}

// Sixteen elements of a query, in two words of e4m3 pieces each.  Through f16: scaled by the row's power of two, it holds a
// bf16 element whole, down to 2^-24.
__device__ __forceinline__ void cut16(const uint4& x, const uint4& y, float f, uint4* hi, uint4* lo) {
  const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  uint32_t h[4], r[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t p[2], q[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t v = pack_f16(bf16_lo(w[2 * k + c]) * f, bf16_hi(w[2 * k + c]) * f);
      p[c] = e4m3x2_of_f16x2(v);
      const uint32_t back = e4m3x2_to_f16x2(p[c]);
      const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&back));
      q[c] = e4m3x2_of_f16x2(*reinterpret_cast<const uint32_t*>(&d));
    }
    h[k] = __byte_perm(p[0], p[1], 0x5410);
    r[k] = __byte_perm(q[0], q[1], 0x5410);
  }
  *hi = make_uint4(h[0], h[1], h[2], h[3]);
  *lo = make_uint4(r[0], r[1], r[2], r[3]);
}

// A row of a tile's queries, from the bf16 in `tile` (as TMA brings them: two halves of 64 columns, rows of 128 bytes) to two
// e4m3 pieces in the same place; a row's pieces lie where its own elements lay.  Returns the factor of its scores.  A row of
// infinities or NaN gets one that is no number, a row of no token pieces of zeros.  Short loops: the code is cold when a
// segment ends (unrolled it took 5300 cycles).
__device__ __forceinline__ float cut_query(unsigned char* tile, bool live, int row) {
  unsigned char* const first = tile + row * WI_D;
  unsigned char* const second = first + kBlockBytes;
  const int turn = (row & 7) << 4;
  uint32_t top = 0;
#pragma unroll 2
  for (int c = 0; c < 8; ++c) {
    const int at = (c << 4) ^ turn;  // (without the swizzle's turn, all rows from the same banks)
    const uint4 x = *reinterpret_cast<const uint4*>(first + at), y = *reinterpret_cast<const uint4*>(second + at);
    const uint32_t m = 0x7fff7fffu;
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & m, x.y & m), __vmaxu2(x.z & m, x.w & m)));
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(y.x & m, y.y & m), __vmaxu2(y.z & m, y.w & m)));
  }
  top = max(top & 0xffffu, top >> 16);
  const bool good = live && top < 0x7f80u;
  // the row's largest element lies in [128, 256)
  const int e = min(max((int)(top >> 7) - 127 - 7, -126), 126);
  const float f = pow2(-e);
  uint4 rest[8];  // the second half, which the first half's pieces would run over
#pragma unroll
  for (int c = 0; c < 8; ++c) rest[c] = *reinterpret_cast<const uint4*>(second + ((c << 4) ^ turn));
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
  for (int c = 0; c < 8; ++c) {
    uint4 x, y, hi, lo;
    if (c < 4) {
      x = *reinterpret_cast<const uint4*>(first + ((2 * c << 4) ^ turn));
      y = *reinterpret_cast<const uint4*>(first + ((2 * c + 1 << 4) ^ turn));
    } else {
      x = rest[0];
      y = rest[1];
#pragma unroll
      for (int k = 0; k < 6; ++k) rest[k] = rest[k + 2];
    }
    cut16(x, y, f, &hi, &lo);
    *reinterpret_cast<uint4*>(first + ((c << 4) ^ turn)) = good ? hi : none;
    *reinterpret_cast<uint4*>(second + ((c << 4) ^ turn)) = good ? lo : none;
  }
  return !live ? 1.f : good ? pow2(e) * kScaleLog2 : __uint_as_float(0x7fc00000u);
}

// 32 bytes to global memory, by one instruction where they are a sector: a thread's row is not its neighbours', so that every
// store instruction of a warp takes 32 turns.
__device__ __forceinline__ void store32(void* to, const uint32_t (&x)[8]) {
  if (reinterpret_cast<uintptr_t>(to) & 31) {
    static_cast<uint4*>(to)[0] = make_uint4(x[0], x[1], x[2], x[3]);
    static_cast<uint4*>(to)[1] = make_uint4(x[4], x[5], x[6], x[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
               "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

// The NaN values that a row sees at positions [from, to), where they were taken out, to 16 columns of its O.
__device__ __forceinline__ void add_poison(const Params& P, int b, int kh, int from, int to, int limit, int c0,
                                           float (&o)[16]) {
  const int end = min(to, limit + 1);
#pragma unroll 1
  for (int p = from; p < end; ++p) {
    const int j = p / P.page, pg = P.a.block_table[(long long)b * P.max_pages + j];
    if (pg < 0 || pg >= P.n_pages) continue;
    const unsigned char* v = static_cast<const unsigned char*>(P.a.v_pages) +
                             (((long long)pg * P.Hkv + kh) * P.page + (p - j * P.page)) * WI_D + c0;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((v[i] & 0x7f) == 0x7f) o[i] = __uint_as_float(0x7fc00000u);
  }
}

// Rows [from, 128) of a block of values as they came: those behind the request's end (row `seen` of the block) are zeroed, and
// so are NaN elements, which `flag` is told of.  One half of every row by each of two warps, the half that it widens.
__device__ __noinline__ void clean_values(unsigned char* v, int lane, int half, int from, int seen, int* flag, int mark) {
  bool found = false;
  for (int i = max(from, 0) * (WI_D / 32) + lane; i < kRows * (WI_D / 32); i += 32) {
    const int r = i / (WI_D / 32), c = i % (WI_D / 32) + half * (WI_D / 32);
    uint4* const at = reinterpret_cast<uint4*>(v + r * WI_D + ((c ^ (r & 7)) << 4));
    if (r >= seen) {
      *at = make_uint4(0u, 0u, 0u, 0u);
      continue;
    }
    const uint4 x = *at;
    uint32_t e[4] = {x.x, x.y, x.z, x.w}, any = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t nan = ((e[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // of bytes whose other bits are all ones
      any |= nan;
      e[k] &= ~((nan >> 7) * 0xffu);
    }
    if (any) {
      *at = make_uint4(e[0], e[1], e[2], e[3]);
      found = true;
    }
  }
  if (found) *reinterpret_cast<volatile int*>(flag) = mark;
  __syncwarp();
}

struct Rows8 {
  Params P;
  WiPagedScales s;
};

template <bool LONG>
__global__ void __launch_bounds__(kThreads, 1) k_paged_attention8(const __grid_constant__ CUtensorMap map_q,
                                                                 const __grid_constant__ CUtensorMap map_k,
                                                                 const __grid_constant__ CUtensorMap map_v,
                                                                 const __grid_constant__ Rows8 A) {
  const Params& P = A.P;
  extern __shared__ __align__(1024) unsigned char raw[];
  pdl_trigger();  // the next kernel may take the SMs as they fall free; it waits for this grid before it reads
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (smem_addr(raw) & 1023u) {  // the swizzled tiles need 1024-byte alignment; never run misaligned
    if (tid == 0) atomicOr(P.err, WI_DEVERR_BAD_ROW);
    return;
  }
  if (tid == 0) {
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_empty[s], kWideWarps);
    }
    for (int s = 0; s < kWStages; ++s) {
      mbar_init(&sm.w_full[s], kWideWarps);
      mbar_init(&sm.w_empty[s], 1);
    }
    for (int s = 0; s < kScaleSlots; ++s) mbar_init(&sm.scale_full[s], 1);
    mbar_init(&sm.q_raw, 1);
    mbar_init(&sm.q_empty, 1);
    mbar_init(&sm.q_full, kSoftWarps);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.s_full[t], 1);
      for (int h = 0; h < 2; ++h) mbar_init(&sm.p_ready[t][h], kSoftWarps / 2);
      mbar_init(&sm.pv_done[t], 1);
      mbar_init(&sm.o_full[t], 1);
    }
    mbar_init(&sm.drained, 1);
    for (int i = 0; i < 8; ++i) sm.poison[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kSoftWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sm.tmem_base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == kSoftWarps && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_q)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_v)) : "memory");
  }
  pdl_wait();
  tc_fence_before();
  const bool any = find_run<kLead, 2, kThreads>(P, 1, P.tickets ? kLead + kWhole : 0, kSlack, sm.scan, &sm.run);  // (with a barrier of all threads)
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;  // S0, S1 at columns 0, 128; O0, O1 at 256, 384
  if (!any) {  // the whole CTA leaves
    if (tid == 0) P.splits[blockIdx.x].last = -1;
    if (warp == kSoftWarps + 1)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    return;
  }

  // a softmax lane holds a row of scores; the registers that the other warps do not need go to those
  // (208 * 8 + 88 * 4 = 168 * 12, what the launch has)
  if (warp < kSoftWarps)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  if (warp < kSoftWarps) {
    // ---------------- softmax
    const int chain = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + (uint32_t)chain * kRows;
    const int tok = (row * ((65536 + P.G - 1) / P.G)) >> 16, head = row - tok * P.G;
    uint32_t s_par = 0, o_par0 = 0, o_par1 = 0;
    bool ok = true;  // after one timed-out wait the warp waits no more and writes nothing, but meets every barrier
    bool split = false;  // the run's last item goes on in the next CTA
    // Only the cursor and what the blocks need live through a segment, beside the scores; the rest is worked out again
    // behind them, from the request as the warp keeps it in shared memory.
    Cursor cur;
    int nb, step, from, base, limit, whole, n0 = 0;  // n0: blocks of the segments before
    // The queries of segment `seg`, before the end of the one in front of it: its first scores are worked out meanwhile.
    auto queries = [&](const Walk<LONG>& w, int seg) {
      if (ok) ok = mbar_wait(&sm.q_raw, seg & 1, P.err);
      if (!w.single || chain == 0) {
        const int ti = w.tile * w.tp + chain * P.tq + tok;
        sm.q_scale[chain][row] = cut_query(sm.q[chain][0], tok < P.tq && ti < w.r.n, row);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full);
    };
    bool more;
    {
      Walk<LONG> w(P, sm.run.start, sm.run.req);
      more = w.next(P);
      cur = w;
      if (lane == 0) sm.reqs[0][warp] = w.r;
      __syncwarp();
      if (more) queries(w, 0);
    }
    for (int seg = 0; more; ++seg) {
      float q_scale;
      {
        Walk<LONG> w(P, cur, sm.reqs[seg & 1][warp]);
        w.next(P);
        const int own_tile = w.single ? 0 : chain, ti = w.tile * w.tp + own_tile * P.tq + tok;
        limit = tok < P.tq && ti < w.r.n ? (int)(w.p0 + ti) : -1;    // the last position that the row sees
        whole = (int)(w.p0 + w.tile * w.tp + own_tile * P.tq);       // ... that all rows of the tile see
        nb = w.nb;
        step = w.single ? 2 : 1;
        from = w.single ? chain : 0;
        base = w.b0 * kRows;
        if (w.single) soft_barrier();  // both chains have the one tile
        q_scale = sm.q_scale[own_tile][row];
      }
      float m = -INFINITY, l = 0.f;  // the row's reference and its sum
      for (int j = from; j < nb; j += step) {
        const int slot = (n0 + j) % kScaleSlots;
        if (ok) ok = mbar_wait(&sm.scale_full[slot], ((n0 + j) / kScaleSlots) & 1, P.err);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const uint32_t tsh = ts + (uint32_t)half * kHalf;
          Scales x8, y8;
          x8.load(sm.scale[slot], 4 * half);
          if (ok && half == 0) ok = mbar_wait(&sm.s_full[chain], s_par, P.err);
          tc_fence_after();
          // P takes the place of the scores, which stay in registers, so that the half can be done again.
          uint32_t a[2][32];
          tmem_ld32_nowait(tsh, a[0]);
          tmem_ld32_nowait(tsh + 32, a[1]);
          tmem_wait_ld();
          const int k0 = base + j * kRows + half * kHalf;
          const bool masked = k0 + kHalf - 1 > whole;
          const int seen = limit - k0;  // the row sees columns 0 .. seen of this half
          // Weights of the two quarters; whether the row's reference is too small for them.  A row without a reference (every
          // score so far minus infinity) looks for one in each half that it sees something of: against 0 its weights might
          // all vanish.  A row that sees nothing of the half, or that no token owns, asks for nothing.
          float zl;
          auto all_weights = [&]() -> bool {
            const float ref = m == -INFINITY ? 0.f : m;  // nothing seen so far: every weight is 2^-inf = 0
            const uint64_t ref2 = pair(-ref, -ref);
            float z = zl = 0.f;
            y8.load(sm.scale[slot], 4 * half + 2);
            weights(a[0], tsh, x8, q_scale, ref2, z, zl);
            weights(a[1], tsh + 16, y8, q_scale, ref2, z, zl);
            return seen >= 0 && (!(z <= kAgain) || !(zl <= kFarMost) || m == -INFINITY);
          };
          // Most halves are seen whole by every row and fit their references: their code stands on its own, without a jump
          // (with the rest in the same loop, jumped over, a block took 1740 cycles here, 290 of them before its first weight).
          const bool first = j == from && half == 0;
          bool grown = first, again = first;
          if (__builtin_expect(!(masked || first), 1)) {
            grown = all_weights();
            again = __any_sync(0xffffffffu, grown);
            if (!again) l += zl;
          }
          if (__builtin_expect(masked || again, 0)) {
            if (masked) mask_scores(a, seen);
            for (;;) {
              if (again) {  // the first half, or the reference is far too small; grown: of this row (other rows keep theirs)
                tmem_wait_st();
                const float top = grown ? fmaxf(m, top_of(a, sm.scale[slot], 4 * half, q_scale)) : m;
                if (!first) {
                  // once the chain's products so far are done (those of earlier blocks are: these scores came behind them)
                  if (ok && half == 1) ok = mbar_wait(&sm.pv_done[chain], s_par, P.err);
                  tc_fence_after();
                  const float f = m == top ? 1.f : ex2(m - top);
                  l *= f;
                  const uint32_t to = tmem + lanes + 256u + (uint32_t)chain * WI_D;
#pragma unroll 1
                  for (int c = 0; c < 8; ++c) {
                    uint32_t o[16];
                    tmem_ld16_nowait(to + 16 * c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                    tmem_st16_nowait(to + 16 * c, o);
                  }
                }
                m = top;
              }
              x8.load(sm.scale[slot], 4 * half);
              grown = all_weights();
              if (again || !__any_sync(0xffffffffu, grown)) {
                l += zl;
                break;
              }
              again = true;
            }
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_ready[chain][half]);
        }
        s_par ^= 1;
      }

      // ---- the segment's end: maximum and sum over both chains where they had one tile, then O
      Walk<LONG> w(P, cur, sm.reqs[seg & 1][warp]);
      w.next(P);
      {
        Walk<LONG> next = w;
        next.advance();
        more = next.next(P);
        cur = next;
        if (lane == 0) sm.reqs[seg + 1 & 1][warp] = next.r;
        __syncwarp();
        if (w.single) soft_barrier();  // both chains have read their factors of the tile's queries
        if (more) queries(next, seg + 1);
      }
      const int own_tile = w.single ? 0 : chain, ti = w.tile * w.tp + own_tile * P.tq + tok;
      const bool live = tok < P.tq && ti < w.r.n;
      const bool both = !w.single || w.nb > 1;  // chain 1 had blocks
      bool part = w.b0 > 0 || w.nb < w.nblk, begun = w.b0 == 0, goes_on = false, join = w.single && both;
      if (ok && (w.single || chain == 0)) ok = mbar_wait(&sm.o_full[0], o_par0, P.err);
      if (ok && both && (w.single || chain == 1)) ok = mbar_wait(&sm.o_full[1], o_par1, P.err);
      o_par0 ^= 1;
      if (both) o_par1 ^= 1;
      tc_fence_after();
      float f0 = 1.f, f1 = 0.f;
      if (w.single) {
        sm.xch[chain][0][row] = m;
        sm.xch[chain][1][row] = l;
        soft_barrier();
        const float m0 = sm.xch[0][0][row], m1 = sm.xch[1][0][row];
        m = fmaxf(m0, m1);
        const float ref = m == -INFINITY ? 0.f : m;
        f0 = ex2(m0 - ref);
        f1 = ex2(m1 - ref);
        l = sm.xch[0][1][row] * f0 + sm.xch[1][1][row] * f1;
      }
      const long long at = (long long)(w.r.s0 + ti) * P.Hq + w.kh * P.G + head;
      const uint32_t to = tmem + lanes + 256u + (w.single ? 0u : (uint32_t)chain * WI_D);
      const int ca = w.single ? 64 * chain : 0, cb = w.single ? ca + 64 : WI_D;  // the columns that this thread takes
      if (LONG && w.nblk > kLongest) {  // maybe not the CTA's first segment of the item, or not its last
        const int spent = sm.run.start.left - w.left;
        begun = spent >= w.at - kLead;
        part = !begun || w.b0 + w.nb < w.nblk;
        goes_on = w.b0 + w.nb < w.nblk && w.took < w.left;
        if (w.at > 0 && spent > 0) {
          const float2 x = add_earlier(P, P.parts.slot(2 * (int)blockIdx.x + begun), own_tile, row, live, m, l, to, ca, cb,
                                       join, f0, f1);
          m = x.x;
          l = x.y;
          join = false;
          if (w.single) soft_barrier();  // both threads of a row have read its maximum and sum
        }
      }
      const int slot = 2 * (int)blockIdx.x + (begun ? 1 : 0);
      float* dst = P.parts.slot(slot);
      const bool poison = *reinterpret_cast<volatile int*>(&sm.poison[seg & 7]) == seg + 1;
      const float inv = part ? 1.f : (l == 0.f ? 0.f : 1.f / l);
#pragma unroll 1
      for (int c = ca; c < cb; c += 16) {
        __syncwarp();
        uint32_t raw_o[16];
        tmem_ld16_nowait(to + c, raw_o);
        tmem_wait_ld();
        float o[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __uint_as_float(raw_o[i]);
        if (join) {
          tmem_ld16_nowait(to + WI_D + c, raw_o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = o[i] * f0 + __uint_as_float(raw_o[i]) * f1;
        }
        if (poison && live)
          add_poison(P, w.b, w.kh, max(max(w.b0, w.first_fix()) * kRows, w.first_clean()),
                     min((w.b0 + w.nb) * kRows, w.r.kv), limit, c, o);
        if (ok && live) {
          if (part) {
#pragma unroll
            for (int i = 0; i < 16; ++i) __stcg(dst + P.parts.o(own_tile, c + i, row), o[i]);
          } else {
            uint32_t x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = pack_bf16(o[2 * i] * inv, o[2 * i + 1] * inv);
            store32(static_cast<bf16*>(P.a.out) + at * WI_D + c, x);
          }
        }
      }
      if (ok && live && (chain == 0 || !w.single)) {
        if (part) {
          __stcg(dst + P.parts.m(own_tile, row), m);
          __stcg(dst + P.parts.l(own_tile, row), l);
        } else if (P.a.lse) {
          P.a.lse[at] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
        }
      }
      tc_fence_before();  // O is read: the next segment may write it
      if (LONG && goes_on) {
        // the rest of the item's end is for the last segment that the CTA has of it
      } else if (part && P.tickets) {
        const long long item = sm.run.end - w.left - w.at + kLead;  // the unit of the item's first block
        const int c0 = cta_of(item, sm.run.total, sm.run.ctas), c1 = cta_of(item + w.nblk - 1, sm.run.total, sm.run.ctas);
        soft_barrier();  // then thread 0's release covers what all of them stored
        if (tid == 0) {
          sm.last = 0;
          if (ok && ticket_acq_rel(P.tickets + c0) == (unsigned)(c1 - c0)) {
            P.tickets[c0] = 0;
            sm.last = 1;
          }
        }
        soft_barrier();
        if (sm.last) {
          const Split sp = {w.r.s0 + w.tile * w.tp, w.kh, w.cnt, c1};
          if (P.parts.rows > kFewRows) {
            merge_tile<kSoftWarps>(P, sp, c0);
          } else {
#pragma unroll 1
            for (int r0 = 0; r0 < tile_rows(P, sp, 0); r0 += 2 * kSoftWarps * 32 / WI_D)
              merge_some<kSoftWarps * 32>(P, sp, c0, 0, r0);
          }
        }
      } else if (part && begun && tid == 0) {
        split = true;
        P.splits[blockIdx.x] = {w.r.s0 + w.tile * w.tp, w.kh, w.cnt,
                                cta_of(sm.run.end - w.left - w.at + kLead + w.nblk - 1, sm.run.total, sm.run.ctas)};
      }
      if (w.single) soft_barrier();  // both chains' O, maxima and sums have been read
      n0 += w.nb;
    }
    if (tid == 0 && !split) P.splits[blockIdx.x].last = -1;
  } else if (warp == kSoftWarps) {
    // ---------------- TMA: keys, values, and the scales of their groups
    Walk<LONG> w(P, sm.run.start, sm.run.req);
    const uint32_t on = elect_one();
    const int per = P.box / kGroup;  // groups of a box
    constexpr int kBatch = 32 / kGroups;
    const uint32_t q_half = (uint32_t)(P.tq * P.G) * 128u;
    int nk = 0, nv = 0, nq = 0;  // blocks of keys and of values, and queries that were asked for
    bool ok = true;
    for (; ok && w.next(P); w.advance()) {
      // The pages and scales of four blocks at a time, a lane to a group: pages are looked up two batches ahead and scales
      // one, so that no block waits for a look-up.
      constexpr int kNone = -0x7fffffff - 1;  // behind the request's end
      auto page_of = [&](int batch) -> int {
        const int j = batch * kBatch + lane / kGroups, p = (w.b0 + j) * kRows + lane % kGroups * kGroup;
        if (j >= w.nb || p >= w.r.kv) return kNone;
        return P.a.block_table[(long long)w.b * P.max_pages + p / P.page];
      };
      // a group's row of the pool, from its page; a bad page is page 0
      auto row_of = [&](int pg, int batch) -> int {
        if (pg == kNone) return -1;
        if (pg < 0 || pg >= P.n_pages) {
          atomicOr(P.err, WI_DEVERR_BAD_PAGE);
          pg = 0;
        }
        return (pg * P.Hkv + w.kh) * P.page + ((w.b0 + batch * kBatch) * kRows + lane * kGroup) % P.page;
      };
      auto scales_of = [&](int row) -> uint32_t {
        return row < 0 ? kScaleBias * 0x101u : (uint32_t)A.s.k[row / kGroup] | (uint32_t)A.s.v[row / kGroup] << 8;
      };
      auto fill = [&](const CUtensorMap* map, unsigned char* to, uint64_t* full, uint64_t* empty, int stages, int n, int row,
                      int j) -> bool {
        bool got = true;
        if (n >= stages) got = mbar_wait(empty, ((uint32_t)(n / stages) & 1u) ^ 1u, P.err);
        if (!__all_sync(0xffffffffu, got)) return false;
        const int first = j % kBatch * kGroups;  // the lane of the block's first group
        // boxes behind the request's end are left out: always the last ones
        const int groups = __popc(__ballot_sync(0xffffffffu, row >= 0) >> first & ((1u << kGroups) - 1));
        const int boxes = (groups + per - 1) / per;
        if (on) mbar_arrive_expect_tx(full, (uint32_t)(boxes * P.box) * WI_D);
        __syncwarp();
        const uint32_t dst = smem_addr(to);
        for (int i = 0; i < boxes; ++i)
          tma_load_2d_warp(on, dst + (uint32_t)(i * P.box) * WI_D, map, 0, __shfl_sync(0xffffffffu, row, first + i * per), full);
        return true;
      };
      // queries, once the scores of the segment before have read theirs
      if (nq > 0) ok = mbar_wait(&sm.q_empty, (uint32_t)(nq - 1) & 1u, P.err);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        const int n = w.single ? 1 : 2;
        mbar_arrive_expect_tx(&sm.q_raw, 2u * q_half * n);
        for (int t = 0; t < n; ++t) {
          const int tk = w.r.s0 + w.tile * w.tp + t * P.tq;
          tma_load_3d(sm.q[t][0], &map_q, 0, w.kh * P.G, tk, &sm.q_raw);
          tma_load_3d(sm.q[t][1], &map_q, 64, w.kh * P.G, tk, &sm.q_raw);
        }
      }
      ++nq;
      const int ahead = w.single ? 2 : 1;
      // the batch that keys are asked for from (rows and scales), and the one that values are, which may lie behind it
      int page, row = 0, row_next, row_v = 0;
      uint32_t e = 0, e_next;
      {
        const int g0 = page_of(0);
        page = page_of(1);
        row_next = row_of(g0, 0);
        e_next = scales_of(row_next);
      }
      auto keys = [&](int j) -> bool {
        if (j % kBatch == 0) {
          row_v = row;
          row = row_next;
          e = e_next;
          row_next = row_of(page, j / kBatch + 1);
          e_next = scales_of(row_next);
          page = page_of(j / kBatch + 2);
        }
        const int st = nk % kKStages, slot = nk % kScaleSlots;
        if (!fill(&map_k, sm.k[st], &sm.k_full[st], &sm.k_empty[st], kKStages, nk, row, j)) return false;
        if (lane / kGroups == j % kBatch) {
          const int ev = scale_exponent((unsigned char)(e >> 8));
          sm.scale[slot].k[lane % kGroups] = pow2(scale_exponent((unsigned char)(e & 0xff)));
          sm.scale[slot].e[lane % kGroups] = make_float2((float)ev, (float)ev);
          sm.scale[slot].back[lane % kGroups] = pow2(-ev);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.scale_full[slot]);
        ++nk;
        return true;
      };
      ok = keys(0);
      if (ok && ahead == 2 && w.nb > 1) ok = keys(1);
      for (int j = 0; ok && j < w.nb; ++j) {
        const int st = nv % kVStages, kj = min(j + ahead - 1, w.nb - 1);  // the last block whose keys were asked for
        ok = fill(&map_v, sm.v[st], &sm.v_full[st], &sm.v_empty[st], kVStages, nv, j / kBatch == kj / kBatch ? row : row_v, j);
        if (!ok) break;
        ++nv;
        if (j + ahead < w.nb) ok = keys(j + ahead);
      }
    }
    // no copy is in flight when the CTA's shared memory goes (after a timed-out wait nobody may have waited for them)
    if (nq > 0) mbar_wait(&sm.q_raw, (uint32_t)(nq - 1) & 1u, P.err);
    for (int s = 0; s < kKStages && s < nk; ++s) mbar_wait(&sm.k_full[s], (uint32_t)((nk - 1 - s) / kKStages) & 1u, P.err);
    for (int s = 0; s < kVStages && s < nv; ++s) mbar_wait(&sm.v_full[s], (uint32_t)((nv - 1 - s) / kVStages) & 1u, P.err);
  } else if (warp == kSoftWarps + 1) {
    // ---------------- tensor cores: one lane issues, the whole warp computes what it issues
    Walk<LONG> w(P, sm.run.start, sm.run.req);
    const uint32_t on = elect_one();
    constexpr uint32_t idesc_s = make_idesc_e4m3(kRows, kRows);
    constexpr uint32_t idesc_o = make_idesc_f16(kRows, WI_D) | kIdescNMajorB;
    int nk = 0, nw = 0;  // blocks of keys and of values done with
    uint32_t p_par = 0;
    bool ok = true;
    auto all_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, P.err));
    };
    auto take_keys = [&]() -> bool {
      if (!all_wait(&sm.k_full[nk % kKStages], (uint32_t)(nk / kKStages) & 1u)) return false;
      tc_fence_after();
      return true;
    };
    // chain t's scores of a block, of the queries of tile q.  (In two products of 64 keys, the second behind the first half's
    // weights, a block takes 3600 cycles: a product of 64 columns costs what one of 128 does.)
    auto scores = [&](int t, int q) {
      const uint32_t d = __shfl_sync(0xffffffffu, tmem + (uint32_t)t * kRows, 0);
      const uint32_t a0 = __shfl_sync(0xffffffffu, desc_lo_kmajor(smem_addr(sm.q[q][0])), 0);
      const uint32_t b0 = __shfl_sync(0xffffffffu, desc_lo_kmajor(smem_addr(sm.k[nk % kKStages])), 0);
#pragma unroll
      for (int kk = 0; kk < 2 * WI_D / 32; ++kk)  // the first pieces, then the rest
        mma_e4m3_warp(on, d, a0 + (kk >> 2) * (kBlockBytes / 16) + (kk & 3) * 2, desc_hi_sw128(1024), b0 + (kk & 3) * 2,
                      desc_hi_sw128(1024), idesc_s, kk > 0);
      mma_commit_warp(on, &sm.s_full[t]);
    };
    auto keys_done = [&] { mma_commit_warp(on, &sm.k_empty[nk % kKStages]); ++nk; };
    // ... and the product of half of its weights, once they are there
    auto values = [&](int t, int half, bool add) -> bool {
      const uint32_t p = __shfl_sync(0xffffffffu, tmem + (uint32_t)t * kRows + (uint32_t)half * kHalf, 0);
      const uint32_t b0 = __shfl_sync(
          0xffffffffu, desc_lo_nmajor(smem_addr(sm.w[nw % kWStages]) + (uint32_t)half * kHalf * WI_D * 2, 1024), 0);
      const uint32_t more = __shfl_sync(0xffffffffu, (uint32_t)add, 0);
      const uint32_t d = __shfl_sync(0xffffffffu, tmem + 256u + (uint32_t)t * WI_D, 0);
      const uint32_t bit = (uint32_t)(t * 2 + half);
      if (!all_wait(&sm.p_ready[t][half], (p_par >> bit) & 1u)) return false;
      p_par ^= 1u << bit;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < kHalf / 16; ++kk)
        mma_bf16_ta_warp(on, d, p + (uint32_t)kk * 8, b0 + (uint32_t)kk * (4096 / 16), desc_hi_sw128(2048), idesc_o,
                         kk > 0 ? 1u : more);
      if (half == 0) mma_commit_warp(on, &sm.pv_done[t]);
      return true;
    };
    for (int seg = 0; ok && w.next(P); ++seg, w.advance()) {
      if (!(ok = all_wait(&sm.q_full, seg & 1))) break;
      tc_fence_after();
      if (!(ok = take_keys())) break;
      const int ahead = w.single ? 2 : 1;
      scores(0, 0);
      if (!w.single) scores(1, 1);
      keys_done();
      if (w.single && w.nb > 1) {
        if (!(ok = take_keys())) break;
        scores(1, 0);
        keys_done();
      }
      if (w.nb <= ahead) mma_commit_warp(on, &sm.q_empty);
      for (int j = 0; ok && j < w.nb; ++j) {
        if (!(ok = all_wait(&sm.w_full[nw % kWStages], (uint32_t)(nw / kWStages) & 1u))) break;
        const bool more = j + ahead < w.nb;
        const int t0 = w.single ? j & 1 : 0, t1 = w.single ? t0 : 1;  // the chains that have the block
#pragma unroll 1
        for (int t = t0; t <= t1; ++t) {
          if (!(ok = values(t, 0, j >= ahead) && values(t, 1, true))) break;
          if (t == t1) mma_commit_warp(on, &sm.w_empty[nw % kWStages]);
          if (!more) {
            mma_commit_warp(on, &sm.o_full[t]);
            continue;
          }
          if (t == t0 && !(ok = take_keys())) break;
          scores(t, w.single ? 0 : t);
          if (t == t1) {
            keys_done();
            if (j + ahead + 1 >= w.nb) mma_commit_warp(on, &sm.q_empty);
          }
        }
        ++nw;
      }
    }
    // every product is done before the tensor memory goes
    mma_commit_warp(on, &sm.drained);
    mbar_wait(&sm.drained, 0, P.err);
  } else {
    // ---------------- values to f16; in blocks that not every row sees whole, what lies behind the request's end is
    // zeroed, and so are NaN elements (0 * NaN is NaN inside the product), which the end of the item adds to the rows that
    // see them
    Walk<LONG> w(P, sm.run.start, sm.run.req);
    const int half = warp - kSoftWarps - 2;
    const int r8 = lane & 7, c = (lane >> 3) + 4 * half, piece = (c & 3) * 2;  // a lane's row of a group, and piece of the row
    int n = 0;
    bool ok = true;
    for (int seg = 0; ok && w.next(P); ++seg, w.advance()) {
      const int fix = w.first_fix() - w.b0;
      for (int j = 0; j < w.nb; ++j, ++n) {
        const int st = n % kVStages, to = n % kWStages;
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sm.v_full[st], (uint32_t)(n / kVStages) & 1u, P.err)))) break;
        if (n >= kWStages &&
            !(ok = __all_sync(0xffffffffu, mbar_wait(&sm.w_empty[to], ((uint32_t)(n / kWStages) & 1u) ^ 1u, P.err))))
          break;
        if (j >= fix) clean_values(sm.v[st], lane, half, w.first_clean() - (w.b0 + j) * kRows, w.r.kv - (w.b0 + j) * kRows,
                                   &sm.poison[seg & 7], seg + 1);
        const unsigned char* const v = sm.v[st] + r8 * WI_D + ((c ^ r8) << 4);
        unsigned char* const o = sm.w[to] + (c >> 2) * 1024 + r8 * 128;
        // a warp takes one half of a row's pieces, four groups of rows at a time: all their loads in front of the first store
#pragma unroll 1
        for (int g0 = 0; g0 < kRows / 8; g0 += 4) {
          uint4 x[4];
#pragma unroll
          for (int g = 0; g < 4; ++g) x[g] = *reinterpret_cast<const uint4*>(v + (g0 + g) * 1024);
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            // columns 16 c .. 16 c + 15: two pieces of the half's eight
            unsigned char* const d = o + (g0 + g) * 2048;
            *reinterpret_cast<uint4*>(d + ((piece ^ r8) << 4)) = e4m3x8_to_f16x8(x[g].x, x[g].y);
            *reinterpret_cast<uint4*>(d + (((piece + 1) ^ r8) << 4)) = e4m3x8_to_f16x8(x[g].z, x[g].w);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.w_full[to]);
          mbar_arrive(&sm.v_empty[st]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps + 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

}  // namespace

cudaError_t wi_launch_paged_attention8(const WiPagedGeom& g, const WiPagedAttn& a, const WiPagedScales& s, int sms,
                                       void* scratch, int* err, cudaStream_t st) {
  if (wi_paged_few(g, a)) return wi_launch_paged_few(g, a, s, sms, scratch, err, st);
  Rows8 A;
  Params& P = A.P;
  A.s = s;
  P.a = a;
  P.Hq = g.Hq;
  P.Hkv = g.Hkv;
  P.G = g.G;
  P.tq = kRows / g.G;
  P.page = g.page;
  P.n_pages = g.n_pages;
  P.max_pages = g.max_pages;
  // a box of a block lies inside one page: the largest power of two that divides the page, 128 at most
  P.box = g.page & -g.page;
  if (P.box > kRows) P.box = kRows;
  const long long rows_here = (long long)a.n_tokens * g.G;
  const bool here = rows_here <= kMergeHere;
  P.tickets = here ? static_cast<unsigned*>(scratch) : nullptr;
  P.splits = reinterpret_cast<Split*>(static_cast<char*>(scratch) + kPagedTicketBytes);
  P.parts = {reinterpret_cast<float*>(static_cast<char*>(scratch) + kPagedTicketBytes + kSplitBytes),
             rows_here <= kFewRows ? kFewRows : here ? kMergeHere : kRows, here ? 1 : 2};
  P.err = err;
  CUtensorMap map_q, map_k, map_v;
  const unsigned long long rows = (unsigned long long)g.n_pages * g.Hkv * g.page;
  if (!wi_encode_heads_sw128(&map_q, a.q, (unsigned long long)a.n_tokens, (unsigned)g.Hq, (unsigned)g.G,
                             (unsigned)P.tq) ||
      !wi_encode_bytes_sw128(&map_k, a.k_pages, rows, (unsigned)P.box) ||
      !wi_encode_bytes_sw128(&map_v, a.v_pages, rows, (unsigned)P.box))
    return cudaErrorInvalidValue;
  static int smem_set[2][kWiSmemDevices] = {};
  const bool is_long = (long long)g.max_pages * g.page > (long long)kLongest * kRows;
  auto* kernel = is_long ? k_paged_attention8<true> : k_paged_attention8<false>;
  cudaError_t e = wi_ensure_smem(kernel, sizeof(Smem), smem_set[is_long]);
  if (e != cudaSuccess) return e;
  const int grid = sms < kPagedMaxSms ? sms : kPagedMaxSms;
  if ((e = wi_launch_chained(kernel, dim3((unsigned)grid), kThreads, sizeof(Smem), st, map_q, map_k, map_v, A)) != cudaSuccess)
    return e;
  if (here) return cudaSuccess;
  return wi_launch_chained(k_paged_merge, dim3((unsigned)grid, 2 * kRows / kMergeRows), kMergeThreads, 0, st, P);
}
