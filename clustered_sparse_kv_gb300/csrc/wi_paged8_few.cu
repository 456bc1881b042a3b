// wi_paged8_few.cu -- attention over the paged cache in 8 bits where a tile has few rows: single tokens above all.
//
// The products are turned, so that the 128 rows of a tensor-core tile are the
// block's 128 positions, and then a head's 128 elements, with the few queries
// as columns:
//   S^T [position][row] = K Q^T       A = K as it lies in the cache, B = Q
//   O^T [element][row] += V^T P^T     A = V as it lies (M-major), B = P
// both in e4m3, which keys and values are held in.  Queries and weights are
// not, and are sums of e4m3 pieces.  A bf16 query is a first piece of four
// significant bits and a rest of four, exactly (over the row's largest element;
// what is below 2^-17 of that may be lost), so Q has two columns per row and S
// is added up.  A weight has six pieces of four bits with a column, and so a sum
// in tensor memory, each: columns cost next to nothing here, and each piece has
// its own power of two, so that together they hold a weight to 2^-33 of the
// largest, or to fp32 (a sink of attention may weigh many million times more
// than what is left of the row).
//
// A thread of the four softmax warps has one position: its group's two scales,
// its score of every row, and its weights' pieces, which it stores as two or
// three 16-byte pieces of B.  The value's scale 2^e goes into the weight,
// p' = 2^(score + e - m), and out of the sum, l += p' 2^-e; m is a row's
// reference, near the largest score + e so far.  It moves only when a weight
// would pass 448 (every thread asks, by one barrier a block): then O is
// rescaled and the block done with the new one.
//
// One warp brings the blocks by TMA into rings of three keys' and three values'
// blocks, with the groups' scales beside the values; one issues the products.
// Two CTAs share an SM, so that one's start and end lie behind the other's
// reads.  Runs of units, and parts that the last CTA of an item adds up, as in
// the bf16 attention.
//
// What bounds it, 32 query and 8 kv heads on one GB300: HBM.  One token over 131K
// positions in 55 us: 6 until the first scores (lengths, tables, first copies), 38
// for 268 MB (7.1 TB/s), then the slowest CTA, and 5 for the parts; 64 single tokens
// over 100 - 8000 positions 70 us, of which 50 are the reads.  A block of 128
// positions costs a CTA 700 cycles of weights (1000 with eight rows; with four pieces
// 600 and 880, and 54 and 69 us), and HBM gives two CTAs one every 1400.  With one CTA to an SM 91 and 122 us (its stages do not matter); with pages
// and scales looked up a block ahead, not four, 68 and 81; with three CTAs of two
// stages 56 and 69; with a block's values asked for before the scales of the block in
// front are stored, the short cases 0.6 us more.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>

#include "wi_common.cuh"
#include "wi_e4m3.cuh"
#include "wi_internal.h"
#include "wi_paged.h"
#include "wi_paged8.h"
#include "wi_paged_walk.cuh"
#include "wi_pipe.cuh"
#include "wi_tc.cuh"

namespace {

constexpr int kStages = 3;
constexpr int kBlockBytes = kRows * WI_D;  // of keys or of values
constexpr int kSoftWarps = 4;
constexpr int kSoftThreads = 32 * kSoftWarps;
constexpr int kThreads = kSoftThreads + 64;
constexpr int kLead = 2;    // units in front of an item's blocks, for what its start and end cost
// Units of a run, at least, and the blocks up to which one request's items are not cut: joining parts costs 3 us, a block 0.7
// (one token over 300 positions 8.9 us whole, 11.6 cut; over 1000 13.6 whole, and cut 11.9, 12.3, 13.3 with runs of 1, 2, 4 at
// least; over 8000 14.9, 14.5, 15.5).
constexpr int kLeast = 2, kWhole = 4;
// What the largest item may have above an equal run, where each item is a run (30 single tokens over 300 - 700 positions 14.6 us
// whole, 21.1 cut; ten over 300 - 900 13.8 cut, 13.4 with eight, but sixteen over 2000 25.0 with sixteen, 23.6 cut).
constexpr int kSlack = 4;
// Blocks after which the tensor cores' sums are added up in fp32: their additions cut bits off.  Sums of numbers of one sign
// come out too small by 1.4e-5 of themselves (by 1e-4 with 1024); reading them costs less than a block.
constexpr int kFlush = 256;
constexpr int kPieces = 6;
constexpr float kScaleLog2 = 0.08838834764831845f * 1.4426950408889634f;  // log2(e) / sqrt(128)
constexpr float kLn2 = 0.6931471805599453f;
// A new reference makes the row's largest weight 2^3 (for values' scales of 2^-64 or more); it is taken where one passes
// 2^8.5, or where a score is so far above it (through values of a tiny scale) that the sum might leave fp32.
constexpr float kTop = 3.f, kMost = 8.5f, kFar = 64.f + kTop, kFarMost = 80.f;

// A piece takes four bits, so that what it leaves, times kStep, is a piece again; the last one is known to 2^-10, 2^-30 of
// a weight's own units.
constexpr float kStep = 16.f;
__device__ __forceinline__ constexpr float size_of(int piece) { return piece == 0 ? 1.f : size_of(piece - 1) / kStep; }

// RP: rows of a tile.
template <int RP>
struct Smem {
  static constexpr int kQCols = 16;            // two columns per row, sixteen at least
  static constexpr int kPCols = (kPieces * RP + 15) / 16 * 16;
  static constexpr int kRings = 2 * kStages * kBlockBytes / (RP * WI_D * 4);  // parts that fit the rings at a time
  static constexpr int kJoin = (kRings + 31) / 32 * 32;
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  // Of two buffers each, block n's in n & 1: who waits for block n's has seen that of block n - 2 (S of a block is issued
  // behind O of the one two before it), so that a phase's parity says which it is.
  uint64_t q_full, s_full[2], p_ready[2], o_done[2], drained;
  uint32_t tmem_base;
  int last;                     // this CTA merges the item that it just added to
  int poison;                   // number + 1 of the last segment with a NaN value that not every row sees
  int mask[kSoftWarps];         // rows that take a new reference
  long long scan[2 * (kThreads / 32)];
  Run run;
  alignas(8) unsigned char next[kSoftWarps][sizeof(WalkOver<kLead, 1, 0>)];  // a softmax warp's segment behind this one
  float q_scale[RP];
  float xch[kSoftWarps][RP];
  float sum[kSoftWarps][RP];
  float scale[kStages][2][kRows / kGroup];  // 2^e of the keys' groups; e of the values'
  alignas(16) float factor[kJoin][RP];  // of the parts that are added up
  float joined[3][RP];
  alignas(1024) unsigned char q[kQCols * WI_D];      // K-major, 128-byte swizzle
  unsigned char p[2][kPCols * kRows];                // [16 columns][position][16 B]
  alignas(1024) unsigned char k[kStages][kBlockBytes];
  unsigned char v[kStages][kBlockBytes];
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void soft_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftThreads) : "memory"); }
// Whether any of the softmax threads says so.
__device__ __forceinline__ bool soft_any(bool x) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)x), "n"(kSoftThreads)
      : "memory");
  return any != 0;
}

// One pass over the pieces of RP weights: word w of piece i holds rows 4w .. 4w + 3.
template <int RP>
__device__ __forceinline__ void split(float (&x)[RP], uint32_t (&out)[kPieces][RP / 4]) {
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
#pragma unroll
    for (int w = 0; w < RP / 4; ++w) {
      float* y = x + 4 * w;
      const uint32_t a = e4m3x2_of(y[0], y[1]), b = e4m3x2_of(y[2], y[3]);
      out[i][w] = a | b << 16;
      if (i + 1 < kPieces) {
        const float2 fa = e4m3x2_to_f32x2(a), fb = e4m3x2_to_f32x2(b);
        y[0] = (y[0] - fa.x) * kStep;
        y[1] = (y[1] - fa.y) * kStep;
        y[2] = (y[2] - fb.x) * kStep;
        y[3] = (y[3] - fb.y) * kStep;
      }
    }
  }
}

// The pieces' sums of this thread's element, the smallest first, to acc.
template <int RP>
__device__ __forceinline__ void add_pieces(uint32_t from, float (&acc)[RP]) {
  float size = size_of(kPieces - 1);
#pragma unroll 1
  for (int i = kPieces - 1; i >= 0; --i, size *= kStep) {
    uint32_t a[RP];
#pragma unroll
    for (int q = 0; q < RP; q += 4) tmem_ld4_nowait(from + i * RP + q, reinterpret_cast<uint32_t(&)[4]>(a[q]));
    tmem_wait_ld();
#pragma unroll
    for (int r = 0; r < RP; ++r) acc[r] += __uint_as_float(a[r]) * size;
  }
}

struct Few {
  Params P;
  WiPagedScales s;
};

// A segment's queries, rows warp, warp + 4 of the tile, four elements to a lane.
template <int RP>
struct Queries {
  uint2 x[RP / kSoftWarps];
  template <typename W>
  __device__ __forceinline__ void ask(const Params& P, const W& w) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int k = 0; k < RP / kSoftWarps; ++k) {
      const int r = warp + k * kSoftWarps, tok = r / P.G, ti = w.tile * w.tp + tok;
      x[k] = make_uint2(0u, 0u);
      if (tok < P.tq && ti < w.r.n)
        x[k] = ldg_u2(static_cast<const bf16*>(P.a.q) +
                      ((long long)(w.r.s0 + ti) * P.Hq + w.kh * P.G + r - tok * P.G) * WI_D + 4 * lane);
    }
  }
  // ... to shared memory as e4m3 pieces, two rows each.  A row of infinities or NaN gets a scale that is no number, and so
  // do all its scores.
  __device__ __forceinline__ void put(Smem<RP>& sm) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int k = 0; k < RP / kSoftWarps; ++k) {
      const int r = warp + k * kSoftWarps;
      float v[4];
      unpack_bf16x4(x[k], v);
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) top = max(top, __float_as_uint(v[c]) & 0x7fffffffu);
      top = __reduce_max_sync(0xffffffffu, top);
      // the row's largest element lies in [128, 256): e is its exponent less 7, within what 2^-e can be
      const int e = min(max((int)(top >> 23) - 127 - 7, -126), 126);
      const float f = pow2(-e);
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = top < 0x7f800000u ? v[c] * f : 0.f;
      const uint32_t a = e4m3x2_of(v[0], v[1]), b = e4m3x2_of(v[2], v[3]);
      const float2 fa = e4m3x2_to_f32x2(a), fb = e4m3x2_to_f32x2(b);
      const uint32_t rest = e4m3x4_of(v[0] - fa.x, v[1] - fa.y, v[2] - fb.x, v[3] - fb.y);
      const uint32_t chunk = lane >> 2, in = (lane & 3) * 4;
      *reinterpret_cast<uint32_t*>(sm.q + r * WI_D + ((chunk ^ (r & 7)) << 4) + in) = a | b << 16;
      *reinterpret_cast<uint32_t*>(sm.q + (RP + r) * WI_D + ((chunk ^ ((RP + r) & 7)) << 4) + in) = rest;
      if (lane == 0) sm.q_scale[r] = top < 0x7f800000u ? pow2(e) * kScaleLog2 : __uint_as_float(0x7fc00000u);
    }
  }
};

// out and lse of an item that was cut between CTAs, added up in CTA order: thread d has column d of every row.  An SM comes
// here once a call, so the code is cold, and what counts is how little of it there is: the parts' columns come to shared
// memory by a short loop of asynchronous copies, `room` parts at a time (38 parts 8.2 us with unrolled loads to registers,
// 2.1 of which went by before the last load was issued; 4 so).
template <int RP>
__device__ __noinline__ void join_parts(const Params& P, Smem<RP>& sm, const Split& sp, int c0, unsigned char* buf, int room) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, parts = sp.last - c0 + 1;
  constexpr int kRecord = RP * WI_D * 4, kVec = RP / 4;  // bytes of a part's columns; pieces of a thread's
  const long long stride = P.parts.slot(2) - P.parts.slot(0);
  const float* const base = P.parts.slot(2 * c0);
  auto part = [&](int i) -> const float* { return base + i * stride + (i == 0 ? stride / 2 : 0); };
  float acc[RP], M[RP / kSoftWarps], L[RP / kSoftWarps];  // M, L: of this warp's rows
#pragma unroll
  for (int r = 0; r < RP; ++r) acc[r] = 0.f;
#pragma unroll
  for (int k = 0; k < RP / kSoftWarps; ++k) {
    M[k] = -INFINITY;
    L[k] = 0.f;
  }
#pragma unroll 1
  for (int i0 = 0; i0 < parts; i0 += room) {
    const int n = min(room, parts - i0);
    const uint32_t to = smem_addr(buf) + tid * 16;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const float* from = part(i0 + i) + (2 + tid) * RP;
#pragma unroll
      for (int q = 0; q < kVec; ++q)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * kRecord + q * (kRecord / kVec)), "l"(from + 4 * q)
                     : "memory");
    }
    if (i0 > 0) soft_barrier();  // the factors before are read
#pragma unroll
    for (int k = 0; k < RP / kSoftWarps; ++k) {  // a warp has a row's factors, a lane one or two parts'
      const int r = warp + k * kSoftWarps;
      constexpr int kEach = Smem<RP>::kJoin / 32;
      static_assert(kEach <= 2, "m and l");
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int h = 0; h < kEach; ++h)
        if (32 * h + lane < n) {
          m[h] = __ldcg(part(i0 + 32 * h + lane) + r);
          l[h] = __ldcg(part(i0 + 32 * h + lane) + RP + r);
        }
      const float top = fmaxf(M[k], warp_max(fmaxf(m[0], m[1]))), ref = top == -INFINITY ? 0.f : top;
      const float back = ex2(M[k] - ref), f0 = ex2(m[0] - ref), f1 = ex2(m[1] - ref);
      L[k] = L[k] * back + warp_sum(f0 * l[0] + f1 * l[1]);
      M[k] = top;
      sm.factor[lane][r] = f0;
      if (kEach > 1) sm.factor[(kEach - 1) * 32 + lane][r] = f1;
      if (lane == 0) {
        sm.joined[0][r] = M[k];
        sm.joined[1][r] = L[k];
        sm.joined[2][r] = back;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // a thread reads what it asked for itself
    soft_barrier();
#pragma unroll
    for (int r = 0; r < RP; ++r) acc[r] *= sm.joined[2][r];
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
#pragma unroll
      for (int q = 0; q < kVec; ++q) {
        const float4 x = *reinterpret_cast<const float4*>(buf + tid * 16 + i * kRecord + q * (kRecord / kVec));
        const float4 f = *reinterpret_cast<const float4*>(&sm.factor[i][4 * q]);
        acc[4 * q] += x.x * f.x;
        acc[4 * q + 1] += x.y * f.y;
        acc[4 * q + 2] += x.z * f.z;
        acc[4 * q + 3] += x.w * f.w;
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RP; ++r) {
    const int tok = r / P.G;
    if (tok >= P.tq || tok >= sp.cnt) break;
    const long long at = (long long)(sp.row0 + tok) * P.Hq + sp.kh * P.G + r - tok * P.G;
    const float l = sm.joined[1][r];
    static_cast<bf16*>(P.a.out)[at * WI_D + tid] = __float2bfloat16_rn(l == 0.f ? 0.f : acc[r] / l);
    if (P.a.lse && tid == r) P.a.lse[at] = l == 0.f ? -INFINITY : sm.joined[0][r] * kLn2 + logf(l);
  }
}

template <int RP>
__global__ void __launch_bounds__(kThreads, 2) k_paged_attention8_few(const __grid_constant__ CUtensorMap map_k,
                                                                     const __grid_constant__ CUtensorMap map_v,
                                                                     const __grid_constant__ Few F) {
  using Sm = Smem<RP>;
  using Walk = WalkOver<kLead, 1, 0>;
  const Params& P = F.P;
  extern __shared__ __align__(1024) unsigned char raw[];
  pdl_trigger();
  Sm& sm = *reinterpret_cast<Sm*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (smem_addr(raw) & 1023u) {  // the swizzled tiles need 1024-byte alignment; never run misaligned
    if (tid == 0) atomicOr(P.err, WI_DEVERR_BAD_ROW);
    return;
  }
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_empty[s], 1);
    }
    mbar_init(&sm.q_full, kSoftWarps);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.s_full[t], 1);
      mbar_init(&sm.p_ready[t], kSoftWarps);
      mbar_init(&sm.o_done[t], 1);
    }
    mbar_init(&sm.drained, 1);
    sm.poison = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  constexpr uint32_t kCols = 32 + Sm::kPCols <= 64 ? 64 : 128;  // S twice (16 columns), O
  if (warp == kSoftWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm.tmem_base)),
                 "n"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == kSoftWarps && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_v)) : "memory");
  }
  for (int i = tid; i < Sm::kQCols * WI_D / 16; i += kThreads)  // columns that no query has: zero
    reinterpret_cast<uint4*>(sm.q)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  pdl_wait();
  tc_fence_before();
  const bool any = find_run<kLead, 1, kThreads>(P, kLeast, kLead + kWhole, kSlack, sm.scan, &sm.run);  // (with a barrier of all threads)
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;  // S at columns 0 and 16, O at 32
  if (!any) {  // the whole CTA leaves
    if (warp == kSoftWarps + 1)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kCols) : "memory");
    return;
  }

  if (warp < kSoftWarps) {
    // ---------------- softmax: a thread per position, then per element
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    bool ok = true;  // after one timed-out wait the warp waits no more and writes nothing, but meets every barrier
    int n = 0;       // blocks so far
    Walk w(P, sm.run.start, sm.run.req);
    bool more = w.next(P);
    Queries<RP> queries;
    auto put = [&] {  // once the products of the segment before are done with theirs
      queries.put(sm);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full);
    };
    if (more) {
      queries.ask(P, w);
      put();
    }
    soft_barrier();
    for (int seg = 0; more; ++seg) {
      float m[RP], l[RP], acc[RP], l_sum[RP], q_scale[RP];
      int lim[RP];  // the last position that a row sees; of no token: -1
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        m[r] = -INFINITY;
        l[r] = acc[r] = l_sum[r] = 0.f;
        const int tok = r / P.G, ti = w.tile * w.tp + tok;
        lim[r] = tok < P.tq && ti < w.r.n ? (int)(w.p0 + ti) : -1;
        q_scale[r] = sm.q_scale[r];
      }
      const int whole = w.first_pos();  // the last position that all rows see
      {  // the next segment, and its queries on their way
        Walk next = w;
        next.advance();
        more = next.next(P);
        if (more) queries.ask(P, next);
        if (lane == 0) *reinterpret_cast<Walk*>(sm.next[warp]) = next;
        __syncwarp();
      }
      for (int j = 0; j < w.nb; ++j, ++n) {
        const int st = n % kStages, buf = n & 1;
        if (ok) ok = mbar_wait(&sm.s_full[buf], (n >> 1) & 1, P.err);
        if (ok) ok = mbar_wait(&sm.v_full[st], (n / kStages) & 1, P.err);
        tc_fence_after();
        float s[RP], y[RP];
        {
          uint32_t a[2 * RP];
          if (RP == 4)
            tmem_ld8_nowait(tmem + lanes + buf * 16, reinterpret_cast<uint32_t(&)[8]>(a));
          else
            tmem_ld16_nowait(tmem + lanes + buf * 16, reinterpret_cast<uint32_t(&)[16]>(a));
          tmem_wait_ld();
#pragma unroll
          for (int r = 0; r < RP; ++r) s[r] = (__uint_as_float(a[r]) + __uint_as_float(a[RP + r])) * q_scale[r];
        }
        const float k_scale = sm.scale[st][0][tid / kGroup], v_exp = sm.scale[st][1][tid / kGroup];
        const int pos = (w.b0 + j) * kRows + tid;
        const bool fresh = j % kFlush == 0;  // O begins anew with this block
        if (fresh && j > 0) {
          if (ok) ok = mbar_wait(&sm.o_done[(n - 1) & 1], ((n - 1) >> 1) & 1, P.err);
          tc_fence_after();
          add_pieces<RP>(tmem + lanes + 32, acc);
#pragma unroll
          for (int r = 0; r < RP; ++r) {  // the sum so far, apart from what is to come
            l_sum[r] += l[r];
            l[r] = 0.f;
          }
        }
        bool grown = false;
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          s[r] = pos <= lim[r] ? s[r] * k_scale : -INFINITY;
          y[r] = s[r] + v_exp;
          grown |= y[r] - m[r] > kMost || s[r] - m[r] > kFarMost;
        }
        if (soft_any(grown)) {
          uint32_t mine = 0;
#pragma unroll
          for (int r = 0; r < RP; ++r) {
            if (y[r] - m[r] > kMost || s[r] - m[r] > kFarMost) mine |= 1u << r;
            const float top = warp_max(fmaxf(y[r] - kTop, s[r] - kFar));
            if (lane == 0) sm.xch[warp][r] = top;
          }
          mine = __reduce_or_sync(0xffffffffu, mine);
          if (lane == 0) sm.mask[warp] = (int)mine;
          soft_barrier();
          const int rows = sm.mask[0] | sm.mask[1] | sm.mask[2] | sm.mask[3];
          float f[RP];
#pragma unroll
          for (int r = 0; r < RP; ++r) {  // the other rows keep theirs
            const float top = fmaxf(fmaxf(sm.xch[0][r], sm.xch[1][r]), fmaxf(sm.xch[2][r], sm.xch[3][r]));
            f[r] = 1.f;
            if (rows >> r & 1) {
              f[r] = ex2(m[r] - fmaxf(m[r], top));
              m[r] = fmaxf(m[r], top);
            }
            l[r] *= f[r];
            l_sum[r] *= f[r];
            acc[r] *= f[r];
          }
          if (!fresh) {
            if (ok) ok = mbar_wait(&sm.o_done[(n - 1) & 1], ((n - 1) >> 1) & 1, P.err);
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < kPieces; ++i)
#pragma unroll
              for (int q = 0; q < RP; q += 4) {
                uint32_t a[4];
                tmem_ld4_nowait(tmem + lanes + 32 + i * RP + q, a);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 4; ++c) a[c] = __float_as_uint(__uint_as_float(a[c]) * f[q + c]);
                tmem_st4_nowait(tmem + lanes + 32 + i * RP + q, a);
              }
            tmem_wait_st();
          }
          soft_barrier();  // maxima and masks are read
        }
        const float back = pow2(-(int)v_exp);
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          y[r] = ex2(y[r] - (m[r] == -INFINITY ? 0.f : m[r]));
          l[r] += y[r] * back;
        }
        uint32_t b[kPieces][RP / 4];
        split<RP>(y, b);
        // piece i, words of four rows, one behind the other; no piece: zero
        auto word = [&](int i) -> uint32_t { return i < kPieces * RP / 4 ? b[i / (RP / 4)][i % (RP / 4)] : 0u; };
#pragma unroll
        for (int c = 0; c < Sm::kPCols / 16; ++c)
          reinterpret_cast<uint4*>(sm.p[buf] + 16 * tid)[c * kRows] =
              make_uint4(word(4 * c), word(4 * c + 1), word(4 * c + 2), word(4 * c + 3));
        if (pos > whole) {
          // A value that not every row sees: 0 * NaN is NaN inside the product, so rows behind the request's end are zeroed,
          // and so are NaN elements, which the end of the segment adds to the rows that see them.
          uint4* const v = reinterpret_cast<uint4*>(sm.v[st]) + tid * (WI_D / 16);
          bool found = false;
#pragma unroll
          for (int c = 0; c < WI_D / 16; ++c) {
            uint4 x = v[c];
            uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              // bit 7 of the bytes whose other bits are all ones
              const uint32_t nan = ((e[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
              if (pos >= w.r.kv) {
                e[k] = 0;
              } else if (nan) {
                e[k] &= ~((nan >> 7) * 0xffu);
                found = true;
              }
            }
            v[c] = make_uint4(e[0], e[1], e[2], e[3]);
          }
          if (found) *reinterpret_cast<volatile int*>(&sm.poison) = seg + 1;
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_ready[buf]);
      }

      // ---- the segment's end
      const Walk done = w;
      w = *reinterpret_cast<const Walk*>(sm.next[warp]);
      __syncwarp();
      soft_barrier();  // the queries' scales are read
      if (more) put();
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        l[r] = warp_sum(l[r] + l_sum[r]);
        if (lane == 0) sm.sum[warp][r] = l[r];
      }
      if (ok) ok = mbar_wait(&sm.o_done[(n - 1) & 1], ((n - 1) >> 1) & 1, P.err);
      tc_fence_after();
      add_pieces<RP>(tmem + lanes + 32, acc);
      tc_fence_before();  // O is read: the next segment may write it
      soft_barrier();
#pragma unroll
      for (int r = 0; r < RP; ++r) l[r] = (sm.sum[0][r] + sm.sum[1][r]) + (sm.sum[2][r] + sm.sum[3][r]);
      if (*reinterpret_cast<volatile int*>(&sm.poison) == seg + 1) {
        const int from = max(max(whole + 1, 0), done.b0 * kRows), to = min((done.b0 + done.nb) * kRows, done.r.kv);
#pragma unroll 1
        for (int p = from; p < to; ++p) {
          const int i = p / P.page, pg = P.a.block_table[(long long)done.b * P.max_pages + i];
          if (pg < 0 || pg >= P.n_pages) continue;
          const unsigned char v = static_cast<const unsigned char*>(
              P.a.v_pages)[(((long long)pg * P.Hkv + done.kh) * P.page + (p - i * P.page)) * WI_D + tid];
          if ((v & 0x7f) == 0x7f) {
#pragma unroll
            for (int r = 0; r < RP; ++r)
              if (p <= lim[r]) acc[r] = __uint_as_float(0x7fc00000u);
          }
        }
      }
      const bool part = done.b0 > 0 || done.nb < done.nblk;
      if (!part) {
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          const int tok = r / P.G, ti = done.tile * done.tp + tok;
          if (!ok || tok >= P.tq || ti >= done.r.n) break;
          const long long at = (long long)(done.r.s0 + ti) * P.Hq + done.kh * P.G + r - tok * P.G;
          static_cast<bf16*>(P.a.out)[at * WI_D + tid] = __float2bfloat16_rn(l[r] == 0.f ? 0.f : acc[r] / l[r]);
          if (P.a.lse && tid == r) P.a.lse[at] = l[r] == 0.f ? -INFINITY : m[r] * kLn2 + logf(l[r]);
        }
      } else {
        float* const dst = P.parts.slot(2 * (int)blockIdx.x + (done.b0 == 0 ? 1 : 0));
#pragma unroll
        for (int q = 0; q < RP; q += 4)
          __stcg(reinterpret_cast<float4*>(dst + (2 + tid) * RP + q), make_float4(acc[q], acc[q + 1], acc[q + 2], acc[q + 3]));
#pragma unroll
        for (int r = 0; r < RP; ++r)
          if (tid == r) {
            __stcg(dst + r, m[r]);
            __stcg(dst + RP + r, l[r]);
          }
        const long long item = sm.run.end - done.left - done.at + kLead;  // the unit of the item's first block
        const int c0 = cta_of(item, sm.run.total, sm.run.ctas), c1 = cta_of(item + done.nblk - 1, sm.run.total, sm.run.ctas);
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
          // behind the CTA's last segment the rings are free, else what the weights took
          join_parts<RP>(P, sm, {done.r.s0 + done.tile * done.tp, done.kh, done.cnt, c1}, c0, more ? sm.p[0] : sm.k[0],
                         more ? (int)(sizeof(sm.p) / (RP * WI_D * 4)) : Sm::kRings);
        }
      }
      soft_barrier();  // what the threads share is read, and the next segment's queries have their scales
    }
  } else if (warp == kSoftWarps) {
    // ---------------- TMA: keys, values, and the scales of their groups
    Walk w(P, sm.run.start, sm.run.req);
    const uint32_t on = elect_one();
    const int per = P.box / kGroup;  // groups of a box
    constexpr int kGroups = kRows / kGroup, kBatch = 32 / kGroups;
    int n = 0, asked[2] = {0, 0};  // blocks done with, blocks of keys and of values that were asked for
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
        return row < 0 ? kScaleBias * 0x101u : (uint32_t)F.s.k[row / kGroup] | (uint32_t)F.s.v[row / kGroup] << 8;
      };
      int page = page_of(0), row = 0, row_next = 0;
      uint32_t e = 0, e_next = 0;
      {
        const int ahead = page_of(1);
        row_next = row_of(page, 0);
        e_next = scales_of(row_next);
        page = ahead;
      }
      for (int j = 0; j < w.nb; ++j, ++n) {
        if (j % kBatch == 0) {
          row = row_next;
          e = e_next;
          row_next = row_of(page, j / kBatch + 1);
          e_next = scales_of(row_next);
          page = page_of(j / kBatch + 2);
        }
        const int st = n % kStages, first = j % kBatch * kGroups;  // first: the lane of the block's first group
        const uint32_t par = ((uint32_t)(n / kStages) & 1u) ^ 1u;
        // boxes behind the request's end are left out: always the last ones
        const int groups = __popc(__ballot_sync(0xffffffffu, row >= 0) >> first & ((1u << kGroups) - 1));
        const int boxes = (groups + per - 1) / per;
        const uint32_t bytes = (uint32_t)(boxes * P.box) * WI_D;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          uint64_t* const full = v ? &sm.v_full[st] : &sm.k_full[st];
          if (ok && n >= kStages) ok = mbar_wait(v ? &sm.v_empty[st] : &sm.k_empty[st], par, P.err);
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          const uint32_t dst = smem_addr(v ? sm.v[st] : sm.k[st]);
          for (int i = 0; i < boxes; ++i)
            tma_load_2d_warp(on, dst + (uint32_t)(i * P.box) * WI_D, v ? &map_v : &map_k, 0,
                             __shfl_sync(0xffffffffu, row, first + i * per), full);
          if (v && lane / kGroups == j % kBatch) {  // behind the copies: the scales may still be on their way here
            sm.scale[st][0][lane % kGroups] = pow2(scale_exponent((unsigned char)(e & 0xff)));
            sm.scale[st][1][lane % kGroups] = (float)scale_exponent((unsigned char)(e >> 8));
          }
          __syncwarp();
          if (on) mbar_arrive_expect_tx(full, bytes);  // the stage's one arrival: it is full when the bytes are there
          ++asked[v];
        }
        if (!ok) break;
      }
    }
    // no copy is in flight when the CTA's shared memory goes (after a timed-out wait nobody may have waited for them)
#pragma unroll
    for (int v = 0; v < 2; ++v)
      for (int s = 0; s < kStages && s < asked[v]; ++s)  // each stage's last use
        mbar_wait(v ? &sm.v_full[s] : &sm.k_full[s], (uint32_t)((asked[v] - 1 - s) / kStages) & 1u, P.err);
  } else {
    // ---------------- tensor cores: one lane issues, the whole warp computes what it issues
    Walk w(P, sm.run.start, sm.run.req);
    const uint32_t on = elect_one();
    constexpr uint32_t idesc_s = make_idesc_e4m3(kRows, Sm::kQCols);
    constexpr uint32_t idesc_o = make_idesc_e4m3(WI_D, Sm::kPCols) | kIdescMMajorA | kIdescNMajorB;
    // P without a swizzle: 128 bytes from eight positions to the next, 2048 from sixteen columns to the next
    constexpr uint32_t kPHi = (2048u >> 4) | (1u << 14), kPLo = (128u >> 4) << 16;
    auto all_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, P.err));
    };
    bool ok = true;
    auto scores = [&](int n) -> bool {
      const int st = n % kStages, buf = n & 1;
      if (!all_wait(&sm.k_full[st], (uint32_t)(n / kStages) & 1u)) return false;
      tc_fence_after();
      const uint32_t d = __shfl_sync(0xffffffffu, tmem + (uint32_t)buf * 16, 0);
      const uint32_t a = __shfl_sync(0xffffffffu, desc_lo_kmajor(smem_addr(sm.k[st])), 0);
      const uint32_t b = __shfl_sync(0xffffffffu, desc_lo_kmajor(smem_addr(sm.q)), 0);
#pragma unroll
      for (int kk = 0; kk < WI_D / 32; ++kk)
        mma_e4m3_warp(on, d, a + kk * 2, desc_hi_sw128(1024), b + kk * 2, desc_hi_sw128(1024), idesc_s, kk > 0);
      mma_commit_warp(on, &sm.s_full[buf]);
      mma_commit_warp(on, &sm.k_empty[st]);
      return true;
    };
    int n = 0;
    for (int seg = 0; ok && w.next(P); ++seg, w.advance()) {
      if (!(ok = all_wait(&sm.q_full, seg & 1))) break;
      tc_fence_after();
      if (!(ok = scores(n))) break;
      for (int j = 0; j < w.nb; ++j, ++n) {
        if (j + 1 < w.nb && !(ok = scores(n + 1))) break;
        const int st = n % kStages, buf = n & 1;
        if (!(ok = all_wait(&sm.p_ready[buf], (uint32_t)(n >> 1) & 1u))) break;
        if (!(ok = all_wait(&sm.v_full[st], (uint32_t)(n / kStages) & 1u))) break;
        tc_fence_after();
        const uint32_t d = __shfl_sync(0xffffffffu, tmem + 32u, 0);
        const uint32_t a = __shfl_sync(0xffffffffu, desc_lo_kmajor(smem_addr(sm.v[st])), 0);
        const uint32_t b = __shfl_sync(0xffffffffu, (smem_addr(sm.p[buf]) >> 4) | kPLo, 0);
        const uint32_t add = __shfl_sync(0xffffffffu, (uint32_t)(j % kFlush != 0), 0);
#pragma unroll
        for (int kk = 0; kk < kRows / 32; ++kk)
          mma_e4m3_warp(on, d, a + kk * (32 * WI_D / 16), desc_hi_sw128(1024), b + kk * 32, kPHi, idesc_o, kk > 0 ? 1u : add);
        mma_commit_warp(on, &sm.v_empty[st]);
        mma_commit_warp(on, &sm.o_done[buf]);
      }
    }
    // every product is done before the tensor memory goes
    mma_commit_warp(on, &sm.drained);
    mbar_wait(&sm.drained, 0, P.err);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps + 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kCols) : "memory");
  }
}

template <int RP>
cudaError_t launch(const Few& F, const CUtensorMap& map_k, const CUtensorMap& map_v, int grid, cudaStream_t st) {
  static int smem_set[kWiSmemDevices] = {};
  auto* kernel = k_paged_attention8_few<RP>;
  static_assert(offsetof(Smem<RP>, q) % 1024 == 0 && offsetof(Smem<RP>, k) % 1024 == 0, "tiles must start 1024-byte aligned");
  static_assert(2 * (sizeof(Smem<RP>) + 1024) <= 228 * 1024, "two CTAs to an SM");
  const cudaError_t e = wi_ensure_smem(kernel, sizeof(Smem<RP>), smem_set);
  if (e != cudaSuccess) return e;
  return wi_launch_chained(kernel, dim3((unsigned)grid), kThreads, sizeof(Smem<RP>), st, map_k, map_v, F);
}

}  // namespace

// Lengths are on the device, so the host goes by the average.  A chunk among single tokens is then cut into tiles of a few rows,
// which read its context once each; that is still less than tiles of 128 rows lose on the single tokens: 255 of them and 769 of
// one request over 2000 positions 312 us (8 heads without grouping), 471 there; 256 requests' four tokens 191 and 433, 64 single
// ones 70 and 130.  Only a chunk beside requests that have no tokens at all is better off there: 256 tokens of one request and
// none of 255 others 208 and 43.
bool wi_paged_few(const WiPagedGeom& g, const WiPagedAttn& a) {
  const int tq = (g.G <= 4 ? 4 : 8) / g.G;
  return a.n_tokens <= (long long)a.batch * tq;
}

cudaError_t wi_launch_paged_few(const WiPagedGeom& g, const WiPagedAttn& a, const WiPagedScales& s, int sms, void* scratch,
                                int* err, cudaStream_t st) {
  const int rp = g.G <= 4 ? 4 : 8;
  Few F;
  Params& P = F.P;
  F.s = s;
  P.a = a;
  P.Hq = g.Hq;
  P.Hkv = g.Hkv;
  P.G = g.G;
  P.tq = rp / g.G;
  P.page = g.page;
  P.n_pages = g.n_pages;
  P.max_pages = g.max_pages;
  // a box of a block lies inside one page: the largest power of two that divides the page, 128 at most
  P.box = g.page & -g.page;
  if (P.box > kRows) P.box = kRows;
  P.splits = nullptr;
  P.tickets = static_cast<unsigned*>(scratch);
  P.parts = {reinterpret_cast<float*>(static_cast<char*>(scratch) + kPagedTicketBytes), rp, 1};
  P.err = err;
  CUtensorMap map_k, map_v;
  const unsigned long long rows = (unsigned long long)g.n_pages * g.Hkv * g.page;
  if (!wi_encode_bytes_sw128(&map_k, a.k_pages, rows, (unsigned)P.box) ||
      !wi_encode_bytes_sw128(&map_v, a.v_pages, rows, (unsigned)P.box))
    return cudaErrorInvalidValue;
  const int grid = 2 * sms < kPagedMaxSms ? 2 * sms : kPagedMaxSms;
  return rp == 4 ? launch<4>(F, map_k, map_v, grid, st) : launch<8>(F, map_k, map_v, grid, st);
}
