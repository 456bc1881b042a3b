// wi_paged_attn.cu -- attention of new tokens over the paged cache on the
// 5th-generation tensor cores.
//
// out = softmax(q K^T / sqrt(128)) V over the positions a token sees, for
// every (token, query head).  The query heads of a kv head share its keys, so
// the rows of a tile are (token, query head of the group) pairs: floor(128/G)
// tokens to a tile of 128 rows.
//
// Work.  An item is one (request, kv head, pair of tiles); its key blocks of
// 128 positions run from 0 to the last position that a row sees.  A unit is
// one block of one item, or one of four more for its start and end; all units
// of the call, item after item, are cut into equal runs, one per CTA (one CTA
// per SM), so single tokens over long contexts split over the machine and
// ragged chunks balance without a plan made on the host.  Lengths live on the
// device: each CTA sums the units of all requests itself (closed form per
// request) and finds its run's start.
// An item cut between CTAs leaves partial results (maximum, sum, O) in the
// scratch, added up in CTA order: by the last of its CTAs where the call has
// 32 rows per kv head at most (single tokens of a few requests, a few tokens
// of one), else by k_paged_merge, which spreads the rows over the machine.
// (Eight tokens over 1000 positions: 13.8 and 26.7 us, over 131K 94 and 121,
// eight requests' single tokens over 4000 34.4 and 38.3.)
//
// A CTA (384 threads) processes its items' blocks in roles:
//   warps 0-3, 4-7  softmax, one thread per row of chain 0 / chain 1
//   warp 8          TMA: queries, key and value blocks (box by box, through
//                   the block table) into a ring of five 32 KB stages
//   warp 9          issues tcgen05.mma: S = Q K^T (both operands in shared
//                   memory), O += P V (P in tensor memory, V N-major)
//   warps 10-11     clean value rows of blocks that not every row sees whole
// The two chains have their own S (P takes S's place) and O in tensor memory
// (all 512 columns), so that one chain's softmax runs while the tensor cores
// work on the other.  In an item of two tiles the chains are the tiles, and
// share the key and value blocks; an item of one tile (single tokens above
// all) gives the chains alternate blocks of the same tile and adds their
// results at the end.
//
// Masked positions.  Keys of unseen positions may hold anything: their scores
// are replaced, not added to.  Values are different: 0 * Inf is NaN inside the
// product.  In blocks that not every row sees whole, rows behind the request's
// end are zeroed in shared memory, and so are infinite and NaN elements, which
// the end of the item then adds to the rows that do see them.
//
// What bounds it, 32 query and 8 kv heads on one GB300.  Chunks: the tensor
// pipe, 72% active while a CTA runs; 2048 tokens behind 14K positions 316 -
// 322 us, 1600 - 1630 TFLOP/s, 0.85 - 0.87 of the measured bf16 peak (behind
// 129K, call after call under the power cap, 3.1 - 3.4 ms, 0.75 - 0.82 of the
// sustained peak; a few calls alone 2.7 - 2.9).  Each role is kept short: one
// thread computing the operands of tcgen05.mma under a branch took 3345 of
// 4230 cycles a block (hence mma_bf16_warp), a maximum of every block and two
// threads to a row 1750 cycles of softmax where 1100 do.  The code's size
// matters as much: loops that were unrolled further, or a form of its own for
// tiles of few rows, slowed every other loop of the kernel.
// Single tokens: HBM; 131K positions in pages of 16 in 90 - 98 us, 5.5 - 6.0
// TB/s, of which the start takes 6, the reads 70 (7.6 TB/s) and the merge of
// twenty parts per head 5.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>

#include "wi_common.cuh"
#include "wi_internal.h"
#include "wi_paged.h"
#include "wi_paged_merge.cuh"
#include "wi_paged_walk.cuh"
#include "wi_pipe.cuh"
#include "wi_tc.cuh"

namespace {

constexpr int kStages = 5;
constexpr int kTileBytes = kRows * WI_D * 2;   // 32 KB: two halves of 64 columns
constexpr int kHalfBytes = kTileBytes / 2;
constexpr int kSoftWarps = 8;
constexpr int kThreads = 32 * (kSoftWarps + 4);
constexpr int kFixWarps = 2;
constexpr float kScaleLog2 = 0.08838834764831845f * 1.4426950408889634f;  // log2(e) / sqrt(128)
// Units in front of an item's blocks, for what its start and end cost (8192 fresh tokens, 32 / 8 heads: 542, 502, 466,
// 439, 444 us at 1, 2, 3, 4, 6 in an earlier form; longer contexts and single tokens do not care).
constexpr int kLead = 4;
// One request of few rows is not cut up to this many blocks: a merge costs 4 us, a block behind the first 0.7 (five
// tokens over 305 positions 10.6 us whole, 12.4 cut; one over 500 11.3 and 12.1, over 800 15.7 and 12.9).  Several
// requests are: as many equal runs as there are items are whole items only where all requests are as long as each other
// (two of four tokens over 305 11.0 us, 12.1 cut), and elsewhere are cut all the same, into fewer parts (four tokens over
// 100 and over 500 16.8 us, 12.0 cut; single tokens over 50, 500, 300 and 200 18.8 and 13.5).
constexpr int kWhole = 4;
// Blocks that one segment has at most: what a CTA has of a longer item is added up in fp32 by its softmax warps, one
// segment after the other (a segment costs 5 us, 2048 blocks 1400).  The tensor cores' own additions cut bits off: equal
// weights over values of one sign came out 0.02% too small after 2^18 positions without a break, 0.3% after 2^20, 0.9% after
// 2^21, and a sum of 2^26 took no more.  The kernel has an instance of its own (LONG) for caches whose requests can be that
// long: the few instructions more at a segment's end cost single tokens over short contexts 4% (64 over 1000 positions
// 75.2 us, 72.4 without), chunks 1%.
constexpr int kLongest = 2048;
// Cycles that a block may take (1500 do), for the waits that may last through a run of a LONG instance.
constexpr long long kBlockCycles = 1 << 14;
// A row's weights are 2^(score - m) with m the row's maximum in the first block of its part, which no later block needs
// to know its own maximum for: only when a block's weights add up to more than this (one of them is 2^9 at least), or to
// no number, the block is done again with the maximum so far, and O rescaled.  Weights below 2^16 cost neither bf16 nor
// fp32 any precision.
constexpr float kAgain = 65536.f;

template <bool LONG>
using Walk = WalkOver<kLead, 2, LONG ? kLongest : 0>;

struct Smem {
  uint64_t full[kStages], empty[kStages];
  uint64_t to_fix[kStages], fixed[kStages];  // a value block that is to be cleaned was asked for; has been cleaned
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_ready[2], o_full[2];
  uint64_t drained;
  uint32_t tmem_base;
  int last;                 // this CTA merges the item that it just added to
  int poison[8];            // segment number + 1 of the last segment (modulo 8) with an infinite or NaN value
  long long scan[kThreads / 32];
  Run run;
  Req reqs[kSoftWarps];     // of the softmax warps' segments
  float xch[2][2][kRows];   // maximum and sum of a row, from chain to chain: [chain][m, l]
  alignas(1024) unsigned char q[2][kTileBytes];          // [k half][128 rows][128 B]
  unsigned char ring[kStages][kTileBytes]; // [group of 8 rows][k half][8 rows][128 B]
};
static_assert(offsetof(Smem, q) == 3 * 1024, "tiles must start 1024-byte aligned");
static_assert(sizeof(Smem) <= 232448, "shared memory");

// A position in the ring: the stage, and the parity of its current use.
struct Ring {
  int s = 0;
  uint32_t par = 0;
  __device__ __forceinline__ void step() {
    if (++s == kStages) {
      s = 0;
      par ^= 1;
    }
  }
  __device__ __forceinline__ void step(int n) {  // n < kStages
    s += n;
    if (s >= kStages) {
      s -= kStages;
      par ^= 1;
    }
  }
};

// Scores behind column `seen` of 64 are not seen.
__device__ __forceinline__ void mask_scores(uint32_t (&s)[2][32], int seen) {
#pragma unroll
  for (int i = 0; i < 64; ++i)
    if (i > seen) s[i >> 5][i & 31] = 0xFF800000u;  // -infinity
}

__device__ __forceinline__ float top_score(const uint32_t (&s)[2][32]) {
  float t[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint32_t* x = s[c >> 1] + (c & 1) * 16;
    t[c] = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
#pragma unroll
    for (int i = 2; i < 16; i += 2) t[c] = max3(t[c], __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
  }
  return fmaxf(max3(t[0], t[1], max3(t[2], t[3], -INFINITY)), -INFINITY);
}

// 32 scores to weights 2^(score * log2(e) / sqrt(128) - ref): added to `sum`, and as bf16 to 16 columns of P.  The
// tensor cores take both operands of a product in one type and the values are bf16, so the weights are too, the one
// rounding before the output's; a second product with what the rounding leaves would be half as much tensor work again.
// Against 64 bits the output is 1.6e-3 - 1.8e-3 off (relative 2-norm), as it is with fp32 weights to within 5e-5: its own
// rounding is most of it.
__device__ __forceinline__ void weights(const uint32_t (&s)[32], uint32_t tp, float ref, uint64_t (&sum)[2]) {
  const uint64_t scale2 = pair(kScaleLog2, kScaleLog2), ref2 = pair(-ref, -ref);
  uint32_t p[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint64_t x = fma2(pair(s[2 * i], s[2 * i + 1]), scale2, ref2);
    const float a = ex2(lo_of(x)), b = ex2(hi_of(x));
    sum[i & 1] = add2(sum[i & 1], pair(a, b));
    p[i] = pack2(a, b);
  }
  tmem_st16_nowait(tp, p);
}

__device__ __forceinline__ void soft_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftWarps * 32) : "memory"); }

__device__ __forceinline__ bool nonfinite16(uint32_t h) { return (h & 0x7F80u) == 0x7F80u; }
// Two bf16 values at once: bit 15 / 31 set where the exponent is all ones (one more in its last place carries over it).
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) { return (w & 0x7F807F80u) + 0x00800080u; }

// Add the infinite and NaN values that a row sees at positions [from, to), where they were taken out, to 16 columns of
// its O.
__device__ __forceinline__ void add_poison(const Params& P, int b, int kh, int from, int to, int limit, int c0,
                                           float (&o)[16]) {
  const int end = min(to, limit + 1);
#pragma unroll 1
  for (int p = from; p < end; ++p) {
    const int j = p / P.page, pg = P.a.block_table[(long long)b * P.max_pages + j];
    if (pg < 0 || pg >= P.n_pages) continue;
    const uint32_t* v = static_cast<const uint32_t*>(P.a.v_pages) +
                        ((((long long)pg * P.Hkv + kh) * P.page + (p - j * P.page)) * WI_D + c0) / 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = v[i];
      if (nonfinite16(w)) o[2 * i] += bf16_lo(w);
      if (nonfinite16(w >> 16)) o[2 * i + 1] += bf16_hi(w);
    }
  }
}

// Units of the requests [rb0, rb1) of this thread, of the threads in front of it, and of all: what the kernel's start
// works out in line, once more for calls that are not in order (a loop around that code took 1% of single tokens' time).
struct Share {
  long long mine, before, total;
};
__device__ __noinline__ Share share_of(const Params& P, long long* scan, int rb0, int rb1) {
  const int tp = 2 * P.tq;
  Share x = {0, 0, 0};
  for (int b = rb0; b < rb1; ++b) {
    const Req r = load_req(P, b);
    if (r.n > 0) x.mine += P.Hkv * units_of<kLead>(r, tp);
  }
  __syncthreads();  // every warp has read the sums that stood there
  add_up<kThreads>(x.mine, scan, x.before, x.total);
  return x;
}

template <bool LONG>
__global__ void __launch_bounds__(kThreads, 1) k_paged_attention(const __grid_constant__ CUtensorMap map_q,
                                                                const __grid_constant__ CUtensorMap map_k,
                                                                const __grid_constant__ CUtensorMap map_v,
                                                                const __grid_constant__ Params P) {
  extern __shared__ __align__(1024) unsigned char raw[];
  pdl_trigger();  // the next kernel may take the SMs as they fall free; it waits for this grid before it reads
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (smem_addr(raw) & 1023u) {  // the swizzled tiles need 1024-byte alignment; never run misaligned
    if (tid == 0) atomicOr(P.err, WI_DEVERR_BAD_ROW);
    return;
  }

  // ---- what needs nothing of the kernels before this one
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
      mbar_init(&sm.to_fix[s], 1);
      mbar_init(&sm.fixed[s], kFixWarps);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sm.s_full[t], 1);
      mbar_init(&sm.p_ready[t], kSoftWarps / 2);
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
  if (P.tq * P.G < kRows) {  // rows of the query tiles that no box fills: zero, not whatever was there
    for (int i = tid; i < 2 * kTileBytes / 16; i += kThreads)
      reinterpret_cast<uint4*>(sm.q)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  pdl_wait();

  // ---- this CTA's run of units
  const int per = (P.a.batch + kThreads - 1) / kThreads;
  const int rb0 = min(tid * per, P.a.batch);
  int rb1 = min(rb0 + per, P.a.batch);
  const int tp = 2 * P.tq;
  long long mine = 0, cost = 0;  // cost: of one kv head of the last request looked at
  Req r = {0, 0, 0, 1};
  for (int b = rb0; b < rb1; ++b) {
    r = load_req(P, b);
    if (!r.ok) {
      if (blockIdx.x == 0) atomicOr(P.err, WI_DEVERR_BAD_LENGTH);
      if (P.a.q_start[b + 1] < r.s0) mine += kFalls;
    }
    if (r.n == 0) continue;
    cost = units_of<kLead>(r, tp);
    mine += P.Hkv * cost;
  }
  long long before, total;
  tc_fence_before();
  add_up<kThreads>(mine, sm.scan, before, total);
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;  // S0, S1 at columns 0, 128; O0, O1 at 256, 384
  // q_start falls somewhere, or lengths add up to more than a run can count (through pages shared by many requests)
  const long long most = (long long)gridDim.x * 0x3fffffff;
  if (total > most) {
    if (blockIdx.x == 0 && tid == 0) atomicOr(P.err, WI_DEVERR_BAD_LENGTH);
    rb1 = min(rb1, requests_in_order(P));
    const Share x = share_of(P, sm.scan, rb0, rb1);
    mine = x.mine;
    before = x.before;
    total = x.total > most ? 0 : x.total;  // too much still: nothing is done
  }
  int ctas = (int)min((long long)gridDim.x, total);
  // (see kWhole: the items of one request are alike, so that a run per kv head is an item)
  if (P.tickets && P.a.batch == 1 && ctas > P.Hkv && total <= (long long)P.Hkv * (kLead + kWhole)) ctas = P.Hkv;
  if ((int)blockIdx.x >= ctas) {  // fewer units than CTAs (the whole CTA leaves)
    if (tid == 0) P.splits[blockIdx.x].last = -1;
    if (warp == kSoftWarps + 1)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    return;
  }
  const long long u0 = quot(total * blockIdx.x, ctas), u1 = quot(total * (blockIdx.x + 1), ctas);
  if (u0 >= before && u0 < before + mine)  // (where each thread has one request, that is at hand)
    begin_run<kLead>(P, tp, rb0, rb1, per == 1, r, cost, before, u0, u1, total, ctas, &sm.run);
  __syncthreads();

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
    // behind them, from the request as the warp keeps it in shared memory.  The next segment begins with the walk that
    // ended the last one (64 single tokens over 1000 positions: 76.0 us with the request read at both ends, now 72.9).
    Cursor cur;
    int nb, step, from, base, limit, whole;
    auto begin = [&](Walk<LONG>& w) {
      const bool more = w.next(P);
      cur = w;
      if (lane == 0) sm.reqs[warp] = w.r;
      __syncwarp();
      const int own_tile = w.single ? 0 : chain, ti = w.tile * w.tp + own_tile * P.tq + tok;
      limit = tok < P.tq && ti < w.r.n ? (int)(w.p0 + ti) : -1;     // the last position that the row sees
      whole = (int)(w.p0 + w.tile * w.tp + own_tile * P.tq);       // ... that all rows of the tile see
      nb = w.nb;
      step = w.single ? 2 : 1;
      from = w.single ? chain : 0;
      base = w.b0 * kRows;
      return more;
    };
    bool more;
    {
      Walk<LONG> w(P, sm.run.start, sm.run.req);
      more = begin(w);
    }
    for (int seg = 0; more; ++seg) {
      float m = -INFINITY, l = 0.f;  // the row's reference maximum and its sum
      for (int j = from; j < nb; j += step) {
        if (ok) ok = mbar_wait(&sm.s_full[chain], s_par, P.err);
        s_par ^= 1;
        tc_fence_after();
        // The second half of the scores comes while the first is worked on; P then takes the place of the first half,
        // which stays in registers, so that the block can be done again.
        uint32_t a[2][32], b[2][32];
        tmem_ld32_nowait(ts, a[0]);
        tmem_ld32_nowait(ts + 32, a[1]);
        tmem_wait_ld();
        tmem_ld32_nowait(ts + 64, b[0]);
        tmem_ld32_nowait(ts + 96, b[1]);
        const bool masked = base + j * kRows + kRows - 1 > whole;
        const int seen = limit - base - j * kRows;  // the row sees columns 0 .. seen of this block
        if (masked) mask_scores(a, seen);
        bool again = j == from, grown = again;  // grown: this row takes a new reference (other rows keep theirs)
        for (;;) {
          if (again) {  // the first block, or the reference is far too small
            tmem_wait_st();
            tmem_wait_ld();
            tmem_ld32_nowait(ts + 64, b[0]);
            tmem_ld32_nowait(ts + 96, b[1]);
            tmem_wait_ld();
            if (masked) mask_scores(b, seen - 64);
            const float top = grown ? fmaxf(m, fmaxf(top_score(a), top_score(b)) * kScaleLog2) : m;
            if (j != from) {
              // the chain's products so far are done: S of this block was issued behind them
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
          const float ref = m == -INFINITY ? 0.f : m;  // nothing seen so far: every weight is 2^-inf = 0
          uint64_t sum[2] = {0ull, 0ull};
          weights(a[0], ts, ref, sum);
          weights(a[1], ts + 16, ref, sum);
          tmem_wait_ld();
          if (masked && !again) mask_scores(b, seen - 64);
          weights(b[0], ts + 32, ref, sum);
          weights(b[1], ts + 48, ref, sum);
          const uint64_t both = add2(sum[0], sum[1]);
          const float z = lo_of(both) + hi_of(both);
          // A row without a reference (every score so far minus infinity) looks for one in each block that it sees
          // something of: against 0 its weights might all vanish.  A row that sees nothing of the block, or that no token
          // owns, asks for nothing, whatever its query holds.
          grown = seen >= 0 && (!(z <= kAgain) || m == -INFINITY);
          if (again || !__any_sync(0xffffffffu, grown)) {
            l += z;
            break;
          }
          again = true;
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_ready[chain]);
      }

      // ---- the segment's end: maximum and sum over both chains where they had one tile, then O
      Walk<LONG> w(P, cur, sm.reqs[warp]);
      w.next(P);
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
            uint4* q = reinterpret_cast<uint4*>(static_cast<bf16*>(P.a.out) + at * WI_D + c);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint4 x;
              x.x = pack2(o[8 * i] * inv, o[8 * i + 1] * inv);
              x.y = pack2(o[8 * i + 2] * inv, o[8 * i + 3] * inv);
              x.z = pack2(o[8 * i + 4] * inv, o[8 * i + 5] * inv);
              x.w = pack2(o[8 * i + 6] * inv, o[8 * i + 7] * inv);
              q[i] = x;
            }
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
      w.advance();
      more = begin(w);
    }
    if (tid == 0 && !split) P.splits[blockIdx.x].last = -1;
  } else if (warp == kSoftWarps) {
    Walk<LONG> w(P, sm.run.start, sm.run.req);
    // ---------------- TMA: queries, keys, values
    const uint32_t on = elect_one();
    const int boxes = kRows / P.box;  // boxes of a block, one lane finds the page of each
    const uint32_t q_half = (uint32_t)(P.tq * P.G) * 128u;
    Ring at;                          // the next ring stage to fill
    int filled = 0;                   // stages filled so far, counted up to the ring's length
    int q_loads = 0, last = 0;        // last: the stage filled last
    bool ok = true;
    for (int seg = 0; ok && w.next(P); ++seg) {
      const int ahead = w.single ? 2 : 1;
      // This lane's box of block j of the segment: its page as the table has it, looked up blocks ahead and looked at
      // when the copy is due (kNone: behind the request's end).
      constexpr int kNone = -0x7fffffff - 1;
      auto page_of = [&](int j) -> int {
        const int p = (w.b0 + j) * kRows + lane * P.box;
        if (j >= w.nb || lane >= boxes || p >= w.r.kv) return kNone;
        return P.a.block_table[(long long)w.b * P.max_pages + p / P.page];
      };
      auto row_of = [&](int pg, int j) -> int {
        if (pg == kNone) return -1;
        if (pg < 0 || pg >= P.n_pages) {
          atomicOr(P.err, WI_DEVERR_BAD_PAGE);
          pg = 0;
        }
        return (pg * P.Hkv + w.kh) * P.page + ((w.b0 + j) * kRows + lane * P.box) % P.page;
      };
      int g0 = page_of(0), g1 = page_of(1), g2 = page_of(2);
      // queries, once the products of the segment before have read theirs
      if (seg > 0) ok = mbar_wait(&sm.q_empty, (seg - 1) & 1, P.err);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      if (lane == 0) {
        const int n = w.single ? 1 : 2;
        mbar_arrive_expect_tx(&sm.q_full, 2u * q_half * n);
        for (int t = 0; t < n; ++t) {
          const int tk = w.r.s0 + w.tile * w.tp + t * P.tq;
          tma_load_3d(sm.q[t], &map_q, 0, w.kh * P.G, tk, &sm.q_full);
          tma_load_3d(sm.q[t] + kHalfBytes, &map_q, 64, w.kh * P.G, tk, &sm.q_full);
        }
      }
      ++q_loads;
      auto fill = [&](const CUtensorMap* map, int pg, int j) -> bool {
        const int rowi = row_of(pg, j);
        bool got = true;
        if (filled == kStages) got = mbar_wait(&sm.empty[at.s], at.par ^ 1u, P.err);
        if (!__all_sync(0xffffffffu, got)) return false;
        // boxes behind the request's end are left out: always the last ones
        const int n = __popc(__ballot_sync(0xffffffffu, rowi >= 0));
        if (on) mbar_arrive_expect_tx(&sm.full[at.s], (uint32_t)(n * P.box) * 256u);
        __syncwarp();
        const uint32_t dst = smem_addr(sm.ring[at.s]);
        for (int i = 0; i < n; ++i)
          tma_load_4d_warp(on, dst + (uint32_t)(i * P.box) * 256u, map, 0, 0, 0, __shfl_sync(0xffffffffu, rowi, i) >> 3,
                           &sm.full[at.s]);
        last = at.s;
        at.step();
        if (filled < kStages) ++filled;
        return true;
      };
      ok = fill(&map_k, g0, 0);
      if (ok && ahead == 2 && w.nb > 1) ok = fill(&map_k, g1, 1);
      for (int j = 0; ok && j < w.nb; ++j) {
        const int g3 = page_of(j + 3);
        ok = fill(&map_v, g0, j);
        if (ok && lane == 0 && w.b0 + j >= w.first_fix()) mbar_arrive(&sm.to_fix[last]);
        if (ok && j + ahead < w.nb) ok = fill(&map_k, ahead == 2 ? g2 : g1, j + ahead);
        g0 = g1;
        g1 = g2;
        g2 = g3;
      }
      w.advance();
    }
    // no copy is in flight when the CTA's shared memory goes (after a timed-out wait the tensor cores may not have
    // waited for them)
    if (q_loads > 0) mbar_wait(&sm.q_full, (uint32_t)(q_loads - 1) & 1u, P.err);
    for (int s = 0; s < filled; ++s)  // the last use of each stage: this turn's in front of `at`, else the turn before
      mbar_wait(&sm.full[s], s < at.s ? at.par : at.par ^ 1u, P.err);
  } else if (warp == kSoftWarps + 1) {
    Walk<LONG> w(P, sm.run.start, sm.run.req);
    // ---------------- tensor cores: one lane issues, the whole warp computes what it issues
    {
      const uint32_t on = elect_one();
      constexpr uint32_t idesc_s = make_idesc(kRows, kRows);
      constexpr uint32_t idesc_o = make_idesc(kRows, WI_D) | kIdescNMajorB;
      Ring at;                   // the next ring stage to consume
      uint32_t p_par = 0, fix_par = 0;
      bool ok = true;
      auto all_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, P.err));
      };
      auto scores = [&](int t, int q, int s) {
        const uint32_t d = __shfl_sync(0xffffffffu, tmem + (uint32_t)t * kRows, 0);
        const uint32_t a0 = __shfl_sync(0xffffffffu, desc_lo_kmajor(smem_addr(sm.q[q])), 0);
        const uint32_t b0 = __shfl_sync(0xffffffffu, desc_lo_kmajor(smem_addr(sm.ring[s])), 0);
#pragma unroll
        for (int kk = 0; kk < WI_D / 16; ++kk) {
          const uint32_t off = ((uint32_t)(kk >> 2) * kHalfBytes + (uint32_t)(kk & 3) * 32) / 16;
          const uint32_t offb = ((uint32_t)(kk >> 2) * 1024 + (uint32_t)(kk & 3) * 32) / 16;
          mma_bf16_warp(on, d, a0 + off, desc_hi_sw128(1024), b0 + offb, desc_hi_sw128(2048), idesc_s, kk > 0);
        }
        mma_commit_warp(on, &sm.s_full[t]);
      };
      auto values = [&](int t, int s, bool add) {
        const uint32_t p = __shfl_sync(0xffffffffu, tmem + (uint32_t)t * kRows, 0);
        const uint32_t b0 = __shfl_sync(0xffffffffu, desc_lo_nmajor(smem_addr(sm.ring[s]), 1024), 0);
        const uint32_t more = __shfl_sync(0xffffffffu, (uint32_t)add, 0);
        const uint32_t d = __shfl_sync(0xffffffffu, tmem + 256u + (uint32_t)t * WI_D, 0);
#pragma unroll
        for (int kk = 0; kk < kRows / 16; ++kk)
          mma_bf16_ta_warp(on, d, p + (uint32_t)kk * 8, b0 + (uint32_t)kk * (4096 / 16), desc_hi_sw128(2048), idesc_o,
                           kk > 0 ? 1u : more);
      };
      auto take = [&](int* st) -> bool {  // the next ring stage, once it is full
        *st = at.s;
        const bool got = all_wait(&sm.full[at.s], at.par);
        at.step();
        tc_fence_after();
        return got;
      };
      for (int seg = 0; ok && w.next(P); ++seg) {
        ok = all_wait(&sm.q_full, seg & 1);
        if (!ok) break;
        tc_fence_after();
        const int fix = w.first_fix() - w.b0;  // from this block of the segment on, values are cleaned first
        int ks, vs;
        if (!(ok = take(&ks))) break;
        scores(0, 0, ks);
        if (w.single) {
          mma_commit_warp(on, &sm.empty[ks]);
          if (w.nb > 1) {
            if (!(ok = take(&ks))) break;
            scores(1, 0, ks);
            mma_commit_warp(on, &sm.empty[ks]);
          }
        } else {
          scores(1, 1, ks);
          mma_commit_warp(on, &sm.empty[ks]);
        }
        if (w.nb <= (w.single ? 2 : 1)) mma_commit_warp(on, &sm.q_empty);
        for (int j = 0; j < w.nb; ++j) {
          if (!(ok = take(&vs))) break;
          if (j >= fix) {
            ok = all_wait(&sm.fixed[vs], (fix_par >> vs) & 1u);
            fix_par ^= 1u << vs;
            if (!ok) break;
          }
          if (w.single) {
            const int t = j & 1;
            if (!(ok = all_wait(&sm.p_ready[t], (p_par >> t) & 1u))) break;
            p_par ^= 1u << t;
            tc_fence_after();
            values(t, vs, j >= 2);
            mma_commit_warp(on, &sm.empty[vs]);
            if (j + 2 >= w.nb) {
              mma_commit_warp(on, &sm.o_full[t]);
            } else {
              if (!(ok = take(&ks))) break;
              scores(t, 0, ks);
              mma_commit_warp(on, &sm.empty[ks]);
              if (j + 3 >= w.nb) mma_commit_warp(on, &sm.q_empty);
            }
          } else {
            const bool more = j + 1 < w.nb;
            if (!(ok = all_wait(&sm.p_ready[0], (p_par >> 0) & 1u))) break;
            p_par ^= 1u;
            tc_fence_after();
            values(0, vs, j > 0);
            if (more) {
              if (!(ok = take(&ks))) break;
              scores(0, 0, ks);
            } else {
              mma_commit_warp(on, &sm.o_full[0]);
            }
            if (!(ok = all_wait(&sm.p_ready[1], (p_par >> 1) & 1u))) break;
            p_par ^= 2u;
            tc_fence_after();
            values(1, vs, j > 0);
            mma_commit_warp(on, &sm.empty[vs]);
            if (more) {
              scores(1, 1, ks);
              mma_commit_warp(on, &sm.empty[ks]);
              if (j + 2 >= w.nb) mma_commit_warp(on, &sm.q_empty);
            } else {
              mma_commit_warp(on, &sm.o_full[1]);
            }
          }
        }
        if (!ok) break;
        w.advance();
      }
      // every product is done before the tensor memory goes
      mma_commit_warp(on, &sm.drained);
      mbar_wait(&sm.drained, 0, P.err);
    }
  } else {
    Walk<LONG> w(P, sm.run.start, sm.run.req);
    // ---------------- clean the value rows of blocks that not every row sees whole
    const int fixer = warp - kSoftWarps - 2;
    Ring at;                     // the ring stage of the next block in turn
    uint32_t fix_par = 0;
    bool ok = true;
    for (int seg = 0; ok && w.next(P); ++seg) {
      // stages in front of value block 0: the leading key blocks; between two: a value and a key block, where there
      // still is one
      const int ahead = w.single ? 2 : 1, from = w.first_fix() - w.b0;
      at.step(min(ahead, w.nb));
      for (int j = 0; j < w.nb; ++j, at.step(j + ahead - 1 < w.nb ? 2 : 1)) {
        if (j < from) continue;
        const int s = at.s;
        // only once the copy has been asked for does the stage's phase stand at this use (these warps are there as soon as
        // they have cleaned what comes before, maybe a whole run ahead)
        const long long limit = kMbarWaitCycles + (LONG ? sm.run.start.left * kBlockCycles : 0);
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sm.to_fix[s], (fix_par >> s) & 1u, P.err, limit)))) break;
        fix_par ^= 1u << s;
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sm.full[s], at.par, P.err)))) break;
        const int k0 = (w.b0 + j) * kRows, seen = w.r.kv - k0;  // rows of the block that the request holds
        uint4* v = reinterpret_cast<uint4*>(sm.ring[s]);  // [16 groups][2][8 rows][8 pieces]
        bool found = false;
        for (int i = max(0, w.first_clean() - k0) * 16 + fixer * 32 + lane; i < kRows * 16; i += 64) {
          if ((i >> 7) * 8 + ((i >> 3) & 7) >= seen) {  // (the swizzle moves pieces inside a row only)
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            continue;
          }
          const uint4 x = v[i];
          if ((nonfinite2(x.x) | nonfinite2(x.y) | nonfinite2(x.z) | nonfinite2(x.w)) & 0x80008000u) {
            uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (nonfinite16(e[k])) e[k] &= 0xFFFF0000u;
              if (nonfinite16(e[k] >> 16)) e[k] &= 0x0000FFFFu;
            }
            v[i] = make_uint4(e[0], e[1], e[2], e[3]);
            found = true;
          }
        }
        if (found) *reinterpret_cast<volatile int*>(&sm.poison[seg & 7]) = seg + 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.fixed[s]);
      }
      w.advance();
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

size_t wi_paged_attention_scratch(int sms) {
  return kPagedTicketBytes + kSplitBytes + (size_t)sms * 2 * kPartBytes;
}

cudaError_t wi_launch_paged_attention(const WiPagedGeom& g, const WiPagedAttn& a, int sms, void* scratch, int* err,
                                      cudaStream_t st) {
  Params P;
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
      !wi_encode_pages_sw128(&map_k, a.k_pages, rows, (unsigned)P.box) ||
      !wi_encode_pages_sw128(&map_v, a.v_pages, rows, (unsigned)P.box))
    return cudaErrorInvalidValue;
  static int smem_set[2][kWiSmemDevices] = {};
  const bool is_long = (long long)g.max_pages * g.page > (long long)kLongest * kRows;
  auto* kernel = is_long ? k_paged_attention<true> : k_paged_attention<false>;
  cudaError_t e = wi_ensure_smem(kernel, sizeof(Smem), smem_set[is_long]);
  if (e != cudaSuccess) return e;
  const int grid = sms < kPagedMaxSms ? sms : kPagedMaxSms;
  if ((e = wi_launch_chained(kernel, dim3((unsigned)grid), kThreads, sizeof(Smem), st, map_q, map_k, map_v,
                             P)) != cudaSuccess)
    return e;
  if (here) return cudaSuccess;
  return wi_launch_chained(k_paged_merge, dim3((unsigned)grid, 2 * kRows / kMergeRows), kMergeThreads, 0, st, P);
}
