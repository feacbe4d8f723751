// Attention over packed prompts in the expanded form (smla_prompt_fwd):
//   o = softmax(sm_scale q K^T) V,  lse = ln sum exp(sm_scale q k)
// in one pass over the keys with a running maximum and sum.
//
// Rows are (token, query head of one key head) pairs: G heads that share a key head (the
// largest power of two that divides their number, at most 128) lie side by side, so that
// few tokens of many grouped heads still fill a tile. A block is 512 rows of one request
// and head group, worked on by a pair of CTAs in two row tiles of 256 rows, 128 in each CTA.
// K and V come in tiles of 128 keys that both row tiles use. While the softmax of one row
// tile runs, the tensor cores work for the other:  PV0(t) QK0(t+1) | PV1(t) QK1(t+1) | PV0(t+1) ...
//
// Why a pair. A 128 x 128 x 16 product of one CTA reads 8 KB of shared memory in the 64 cycles that it
// takes, all that shared memory gives, and the loads of K and V come on top (80 KB a tile pair, 640 cycles of
// 2,560: QK and PV measured 3,000-3,200 together). With cta_group::2 each CTA holds half of the keys of
// K and half of the values of V: 6 KB a product and half of the loads.
//
// Tensor memory (512 columns): S0 | S1 | O0 | O1, 128 fp32 columns each; P takes the
// place of its logits as bf16 (64 columns), as MMA operand A. Products of one tile are
// issued in order, so S(t+1) overwrites P(t) only after PV(t) has read it, and when S(t+1) is
// complete O holds everything up to t.
// Shared memory: Q of both tiles, and a ring of 8 KB slots (64 keys x 64 values of K; two slots for
// 128 keys x 64 values of V; 128-byte swizzled) that K and V tiles go through in turn.
// Warps of each CTA: 0 TMA loads (CTA 0: and the schedule), 1 MMA issue (CTA 1: tells CTA 0 what has
// arrived), 2-3 look V over (below), 4-7 and 8-11 softmax and results of the two row tiles, a
// thread a row.
//
// 0 * NaN. V rows that a row does not see meet its zero probabilities. Tiles that
// some row of the block sees only in part are looked over before they are used: values
// that are not finite are zeroed in shared memory, and the first key that holds +inf, -inf or
// NaN is noted for each of the 128 columns; rows that see it get it added to their result.
//
// The plan. A small kernel turns the requests' bounds into a list of blocks. Where blocks
// are many, pairs take them one by one, longest first, a few key heads at a time (so that
// their K and V stay in L2). Where the longest would end late (few rows, many keys), all
// tiles lie on one line that is cut into equal stretches, one per pair; blocks that are cut
// leave fp32 partial results, which join_kernel joins. No pair waits for another.
//
// Bound by the tensor pipe and, in long runs, by power where prompts are long: 16,384 tokens of 64 heads
// in 3.2-3.3 ms, 1,670-1,700 TFLOP/s (cuBLAS in long runs: 1,715; the first calls on a cool GPU 2.98 ms). Prompts of
// some thousand tokens wait for their softmax: a tile's chain is 1,500 cycles of softmax, 1,280 of products and 300 of
// hand-overs against 2,560 of products for both row tiles (8,192 tokens of 64 heads on 8: 669 us, 1,640
// TFLOP/s). Short ones, 37 prompts of up to 2,047 tokens: 1,094 us for a floor of 542, from products that the
// mask hides (row tiles of 256 against key tiles of 128: 1.3 to 1.4 times the definition's, some 730 us at the
// burst rate; 1.03 at 8,192 tokens) and from the starts and results of items, which the softmax warps do
// themselves (about 8,000 cycles an item against 15,000 of products). A few tokens on many keys cost as much tensor
// time as 256 rows would (5 x 3 tokens on 9K keys: 316 us, 4.7 TB/s; 244 us of products at the burst rate). 1 x 100
// tokens of 16 heads: 9.5 us, a chain of latencies.
#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>

#include "../../include/smla_prompt.h"
#include "prompt_layout.h"
#include "rows.cuh"

namespace smla {
namespace {

constexpr int kVal = kPromptVal;
constexpr int kPe = 64;
constexpr int kTile = 128;  // rows of a row tile in each CTA, keys of a key tile
constexpr int kBlock = kPromptRows;
static_assert(kBlock == 4 * kTile, "two row tiles of both CTAs");
constexpr int kQChunk = kTile * 128;  // bytes of 128 rows x 64 values
constexpr int kSlot = 64 * 128;       // of 64 keys x 64 values
constexpr int kAhead = 8;             // tiles of the ring at most, and barriers for them
constexpr int kThreads = 384;
constexpr int kTmaWarp = 0, kMmaWarp = 1, kScanWarp0 = 2, kSoftWarp0 = 4;
constexpr float kRaise = 8.0f;  // log2: the reference maximum is raised only when exceeded by this much
constexpr int kStart = 2;       // a piece's start and end on the line of work, in tiles (1, 2 and 5: within 2%)
// Blocks of no more tiles are never cut, and calls of no more keys have no join to launch. With 4 / 8 / 16 tiles, us on the
// device: 7 x 100 tokens of 8 heads 16.3 / 10.9 / 10.9, one token on 1,000 keys of 16 heads 20.3 / 16.2 / 16.0, on 2,048 keys
// 21.9 / 23.4 / 22.6 (64 heads: 31 / 31 / 24), 300 tokens on 4,000 keys of 4 heads 32 with each.
constexpr int kLongTiles = 8;
constexpr int kDirectSeqs = 8;  // requests that a thread looks through (8 x 20 tokens of 8 heads: 10.7 us, 14.4 with a plan)
constexpr uint32_t kColS = 0, kColO = 256;

struct PromptParams {
  int32_t total_q, total_k, n_seqs;
  const int32_t *cu_q, *cu_k;
  int32_t n_heads, group, causal;
  int32_t gshift;     // G = 1 << gshift heads of a row tile's tokens
  int32_t units;      // head groups: n_heads >> gshift
  int32_t units_a;    // of those that are worked on at a time
  int32_t d_k;        // values of k (the others of a key are k_pe's)
  int32_t max_blocks, pairs, can_cut;
  int32_t direct;     // no plan: every pair has one block at most and finds it itself
  float scale_log2;   // sm_scale log2 e, not 0
  const float *prev_out, *prev_lse;
  void* out;
  int32_t out_fp32, out_sectors;  // fp32; on a 32-byte boundary
  float* lse;
  uint32_t* status;
  Plan* plan;
  Block* blocks;
  Block* sorted;        // longest first
  long long* line_at;   // where each block starts on the line
  int32_t* block_at;    // first block of each request
  Cut* cuts;            // [pairs]
  float2* part_ml;      // [2 * pairs][512]
  float4* part_o;       // [2 * pairs][512][32], on a 32-byte boundary
};

// ------------------------------------------------------------------ the plan
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ long long plan_scan(long long v, long long* warp_sums, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  long long w = warp_sums[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xFFFFFFFFu, w, d);
    if (lane >= d) w += o;
  }
  total = __shfl_sync(0xFFFFFFFFu, w, 31);
  const long long before = __shfl_sync(0xFFFFFFFFu, w, (warp + 31) & 31);
  return v + (warp ? before : 0);
}

// The bounds of a request: tokens q0 .. q0 + nq - 1, keys k0 .. k0 + nk - 1; false where they run
// backwards or leave the tensors.
struct Request {
  int32_t q0, nq, k0, nk;
};
__device__ __forceinline__ bool request_of(const PromptParams& p, int b, Request& r) {
  const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], k0 = p.cu_k[b], k1 = p.cu_k[b + 1];
  r = Request{q0, q1 - q0, k0, k1 - k0};
  return q0 >= 0 && q1 >= q0 && q1 <= p.total_q && k0 >= 0 && k1 >= k0 && k1 <= p.total_k;
}
// The block of a request that begins with its token i0.
__device__ __forceinline__ Block block_of(const PromptParams& p, const Request& r, int i0, int per) {
  Block k;
  k.tok0 = r.q0 + i0;
  k.n_tok = min(per, r.nq - i0);
  k.key0 = r.k0;
  k.lim0 = p.causal ? r.nk - r.nq + i0 + 1 : r.nk;
  k.n_keys = p.causal ? max(0, k.lim0 + k.n_tok - 1) : r.nk;
  k.tiles = max(1, static_cast<int>((static_cast<uint32_t>(k.n_keys) + kTile - 1) / kTile));
  k.pad[0] = k.pad[1] = 0;
  return k;
}

// One block of threads: requests -> blocks -> longest first, and whether the line is cut. Bound by latency: a few
// scans and loads that depend on one another, 5 us of a small call.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PromptParams p) {
  __shared__ long long warp_sums[32];
  __shared__ int bins[1024];
  __shared__ int s_most, s_bad;
  __shared__ long long s_bound;
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;");  // prompt_kernel may set up
  if (tid == 0) s_most = 1, s_bad = 0, s_bound = 0;
  for (int i = tid; i < 1024; i += kPlanThreads) bins[i] = 0;
  for (int i = tid; i < p.pairs; i += kPlanThreads) p.cuts[i] = Cut{0, 0, 0, 0};
  const int per = kBlock >> p.gshift;  // tokens of a block
  // blocks of each request
  long long before = 0;
  bool bad = false;
  for (int c0 = 0; c0 < p.n_seqs; c0 += kPlanThreads) {
    const int b = c0 + tid;
    int n = 0;
    if (b < p.n_seqs) {
      Request r;
      if (request_of(p, b, r)) n = (r.nq + per - 1) / per;
      else bad = true;
    }
    long long total;
    const long long upto = before + plan_scan(n, warp_sums, total);
    if (b < p.n_seqs) {  // (bounds that overlap can make more blocks than there is room for)
      if (upto > p.max_blocks) bad = true;
      p.block_at[b] = static_cast<int>(min(upto - n, static_cast<long long>(p.max_blocks)));
    }
    before += total;
  }
  if (bad) s_bad = 1;
  const int n_blocks = static_cast<int>(min(before, static_cast<long long>(p.max_blocks)));
  if (tid == 0) p.block_at[p.n_seqs] = n_blocks;
  __syncthreads();
  // the blocks, and where each lies on the line
  long long line = 0;
  for (int c0 = 0; c0 < n_blocks; c0 += kPlanThreads) {
    const int i = c0 + tid;
    long long cost = 0;
    if (i < n_blocks) {
      int lo = 0, hi = p.n_seqs;  // block_at[lo] <= i < block_at[hi], empty requests passed over
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.block_at[mid] <= i) lo = mid; else hi = mid;
      }
      Request r;
      request_of(p, lo, r);
      const Block k = block_of(p, r, (i - p.block_at[lo]) * per, per);
      p.blocks[i] = k;
      atomicMax(&s_most, k.tiles);
      cost = static_cast<long long>(k.tiles + kStart) * p.units;
    }
    long long total;
    const long long upto = line + plan_scan(cost, warp_sums, total);
    if (i < n_blocks) p.line_at[i] = upto - cost;
    line += total;
  }
  __syncthreads();
  // longest first, by bins of tiles
  int shift = 0;
  while ((s_most >> shift) >= 1024) ++shift;
  for (int i = tid; i < n_blocks; i += kPlanThreads) atomicAdd(&bins[1023 - (p.blocks[i].tiles >> shift)], 1);
  __syncthreads();
  const int count = bins[tid];
  const long long t = (static_cast<long long>(1023 - tid) << shift) + (shift ? (1 << shift) - 1 : 0) + kStart;  // of the bin's longest
  long long all;
  const long long first = plan_scan(count, warp_sums, all) - count;
  // Taken one by one in this order, an item ends by (work before it) / pairs + its own: the
  // last of a bin's is the latest of the bin.
  const long long work = plan_scan(t * count * p.units, warp_sums, all);
  if (count > 0) atomicMax(reinterpret_cast<unsigned long long*>(&s_bound), static_cast<unsigned long long>((work - t) / p.pairs + t));
  __syncthreads();
  bins[tid] = static_cast<int>(first);
  __syncthreads();
  // (the order within a bin decides only which pair takes a block)
  for (int i = tid; i < n_blocks; i += kPlanThreads) p.sorted[atomicAdd(&bins[1023 - (p.blocks[i].tiles >> shift)], 1)] = p.blocks[i];
  if (tid == 0) {
    const long long even = line / p.pairs;
    p.plan->next = 0;
    p.plan->line = line;
    p.plan->n_blocks = n_blocks;
    // Cut evenly where whole blocks would end a tenth and six tiles later: pieces cost a start and a join each, and blocks
    // in a row on one line do not share K and V in L2. Never / by this rule / always, us: 5 x 3 tokens on 9K keys 346 / 296 /
    // 296, 300 tokens on 4,000 keys of 4 heads 62 / 32 / 32, 4,096 tokens of 16 heads 93 / 83 / 83, 37 ragged prompts of 64
    // heads 950 / 952 / 1,035; 2,048 tokens of 16 heads 40 / 44 / 44 and 8,192 of 16 heads 262 / 263 / 224 on the wrong side.
    p.plan->even = p.can_cut && s_most > kLongTiles && s_bound > even + even / 10 + 6;
    p.plan->pairs = static_cast<int>(max(1LL, min(static_cast<long long>(p.pairs), line / 4)));
    *p.status = s_bad ? kStatusBounds : 0u;
  }
}

// ------------------------------------------------------------------ waits, TMA, MMA
__device__ __forceinline__ bool try_bar(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Gives up after kWaitLimitCycles, or when another role has: false, and *abort is raised
// (the end of the kernel reports it). The loops are functions of their own: in line at every
// wait they made the kernel too long for the instruction cache. One thread:
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort) {
  const long long t0 = clock64();
  for (uint32_t it = 1; !try_bar(bar, parity); ++it) {
    if ((it & 63u) != 0) continue;
    if (*abort || clock64() - t0 > kWaitLimitCycles) {
      *abort = 2;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint32_t a = smem_u32(bar);
  return try_bar(a, parity) || wait_on(a, parity, abort);
}
// The same by a whole warp: every lane sees the phase, all leave together.
__device__ __noinline__ bool wait_on_warp(uint32_t bar, uint32_t parity, volatile int* abort) {
  const long long t0 = clock64();
  for (uint32_t it = 1; !__all_sync(0xFFFFFFFFu, try_bar(bar, parity)); ++it) {
    if ((it & 63u) != 0) continue;
    if (__any_sync(0xFFFFFFFFu, *abort != 0 || clock64() - t0 > kWaitLimitCycles)) {
      *abort = 2;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint32_t a = smem_u32(bar);
  return __all_sync(0xFFFFFFFFu, try_bar(a, parity)) || wait_on_warp(a, parity, abort);
}
// The same without a call, for the softmax warps (a call would move their values to local memory).
__device__ __forceinline__ bool wait_here(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint32_t a = smem_u32(bar);
  long long t0 = 0;
  for (uint32_t it = 1; !__all_sync(0xFFFFFFFFu, try_bar(a, parity)); ++it) {
    if ((it & 255u) != 0) continue;
    if (t0 == 0) t0 = clock64();
    if (__any_sync(0xFFFFFFFFu, *abort != 0 || clock64() - t0 > kWaitLimitCycles)) {
      *abort = 2;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t addr_in(uint32_t saddr, uint32_t rank) {  // the same place in CTA `rank` of the pair
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Arrivals across the pair speak of tensor memory and of TMA's bytes, not of what this thread wrote to memory:
// they carry no release at cluster scope, which waits for the warp's memory operations (1,000
// cycles a tile at the end of the softmax). Where memory was written for the other CTA, cluster_fence comes first.
__device__ __forceinline__ void arrive_in(uint64_t* bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr_in(smem_u32(bar), rank)) : "memory");
}
__device__ __forceinline__ void cluster_fence() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }
__device__ __forceinline__ void store_in(const void* at, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr_in(smem_u32(at), rank)), "r"(v) : "memory");
}
// Counters in shared memory that only grow, in both CTAs: a waiter may lag behind by any number of steps.
__device__ __forceinline__ void count_up(uint32_t* counter) {  // one thread
#pragma unroll
  for (uint32_t r = 0; r < 2; ++r)
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], 1;" ::"r"(addr_in(smem_u32(counter), r)) : "memory");
}
__device__ __forceinline__ bool wait_count(const uint32_t* counter, uint32_t n, volatile int* abort) {  // a whole warp
  auto there = [&] {
    uint32_t v;
    asm volatile("ld.relaxed.cluster.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(smem_u32(counter)) : "memory");
    return __all_sync(0xFFFFFFFFu, static_cast<int32_t>(v - n) >= 0);
  };
  long long t0 = 0;
  for (uint32_t it = 1; !there(); ++it) {
    if ((it & 255u) != 0) continue;
    if (t0 == 0) t0 = clock64();
    if (__any_sync(0xFFFFFFFFu, *abort != 0 || clock64() - t0 > kWaitLimitCycles)) {
      *abort = 2;
      return false;
    }
  }
  return true;
}
template <typename M>
__device__ __forceinline__ bool wait_scanned(const M& m, uint32_t n, volatile int* abort) {
  // all four at a look; one after the other where that does not do
  uint32_t a, b, c, d;
  asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(smem_u32(m.scanned)) : "memory");
  bool ok = true;
  if (!__all_sync(0xFFFFFFFFu, min(min(static_cast<int32_t>(a - n), static_cast<int32_t>(b - n)), min(static_cast<int32_t>(c - n), static_cast<int32_t>(d - n))) >= 0))
#pragma unroll 1
    for (int i = 0; ok && i < 4; ++i) ok = wait_count(&m.scanned[i], n, abort);
  return ok;
}
// true in one thread of the (converged) warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// Shared-memory operand of an MMA: the low word of its descriptor holds the address
// (in 16 bytes), the high word is the same wherever the operand starts.
struct Operand {
  uint32_t lo, hi;
  __device__ __forceinline__ Operand operator+(int bytes) const { return {lo + static_cast<uint32_t>(bytes >> 4), hi}; }
};
__device__ __forceinline__ Operand operand(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  const uint64_t d = smem_desc(saddr, lbo, sbo);
  return {static_cast<uint32_t>(d), static_cast<uint32_t>(d >> 32)};
}
// A from tensor memory
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, Operand b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A from shared memory
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, Operand a, Operand b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %6, 0;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// arrives on the barrier at this address in both CTAs when the products issued so far are done
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\t"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {  // relative error about 2^-22; 2^-inf = 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// ------------------------------------------------------------------ items
struct Item {        // tiles [t0, t1) of a block and head group; t1 = 0: no more
  int32_t tok0, n_tok, key0, lim0, n_keys, t0, t1;
  int32_t unit;
  int32_t whole;     // all tiles of the block
  int32_t slot;      // where its partial results go
};
// Tiles that row tile x takes part in: [t0, end), none where end <= t0. (Both CTAs alike.)
__device__ __forceinline__ int tokens_of(const PromptParams& p, const Item& it, int x) {
  return min(it.n_tok - x * (2 * kTile >> p.gshift), 2 * kTile >> p.gshift);
}
__device__ __forceinline__ int seen_by(const PromptParams& p, const Item& it, int token) {  // keys that a token of the block sees
  return p.causal ? max(0, it.lim0 + token) : it.n_keys;
}
// A block of one row tile: its key tiles go to both halves of the pipeline in turn, which hold the
// same rows and are joined at the end. (One row tile alone leaves the tensor cores waiting for its softmax:
// 5 x 3 tokens of 64 heads on 9K keys, 531 us, against 322 with both halves at work.)
__device__ __forceinline__ bool two_halves(const PromptParams& p, const Item& it) { return tokens_of(p, it, 1) <= 0 && it.t1 - it.t0 >= 2; }
__device__ __forceinline__ int end_of(const PromptParams& p, const Item& it, int x) {
  if (two_halves(p, it)) return it.t1;
  const int n = tokens_of(p, it, x);
  if (n <= 0) return 0;
  const int seen = seen_by(p, it, x * (2 * kTile >> p.gshift) + n - 1);
  return min(it.t1, max(1, static_cast<int>((static_cast<uint32_t>(seen) + kTile - 1) / kTile)));
}

#define SMLA_W4(i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      SMLA_W4(0), SMLA_W4(4), SMLA_W4(8), SMLA_W4(12)
      : "memory");
}
#undef SMLA_W4

template <int D>
struct Sizes {
  static constexpr int kChunks = D / 64;                // of a row of q or k
  static constexpr int kSlots = D == 192 ? 16 : 20;
  static constexpr int kQTile = kChunks * kQChunk;
  static constexpr int kOffRing = 2 * kQTile, kOffMeta = kOffRing + kSlots * kSlot;
};
// Ring positions: K takes kChunks slots, each for itself; V two that lie next to each
// other (its tile is one operand), so it passes over the ring's last slot.
template <int D>
__device__ __forceinline__ int after_k(int pos) {
  pos += Sizes<D>::kChunks;
  if (pos >= Sizes<D>::kSlots) pos -= Sizes<D>::kSlots;
  return pos == Sizes<D>::kSlots - 1 ? 0 : pos;  // where V goes
}
template <int D>
__device__ __forceinline__ int after_v(int pos) {
  pos += 2;
  return pos >= Sizes<D>::kSlots ? pos - Sizes<D>::kSlots : pos;
}

struct Meta {
  Item items[2];
  uint64_t item_full[2], item_free[2];
  uint64_t q_full[2], q_free[2], s_full[2], p_half[2], p_full[2], o_full[2];
  uint64_t ml_full, ml_free;
  uint64_t k_full[kAhead], v_full[kAhead], v_ok[kAhead];
  uint64_t slot_free[20];
  int odd[2][kVal];     // first key whose value in this column is +inf or NaN, -inf or NaN; noted by the CTA that has the column
  uint32_t odd_item[2]; // the item (from 1 on) that they are of, for each CTA's columns
  uint32_t odd_lock;
  alignas(16) uint32_t scanned[4];  // V tiles that each of the four warps has looked over
  uint32_t ended;       // warps (of both CTAs) that are done with what was noted for an item
  uint32_t tmem_slot, status;
  int abort_flag;
  float2 ml[kTile];     // maximum and sum of the second row tile's half of the keys (two_halves)
};
template <int D>
constexpr size_t kSmemBytes = Sizes<D>::kOffMeta + sizeof(Meta);
static_assert(kSmemBytes<192> <= 232448 && kSmemBytes<128> <= 232448, "shared memory budget");

// Values that are not finite in the rows of this CTA's half of a V tile that `hit` names (bit i: row
// 8 i + 4 mine + lane / 8): zeroed, and where some row of the block sees them noted in both CTAs.
__device__ __noinline__ bool note_odd(Meta& M, uint8_t* tile, uint32_t hit, int mine, uint32_t rank, uint32_t n, int key0, int all_see,
                                      int n_keys, volatile int* abort) {
  const int lane = threadIdx.x & 31;
  // The results of the items before are out: what was noted for them goes, once.
  if (!wait_count(&M.ended, 16 * (n - 1), abort)) return false;
  if (lane == 0)
    for (uint32_t i = 0; atomicCAS(&M.odd_lock, 0u, 1u) != 0 && i < (1u << 24); ++i) __nanosleep(32);
  __syncwarp();
  if (*const_cast<volatile uint32_t*>(&M.odd_item[rank]) != n) {
    for (int i = lane; i < 2 * 64; i += 32)
      for (uint32_t r = 0; r < 2; ++r) store_in(&M.odd[i >> 6][64 * rank + (i & 63)], r, INT_MAX);
    __syncwarp();
    if (lane == 0) {
      cluster_fence();
      for (uint32_t r = 0; r < 2; ++r) store_in(&M.odd_item[rank], r, n);
    }
  }
  cluster_fence();
  __syncwarp();
  if (lane == 0) atomicExch(&M.odd_lock, 0u);
  for (; hit; hit &= hit - 1) {
    const int r = 8 * (__ffs(hit) - 1) + 4 * mine + (lane >> 3), key = key0 + r;
    if (key < all_see) continue;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      uint16_t* v = reinterpret_cast<uint16_t*>(tile + r * 128 + (lane & 7) * 16) + i;
      const uint16_t w = *v;
      if ((w & 0x7F80u) != 0x7F80u) continue;
      *v = 0;
      const int col = 64 * rank + 8 * ((lane & 7) ^ (r & 7)) + i;
      if (key < n_keys)
        for (uint32_t c = 0; c < 4; ++c)
          if (w != ((c & 1) ? 0x7F80u : 0xFF80u))  // a NaN counts as both
            asm volatile("red.relaxed.cluster.shared::cluster.min.s32 [%0], %1;" ::"r"(addr_in(smem_u32(&M.odd[c & 1][col]), c >> 1)), "r"(key) : "memory");
    }
  }
  cluster_fence();  // before the counters and barriers that say so
  __syncwarp();
  return true;
}

// ------------------------------------------------------------------ results
// 32 bytes, a whole sector, at once where they lie on a 32-byte boundary
__device__ __forceinline__ void store8(float* p, const float* v, bool sector) {
  if (sector) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
                 "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}
__device__ __forceinline__ void load8(const float* p, float* v) {  // (no .nc: it may be the output)
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
struct Joined {  // how a row's sum goes into its result: out = own * f + prev_out * fp (fp -1: nothing of prev_out)
  float f, fp, lse;
};
__device__ __noinline__ void join_with(float was, float l, Joined& j) {
  if (was == -INFINITY) return;
  const float top = fmaxf(was, j.lse);
  const float both = l != 0.0f ? top + logf(expf(was - top) + expf(j.lse - top)) : was;
  j.f *= expf(j.lse - both);
  j.fp = expf(was - both);
  j.lse = both;
}
__device__ __forceinline__ Joined join_prev(const PromptParams& p, long long flat, float m, float l) {
  Joined j;
  j.f = l != 0.0f ? 1.0f / l : 0.0f;
  j.fp = -1.0f;
  j.lse = l != 0.0f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
  if (p.prev_lse) join_with(p.prev_lse[flat], l, j);
  return j;
}
__device__ __forceinline__ void add_prev(const PromptParams& p, long long at, float f, float* v) {
  float was[16];
  load8(p.prev_out + at, was);
  load8(p.prev_out + at + 8, was + 8);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] += f * was[i];
}
// What a row that sees `seen` keys gets in a column from values that are not finite: added to its
// finite sum, +inf, -inf or NaN; 0: nothing.
__device__ __forceinline__ float odd_of(const Meta& M, uint32_t item, int col, int seen) {
  if (M.odd_item[col >> 6] != item) return 0.0f;
  const bool up = M.odd[0][col] < seen, down = M.odd[1][col] < seen;
  return up && down ? NAN : up ? INFINITY : down ? -INFINITY : 0.0f;
}
__device__ __forceinline__ void store4(const PromptParams& p, long long flat, int col, float4 v) {
  const long long at = flat * kVal + col;
  if (p.out_fp32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = v;
  else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = make_uint2(bf_pack(v.x, v.y), bf_pack(v.z, v.w));
}

template <int D, bool NEG>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap pe_map, const PromptParams p) {
  using Z = Sizes<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Meta& M = *reinterpret_cast<Meta*>(smem + Z::kOffMeta);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const bool aligned = (smem_u32(smem) & 1023u) == 0;  // (alike in both CTAs)
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&M.item_full[i], 1);
      mbar_init(&M.item_free[i], 11 + 12);  // in CTA 0: the warps of both but its own that writes
      mbar_init(&M.q_full[i], rank == 0 ? 2 : 1);
      mbar_init(&M.q_free[i], 1);
      mbar_init(&M.s_full[i], 1);
      mbar_init(&M.p_half[i], 8);
      mbar_init(&M.p_full[i], 8);
      mbar_init(&M.o_full[i], 1);
    }
    for (int i = 0; i < kAhead; ++i) {
      mbar_init(&M.k_full[i], rank == 0 ? 2 : 1);  // CTA 0's: its own half, and the other's is there
      mbar_init(&M.v_full[i], 1);
      mbar_init(&M.v_ok[i], 4);
    }
    for (int i = 0; i < Z::kSlots; ++i) mbar_init(&M.slot_free[i], 1);
    mbar_init(&M.ml_full, 4);
    mbar_init(&M.ml_free, 4);
    M.odd_item[0] = M.odd_item[1] = M.odd_lock = M.ended = 0;
    for (int i = 0; i < 4; ++i) M.scanned[i] = 0;
    M.abort_flag = aligned ? 0 : 2;
    M.status = aligned ? 0 : kStatusSetup;
    fence_mbar_init();
  }
  for (int i = tid; i < 2 * kVal; i += kThreads) (&M.odd[0][0])[i] = INT_MAX;
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&M.tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    prefetch_tensormap(&q_map);
    prefetch_tensormap(&k_map);
    prefetch_tensormap(&v_map);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's barriers are set up before either CTA signals the other
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan
  const uint32_t tmem = M.tmem_slot;
  const uint32_t sbase = smem_u32(smem);
  volatile int* abort_v = &M.abort_flag;

  // 168 registers a thread at launch, for three warpgroups: 88 + 2 x 208 of them are used. The
  // softmax threads hold a row's 128 logits.
  if (!aligned) {
    // nothing: the status says so
  } else if (warp < kSoftWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == kTmaWarp) {
      // -------------------------------------------------------------- schedule and TMA loads
      if (lane == 0) {
        const Plan plan = p.direct ? Plan{} : *p.plan;
        const int pair = blockIdx.x >> 1;
        const long long items = static_cast<long long>(plan.n_blocks) * p.units;
        // even: this pair's stretch [x, y) of the line and where it stands
        long long x = 0, y = 0, at = 0;
        int blk = 0, unit = 0;
        if (plan.even && pair < plan.pairs) {
          x = plan.line * pair / plan.pairs;
          y = plan.line * (pair + 1) / plan.pairs;
          int hi = plan.n_blocks;
          while (hi - blk > 1) {
            const int mid = (blk + hi) >> 1;
            if (p.line_at[mid] <= x) blk = mid; else hi = mid;
          }
          const int cost = p.blocks[blk].tiles + kStart;
          unit = static_cast<int>((x - p.line_at[blk]) / cost);
          at = p.line_at[blk] + static_cast<long long>(unit) * cost;
        }
        auto pair_of = [&](long long pos) {  // that has this place of the line
          return static_cast<int>(((pos + 1) * plan.pairs + plan.line - 1) / plan.line) - 1;
        };
        bool found = false;  // direct: this pair's block has been looked for
        auto next = [&](Item& it) {
          if (p.direct) {
            if (found) return false;
            found = true;
            const int per = kBlock >> p.gshift, u = pair % p.units;
            int want = pair / p.units;
            bool have = false, bad = false;
            for (int b = 0; b < p.n_seqs; ++b) {
              Request r;
              if (!request_of(p, b, r)) {
                bad = true;
                continue;
              }
              const int n = (r.nq + per - 1) / per;
              if (!have && want < n) {
                const Block k = block_of(p, r, want * per, per);
                it = Item{k.tok0, k.n_tok, k.key0, k.lim0, k.n_keys, 0, k.tiles, u, 1, 0};
                have = true;
              }
              want -= n;
              if (have && pair > 0) break;
            }
            bad |= -want > p.max_blocks;  // (pair 0: bounds that overlap can make more blocks than there are pairs for)
            if (pair == 0) *p.status = bad ? kStatusBounds : 0u;  // (what other CTAs report comes seconds later)
            return have;
          }
          if (plan.even) {
            while (at < y) {
              const Block b = p.blocks[blk];
              const long long from = at + kStart;
              const int t0 = static_cast<int>(min(max(x - from, 0LL), static_cast<long long>(b.tiles)));
              const int t1 = static_cast<int>(min(max(y - from, 0LL), static_cast<long long>(b.tiles)));
              const int u = unit;
              at += b.tiles + kStart;
              if (++unit == p.units) unit = 0, ++blk;
              if (t1 <= t0) continue;
              it = Item{b.tok0, b.n_tok, b.key0, b.lim0, b.n_keys, t0, t1, u, t0 == 0 && t1 == b.tiles, 2 * pair + (t0 == 0)};
              if (t0 == 0 && !it.whole)  // (a pair has one such piece at most, its last)
                p.cuts[pair] = Cut{b.tok0, b.n_tok, u, pair_of(from + b.tiles - 1) - pair + 1};
              return true;
            }
            return false;
          }
          const long long i = static_cast<long long>(atomicAdd(&p.plan->next, 1ULL));
          if (i >= items) return false;
          const long long per = static_cast<long long>(plan.n_blocks) * p.units_a;
          const int g = static_cast<int>(i / per), u0 = g * p.units_a, n = min(p.units_a, p.units - u0);
          const long long r = i - g * per;
          const int place = static_cast<int>(r / n);
          const Block b = p.sorted[place];
          it = Item{b.tok0, b.n_tok, b.key0, b.lim0, b.n_keys, 0, b.tiles, u0 + static_cast<int>(r - static_cast<long long>(place) * n), 1, 0};
          return true;
        };
        uint32_t n = 0, kg = 0, vg = 0, used = 0;  // items, K tiles, V tiles, parity of each slot's use
        uint32_t nq[2] = {0, 0};
        int pos = 0;
        bool ok = true, more = true;
        auto take_slot = [&](int s) {
          const bool got = wait_one(&M.slot_free[s], ((used >> s) & 1u) ^ 1u, abort_v);
          used ^= 1u << s;
          return got;
        };
        Item it{}, after{};  // the next item is looked up while this one's first loads are under way
        if (rank == 0) more = next(after);
        while (ok) {
          if (rank == 0) {
            it = more ? after : Item{};
            if (n >= 2 && !wait_one(&M.item_free[n & 1], ((n >> 1) - 1) & 1, abort_v)) break;
            for (uint32_t r = 0; r < 2; ++r) {
#pragma unroll
              for (uint32_t i = 0; i < sizeof(Item) / 4; ++i) store_in(reinterpret_cast<uint32_t*>(&M.items[n & 1]) + i, r, reinterpret_cast<uint32_t*>(&it)[i]);
              cluster_fence();
              arrive_in(&M.item_full[n & 1], r);
            }
          } else {
            if (!wait_one(&M.item_full[n & 1], (n >> 1) & 1, abort_v)) break;
            it = M.items[n & 1];
            arrive_in(&M.item_free[n & 1], 0);
          }
          ++n;
          if (it.t1 == 0) break;
          const int kv_head = static_cast<int>((static_cast<long long>(it.unit) << p.gshift) / p.group);
          auto load_q = [&](int x) {
            if (end_of(p, it, x) <= it.t0) return true;
            if (nq[x] > 0 && !wait_one(&M.q_free[x], (nq[x] - 1) & 1, abort_v)) return false;
            ++nq[x];
            mbar_arrive_expect_tx(&M.q_full[x], Z::kQTile);
            const int token = it.tok0 + ((two_halves(p, it) ? 0 : 2 * x) + static_cast<int>(rank)) * (kTile >> p.gshift);
#pragma unroll 1
            for (int c = 0; c < Z::kChunks; ++c)
              tma_box(smem + x * Z::kQTile + c * kQChunk, &q_map, &M.q_full[x], 64 * c, it.unit << p.gshift, token);
            return true;
          };
          for (int t = it.t0; ok && t < it.t1; ++t) {
            if (t == it.t0 && !load_q(0)) { ok = false; break; }
            const int key = it.key0 + t * kTile;
            uint64_t* k_bar = &M.k_full[kg++ & (kAhead - 1)];
#pragma unroll
            for (int c = 0; c < Z::kChunks; ++c) {
              ok = ok && take_slot(pos);
              if (!ok) break;
              if (c == 0) mbar_arrive_expect_tx(k_bar, Z::kChunks * kSlot);
              const bool shared = 64 * c >= p.d_k;
              tma_box(smem + Z::kOffRing + pos * kSlot, shared ? &pe_map : &k_map, k_bar, shared ? 0 : 64 * c, shared ? 0 : kv_head, key + 64 * static_cast<int>(rank));
              if (++pos == Z::kSlots) pos = 0;
            }
            ok = ok && (t != it.t0 || load_q(1));
            uint64_t* v_bar = &M.v_full[vg++ & (kAhead - 1)];
            if (pos == Z::kSlots - 1) pos = 0;
            ok = ok && take_slot(pos) && take_slot(pos + 1);
            if (!ok) break;
            mbar_arrive_expect_tx(v_bar, 2 * kSlot);
            tma_box(smem + Z::kOffRing + pos * kSlot, &v_map, v_bar, 64 * static_cast<int>(rank), kv_head, key);
            pos = after_v<D>(pos);
            if (rank == 0 && t == it.t0) more = next(after);
          }
        }
      }
    } else if (warp == kMmaWarp && rank == 1) {
      // -------------------------------------------------------------- what has arrived here, told to CTA 0
      uint32_t n = 0, kg = 0;
      uint32_t nq[2] = {0, 0};
      bool ok = true;
      while (ok) {
        if (!wait_warp(&M.item_full[n & 1], (n >> 1) & 1, abort_v)) break;
        const Item it = M.items[n & 1];
        __syncwarp();
        if (lane == 0) arrive_in(&M.item_free[n & 1], 0);
        ++n;
        if (it.t1 == 0) break;
        auto tell_q = [&](int x) {
          if (end_of(p, it, x) <= it.t0) return true;
          if (!wait_warp(&M.q_full[x], nq[x] & 1, abort_v)) return false;
          ++nq[x];
          if (lane == 0) arrive_in(&M.q_full[x], 0);
          return true;
        };
        ok = tell_q(0);
        for (int t = it.t0; ok && t < it.t1; ++t) {
          ok = wait_warp(&M.k_full[kg & (kAhead - 1)], (kg / kAhead) & 1, abort_v);
          if (!ok) break;
          if (lane == 0) arrive_in(&M.k_full[kg & (kAhead - 1)], 0);
          ++kg;
          if (t == it.t0) ok = tell_q(1);
        }
      }
    } else if (warp == kMmaWarp) {
      // -------------------------------------------------------------- MMA issue
      // Warp-wide on warp-uniform values, each batch of MMAs unrolled and issued by one
      // elected thread: descriptors come from uniform registers.
      constexpr uint32_t id_qk = instr_desc(256, 128, kFmtBF16, kFmtBF16, false, false);
      constexpr uint32_t id_pv = instr_desc(256, 128, kFmtBF16, kFmtBF16, false, true);
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      const uint32_t sb = __shfl_sync(0xFFFFFFFFu, sbase, 0);
      const Operand q_desc = operand(sb, 16, 1024);
      const Operand k_desc = operand(sb + Z::kOffRing, 16, 1024);
      const Operand v_desc = operand(sb + Z::kOffRing, 2 * kSlot, 1024);  // read as values x keys
      uint32_t n = 0, kg = 0, vg = 0;
      uint32_t nq[2] = {0, 0}, ns[2] = {0, 0};  // row tiles begun, P tiles used
      int pos = 0;
      bool ok = true;
      auto qk = [&](int x, int kpos, bool last) {
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < Z::kChunks; ++c) {
            const int s = kpos + c >= Z::kSlots ? kpos + c - Z::kSlots : kpos + c;
            const Operand k = k_desc + s * kSlot;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ss(tm + kColS + kTile * x, q_desc + (x * Z::kQTile + c * kQChunk + 32 * kk), k + 32 * kk, id_qk, c != 0 || kk != 0);
          }
          commit_pair(&M.s_full[x]);
          if (last) commit_pair(&M.q_free[x]);
        }
        __syncwarp();
      };
      auto pv = [&](int x, int vpos, int k0, bool first, bool last) {  // four steps of 16 keys from step k0 on
        tc_fence_after();
        if (elect_one()) {
          const Operand v = v_desc + vpos * kSlot;
#pragma unroll
          for (int kk = k0; kk < k0 + 4; ++kk)
            mma_ts(tm + kColO + kVal * x, tm + kColS + kTile * x + 8 * kk, v + 2048 * kk, id_pv, kk != 0 || !first);
          if (last) commit_pair(&M.o_full[x]);
        }
        __syncwarp();
      };
      // slots whose products are all issued: V's two (vpos >= 0), K's
      auto free_slots = [&](int vpos, int kpos, bool k) {
        if (elect_one()) {
          if (vpos >= 0) {
            commit_pair(&M.slot_free[vpos]);
            commit_pair(&M.slot_free[vpos + 1]);
          }
          if (k)
#pragma unroll
            for (int c = 0; c < Z::kChunks; ++c) commit_pair(&M.slot_free[kpos + c >= Z::kSlots ? kpos + c - Z::kSlots : kpos + c]);
        }
        __syncwarp();
      };
      while (ok) {
        if (!wait_warp(&M.item_full[n & 1], (n >> 1) & 1, abort_v)) { ok = false; break; }
        const Item it = M.items[n & 1];
        __syncwarp();
        if (lane == 0) arrive_in(&M.item_free[n & 1], 0);
        ++n;
        if (it.t1 == 0) break;
        const int t0 = __shfl_sync(0xFFFFFFFFu, it.t0, 0), t1 = __shfl_sync(0xFFFFFFFFu, it.t1, 0);
        const int end[2] = {__shfl_sync(0xFFFFFFFFu, end_of(p, it, 0), 0), __shfl_sync(0xFFFFFFFFu, end_of(p, it, 1), 0)};
        int kpos = pos;
        if (__shfl_sync(0xFFFFFFFFu, two_halves(p, it), 0)) {
          // QK0(t0) QK1(t0+1) | PV0(t0) QK0(t0+2) | PV1(t0+1) QK1(t0+3) ...
          int kn = kpos;  // where the next K tile is
#pragma unroll 1
          for (int t = t0 - 2; ok && t < t1; ++t) {
            const int x = (t - t0) & 1;
            if (t >= t0) {
              const int vpos = after_k<D>(kpos);
              kpos = after_v<D>(vpos);
              ok = wait_warp(&M.v_ok[vg & (kAhead - 1)], (vg / kAhead) & 1, abort_v) && wait_warp(&M.p_half[x], ns[x] & 1, abort_v);
              ++vg;
              if (!ok) break;
              pv(x, vpos, 0, t < t0 + 2, false);
              ok = wait_warp(&M.p_full[x], ns[x] & 1, abort_v);
              ++ns[x];
              if (!ok) break;
              pv(x, vpos, 4, false, t + 2 >= t1);
              free_slots(vpos, 0, false);
            }
            if (t + 2 < t1) {
              if (t < t0) {
                ok = wait_warp(&M.q_full[x], nq[x] & 1, abort_v);
                ++nq[x];
              }
              ok = ok && wait_warp(&M.k_full[kg & (kAhead - 1)], (kg / kAhead) & 1, abort_v);
              ++kg;
              if (!ok) break;
              qk(x, kn, t + 4 >= t1);
              free_slots(-1, kn, true);
              kn = after_v<D>(after_k<D>(kn));
            }
          }
          pos = kpos;
          if (!ok) break;
          continue;
        }
        ok = wait_warp(&M.k_full[kg & (kAhead - 1)], (kg / kAhead) & 1, abort_v);
        ++kg;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (!ok || end[x] <= t0) continue;
          ok = wait_warp(&M.q_full[x], nq[x] & 1, abort_v);
          ++nq[x];
          if (ok) qk(x, kpos, t0 + 1 == end[x]);
        }
        if (!ok) break;
        free_slots(-1, kpos, true);
#pragma unroll 1
        for (int t = t0; t < t1; ++t) {
          const int vpos = after_k<D>(kpos);
          kpos = after_v<D>(vpos);
          bool have_k = false;
          ok = wait_warp(&M.v_ok[vg & (kAhead - 1)], (vg / kAhead) & 1, abort_v);
          ++vg;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!ok || t >= end[x]) continue;
            ok = wait_warp(&M.p_half[x], ns[x] & 1, abort_v);
            if (!ok) continue;
            const bool last = t + 1 == end[x];
            pv(x, vpos, 0, t == t0, false);
            ok = wait_warp(&M.p_full[x], ns[x] & 1, abort_v);
            ++ns[x];
            if (!ok) continue;
            pv(x, vpos, 4, false, last);
            if (last) continue;
            if (!have_k) {
              ok = wait_warp(&M.k_full[kg & (kAhead - 1)], (kg / kAhead) & 1, abort_v);
              ++kg;
              have_k = true;
            }
            if (ok) qk(x, kpos, t + 2 == end[x]);
          }
          if (!ok) break;
          free_slots(vpos, kpos, t + 1 < t1);
        }
        pos = kpos;
      }
      if (!ok) *abort_v = 2;
    } else {
      // -------------------------------------------------------------- V rows that some row does not see
      const int mine = warp - kScanWarp0;
      uint32_t n = 0, vg = 0;
      int pos = 0;
      bool ok = true;
      while (ok) {
        if (!wait_warp(&M.item_full[n & 1], (n >> 1) & 1, abort_v)) break;
        const Item it = M.items[n & 1];
        __syncwarp();
        if (lane == 0) arrive_in(&M.item_free[n & 1], 0);
        if (it.t1 == 0) break;
        ++n;
        const int all_see = seen_by(p, it, 0);  // keys before this one are seen by every row
        for (int t = it.t0; t < it.t1; ++t) {
          const int vpos = after_k<D>(pos);
          pos = after_v<D>(vpos);
          if (!wait_warp(&M.v_full[vg & (kAhead - 1)], (vg / kAhead) & 1, abort_v)) { ok = false; break; }
          if ((t + 1) * kTile > all_see) {
            // Eight lanes read the eight pieces of a row; the rows that every row sees left out.
            const int first = (max(0, all_see - t * kTile) & ~7) + 4 * mine;
            uint32_t hit = 0;
#pragma unroll 4
            for (int r = first; r < kTile; r += 8) {
              const uint8_t* at = smem + Z::kOffRing + vpos * kSlot + (r + (lane >> 3)) * 128 + (lane & 7) * 16;
              const uint4 w = *reinterpret_cast<const uint4*>(at);
              // an exponent of all ones carries into the sign's place
              auto odd = [](uint32_t v) { return (v & 0x7F807F80u) + 0x00800080u; };
              const uint32_t any = odd(w.x) | odd(w.y) | odd(w.z) | odd(w.w);
              hit |= static_cast<uint32_t>((any & 0x80008000u) != 0) << (r >> 3);
            }
            if (__any_sync(0xFFFFFFFFu, hit != 0)) {
              if (!note_odd(M, smem + Z::kOffRing + vpos * kSlot, hit, mine, rank, n, t * kTile, all_see, it.n_keys, abort_v)) { ok = false; break; }
              fence_proxy_async_smem();
            }
          }
          __syncwarp();
          if (lane == 0) {
            arrive_in(&M.v_ok[vg & (kAhead - 1)], 0);
            count_up(&M.scanned[2 * rank + mine]);
          }
          ++vg;
        }
        __syncwarp();
      }
    }
  } else {
    // -------------------------------------------------------------- softmax, results
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int x = (warp - kSoftWarp0) >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;  // of the row tile
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t s_col = tmem + lanes + kColS + kTile * x, o_col = tmem + lanes + kColO + kVal * x;
    const float hidden = NEG ? INFINITY : -INFINITY;  // times a negative scale: -inf
    uint32_t n = 0, g = 0, no = 0, vg = 0, nh = 0;  // items, tiles, results, V tiles, items in two halves
    bool ok = true;
    while (ok) {
      if (!wait_here(&M.item_full[n & 1], (n >> 1) & 1, abort_v)) break;
      const Item it = M.items[n & 1];
      __syncwarp();
      if (lane == 0) arrive_in(&M.item_free[n & 1], 0);
      if (it.t1 == 0) break;
      const bool halves = two_halves(p, it);
      const int first = ((halves ? 0 : 2 * x) + static_cast<int>(rank)) * (kTile >> p.gshift);  // this CTA's first token in the tile
      const int end = end_of(p, it, x), n_tok = min(it.n_tok - first, kTile >> p.gshift);
      const int token = first + (row >> p.gshift);  // of the block
      const bool exists = (row >> p.gshift) < n_tok;
      // (rows that do not exist count like the last one that does)
      const int seen = seen_by(p, it, min(token, it.n_tok - 1));
      const int least_seen = __reduce_min_sync(0xFFFFFFFFu, seen), most_seen = __reduce_max_sync(0xFFFFFFFFu, seen);
      float m = -INFINITY, l = 0.0f;
      const int t_first = it.t0 + (halves ? x : 0), t_step = halves ? 2 : 1;
      for (int t = t_first; t < end; t += t_step, ++g) {
        if (!wait_here(&M.s_full[x], g & 1, abort_v)) { ok = false; break; }
        tc_fence_after();
        // Keys that the row does not see: their logits are replaced where they lie, 32 keys at a time (a
        // short loop: it runs once or twice an item, and unrolled over the tile it would
        // push the tile's own code out of the instruction cache).
        const int left = seen - t * kTile, least = least_seen - t * kTile, most = most_seen - t * kTile;
        if (least < kTile) {
#pragma unroll 1
          for (int c = max(0, least) & ~31; c < kTile; c += 32) {
            uint32_t v[32];
            if (most > c) {  // (else no row of the warp sees any of them)
              tmem_ld_32x32b_x32(s_col + c, v);
              tmem_wait_ld();
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = c + i < left ? v[i] : __float_as_uint(hidden);
            tmem_st_32x32b_x32(s_col + c, v);
          }
          tmem_wait_st();
        }
        float s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(s_col + 32 * c, reinterpret_cast<uint32_t*>(s + 32 * c));
        tmem_wait_ld();
        float top = hidden, other = hidden;
#pragma unroll
        for (int i = 0; i < 128; i += 4) {
          top = NEG ? min3(top, s[i], s[i + 1]) : max3(top, s[i], s[i + 1]);
          other = NEG ? min3(other, s[i + 2], s[i + 3]) : max3(other, s[i + 2], s[i + 3]);
        }
        top = NEG ? fminf(top, other) : fmaxf(top, other);
        top *= p.scale_log2;
        const bool raise = top > m + kRaise || (m == -INFINITY && top > -INFINITY);
        float alpha = 1.0f;
        if (raise) {
          alpha = m == -INFINITY ? 0.0f : exp2_fast(m - top);
          m = top;
          l *= alpha;
        }
        const float ref = m == -INFINITY ? 0.0f : m;
        if (t > t_first && __any_sync(0xFFFFFFFFu, raise)) {  // O holds every tile before this one
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(o_col + 16 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st_x16(o_col + 16 * c, o);
          }
        }
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        const float2 factor = make_float2(p.scale_log2, p.scale_log2), minus = make_float2(-ref, -ref);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 y = fma2(make_float2(s[32 * h + i], s[32 * h + i + 1]), factor, minus);
            const float2 e = make_float2(exp2_fast(y.x), exp2_fast(y.y));
            sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], e);
            // P is rounded to bf16 (off by at most 2^-8 of a probability): a product's operands have one type, and
            // V in f16 would lose its range. Rows are off by 2^-8 / sqrt(3) of their length from it, about what rounding
            // the result to bf16 adds. The sum l is not rounded.
            pk[i >> 1] = bf_pack(e.x, e.y);
          }
          tmem_st_x16(s_col + 16 * h, pk);
          // The product with the first 64 keys may begin. (Handed over after 32, 64 or 96 keys, in quarters, at once: 8,192
          // tokens of 64 heads on 8 take 719, 661, 684, 709 and 735 us.)
          if (h == 1) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_in(&M.p_half[x], 0);
          }
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_in(&M.p_full[x], 0);
      }
      if (!ok) break;
      // ---- results
      const int head = it.unit << p.gshift;
      const long long flat = (static_cast<long long>(it.tok0) + token) * p.n_heads + head + (row & ((1 << p.gshift) - 1));
      const bool some = end > it.t0;  // (the items' tiles, or this half's)
      // What needs no product is done while the last one runs.
      Joined j{0.0f, -1.0f, -INFINITY};
      const bool alone = exists && it.whole && !halves;
      if (alone) {
        j = join_prev(p, flat, m, l);
        if (p.lse) p.lse[flat] = j.lse;
      }
      bool any_odd = false;
      if (some) {
        if (!wait_here(&M.o_full[x], no & 1, abort_v)) break;
        ++no;
        tc_fence_after();
        const uint32_t used = vg + static_cast<uint32_t>(end - it.t0);
        if (!wait_scanned(M, used, abort_v)) break;
        any_odd = *const_cast<volatile uint32_t*>(&M.odd_item[0]) == n + 1 || *const_cast<volatile uint32_t*>(&M.odd_item[1]) == n + 1;
        if (any_odd) cluster_fence();
      }
      vg += it.t1 - it.t0;
      // (nothing was noted that this warp needs: no need to wait for its stores)
      const bool done = !__any_sync(0xFFFFFFFFu, any_odd);
      if (done && lane == 0) count_up(&M.ended);
      // Two halves: the first one's warps join both and write the results.
      float w0 = 1.0f, w1 = 0.0f;
      if (halves) {
        if (x == 1) {
          M.ml[row] = make_float2(m, l);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&M.ml_full);
          if (!wait_here(&M.ml_free, nh & 1, abort_v)) break;  // it has read this half's O
        } else {
          if (!wait_here(&M.ml_full, nh & 1, abort_v)) break;
          tc_fence_after();
          const float2 other = M.ml[row];
          const float top = fmaxf(l != 0.0f ? m : -INFINITY, other.y != 0.0f ? other.x : -INFINITY);
          w0 = l != 0.0f ? exp2_fast(m - top) : 0.0f;
          w1 = other.y != 0.0f ? exp2_fast(other.x - top) : 0.0f;
          l = (l != 0.0f ? w0 * l : 0.0f) + (other.y != 0.0f ? w1 * other.y : 0.0f);
          m = top;
        }
        ++nh;
      }
      const bool writes = !(halves && x == 1);
      // 16 values of the row's sum
      auto sums = [&](int c, float* v) {
        tmem_ld_32x32b_x16(o_col + c, reinterpret_cast<uint32_t*>(v));
        if (halves) {
          float u[16];
          tmem_ld_32x32b_x16(o_col + kVal + c, reinterpret_cast<uint32_t*>(u));
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = w0 * v[i] + w1 * u[i];  // (both halves have tiles; a weight of 0 keeps a NaN)
        } else {
          tmem_wait_ld();
        }
      };
      if (writes && n_tok > 0 && it.whole) {
        if (exists && !alone) {
          j = join_prev(p, flat, m, l);
          if (p.lse) p.lse[flat] = j.lse;
        }
        // (a short loop: the tile loop's code fills the instruction cache, and what runs once an item
        // is fetched anew. 128 columns unrolled took 5,000 cycles, most of them waiting for code.)
        const float f = l != 0.0f ? j.f : 0.0f;
        const bool plain = !halves && !p.prev_lse && !p.out_fp32 && p.out_sectors;
#pragma unroll 1
        for (int c = 0; plain && c < kVal; c += 32) {  // the usual case by itself: less code to fetch
          float v[32];
          tmem_ld_32x32b_x32(o_col + c, reinterpret_cast<uint32_t*>(v));
          tmem_wait_ld();
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = l != 0.0f ? bf_pack(v[2 * i] * f, v[2 * i + 1] * f) : 0u;
          if (exists) {
            float* to = reinterpret_cast<float*>(static_cast<uint16_t*>(p.out) + flat * kVal + c);
            store8(to, reinterpret_cast<const float*>(w), true);
            store8(to + 8, reinterpret_cast<const float*>(w + 8), true);
          }
          __syncwarp();
        }
#pragma unroll 1
        for (int c = 0; !plain && c < kVal; c += 16) {
          float v[16];
          sums(c, v);
          if (exists) {
            const long long at = flat * kVal + c;
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = l != 0.0f ? v[i] * f : 0.0f;
            if (j.fp != -1.0f) add_prev(p, at, j.fp, v);
            if (p.out_fp32) {
              store8(static_cast<float*>(p.out) + at, v, p.out_sectors);
              store8(static_cast<float*>(p.out) + at + 8, v + 8, p.out_sectors);
            } else {
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = bf_pack(v[2 * i], v[2 * i + 1]);
              store8(reinterpret_cast<float*>(static_cast<uint16_t*>(p.out) + at), reinterpret_cast<const float*>(w), p.out_sectors);
            }
          }
          __syncwarp();
        }
        if (any_odd && exists && l != 0.0f) {
          for (int c = 0; c < kVal; ++c) {
            const float o = odd_of(M, n + 1, c, seen);
            if (o == 0.0f) continue;
            const long long at = flat * kVal + c;
            if (p.out_fp32) {
              static_cast<float*>(p.out)[at] += o;
            } else {
              uint16_t* to = static_cast<uint16_t*>(p.out) + at;
              *to = static_cast<uint16_t>(bf_pack(bf_lo(*to) + o, 0.0f));
            }
          }
        }
        __syncwarp();
      } else if (writes && quad * 32 >> p.gshift < n_tok) {  // a piece: some row of the warp exists
        const int r0 = (2 * x + static_cast<int>(rank)) * kTile + quad * 32;  // the warp's first row in the block
        const long long at = static_cast<long long>(it.slot) * kBlock + r0 + lane;
        float* part = reinterpret_cast<float*>(p.part_o + at * 32);
#pragma unroll 1
        for (int c = 0; c < kVal && some; c += 16) {
          float v[16];
          sums(c, v);
          if (exists) {
            store8(part + c, v, true);
            store8(part + c + 8, v + 8, true);
          }
          __syncwarp();
        }
        if (any_odd && exists) {
          for (int c = 0; c < kVal; ++c) {
            const float o = odd_of(M, n + 1, c, seen);
            if (o != 0.0f) part[c] += o;
          }
        }
        if (exists) p.part_ml[at] = make_float2(m, some ? l : -1.0f);  // -1: no tile, no values
      }
      tc_fence_before();
      __syncwarp();
      if (halves && x == 0 && lane == 0) mbar_arrive(&M.ml_free);
      if (!done && lane == 0) count_up(&M.ended);
      ++n;
    }
    if (!ok) *abort_v = 2;
  }

  __syncwarp();
  if (*abort_v == 2 && !M.status) set_status(&M.status, kStatusTimeout);
  if (*abort_v) {  // a wait gave up: let copies that are still under way land before the memory goes
    const long long t0 = clock64();
    while (clock64() - t0 < 4000000) __nanosleep(1000);
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && M.status) set_status(p.status, M.status);
  cluster_sync();  // the other CTA may still signal this one's shared memory until here
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// ------------------------------------------------------------------ joining the pieces
// Rows of the blocks that the line's cuts went through: their pieces' partial results, weighted by their maxima and
// sums, in the order of the pieces. A warp takes eight rows, a row's 128 values over its lanes. (In
// prompt_kernel, by the warp that ends last, it saved a launch and cost the tile loop its registers: 16,384 tokens
// 3.10 ms against 2.95.) 5 x 3 tokens on 9K keys: 76 blocks of up to three pieces, 3 us.
constexpr int kJoinThreads = 512;

__global__ void __launch_bounds__(kJoinThreads) join_kernel(const PromptParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Cut cut = p.cuts[blockIdx.x];
  const int lane = threadIdx.x & 31, r0 = (blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5)) * 8;
  const int n = min(8, (cut.n_tok << p.gshift) - r0);  // rows of the block are its tokens' heads
  if (cut.pieces == 0 || n <= 0) return;
  auto slot_of = [&](int i) { return static_cast<long long>(2 * (blockIdx.x + i) + (i == 0)) * kBlock + r0; };
  float best = -INFINITY, sum = 0.0f;  // of row lane mod 8
  const int mine = min(lane & 7, n - 1);
  for (int i = 0; i < cut.pieces; ++i) {
    const float2 ml = p.part_ml[slot_of(i) + mine];
    if (!(ml.y <= 0.0f)) best = fmaxf(best, ml.x);
  }
  for (int i = 0; i < cut.pieces; ++i) {
    const float2 ml = p.part_ml[slot_of(i) + mine];
    if (!(ml.y <= 0.0f)) sum += ml.y * exp2_fast(ml.x - best);
  }
  const int row = r0 + mine;
  const long long flat = (static_cast<long long>(cut.tok0) + (row >> p.gshift)) * p.n_heads + (cut.unit << p.gshift) + (row & ((1 << p.gshift) - 1));
  const Joined j = join_prev(p, flat, best, sum);
  __syncwarp();  // (lse may be prev_lse: every lane has read it)
  if (p.lse && lane < n) p.lse[flat] = j.lse;
  float4 acc[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) acc[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
  for (int i = 0; i < cut.pieces; ++i) {
    const long long s = slot_of(i);
    const float2 ml = p.part_ml[s + mine];
    // -1: nothing to add. (A piece with values is added even where its weight is 0: they may be NaN. A row that sees
    // nothing anywhere is 0.)
    const float w = sum == 0.0f || ml.y < 0.0f ? -1.0f : exp2_fast(ml.x - best);
    float4 v[8];
    float wr[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      wr[r] = r < n ? __shfl_sync(0xFFFFFFFFu, w, r) : -1.0f;
      if (wr[r] != -1.0f) v[r] = p.part_o[(s + r) * 32 + lane];
    }
#pragma unroll
    for (int r = 0; r < 8; ++r)
      if (wr[r] != -1.0f) acc[r].x += wr[r] * v[r].x, acc[r].y += wr[r] * v[r].y, acc[r].z += wr[r] * v[r].z, acc[r].w += wr[r] * v[r].w;
  }
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    if (r >= n) break;
    const float f = __shfl_sync(0xFFFFFFFFu, j.f, r), fp = __shfl_sync(0xFFFFFFFFu, j.fp, r);
    const long long to = __shfl_sync(0xFFFFFFFFu, flat, r);
    float4 v = make_float4(acc[r].x * f, acc[r].y * f, acc[r].z * f, acc[r].w * f);
    if (fp != -1.0f) {  // (a weight of 0 keeps a NaN)
      const float4 was = *reinterpret_cast<const float4*>(p.prev_out + to * kVal + 4 * lane);
      v.x += fp * was.x, v.y += fp * was.y, v.z += fp * was.z, v.w += fp * was.w;
    }
    store4(p, to, 4 * lane, v);
  }
}

// ------------------------------------------------------------------ host
// Heads as [rows][heads][width] 16-bit values, loaded in boxes of 64 values, `heads` heads and
// `rows` rows, 128-byte swizzled.
bool encode_heads(CUtensorMap* map, const smla_heads& t, uint64_t width, uint64_t n_heads, uint64_t rows, uint32_t box_heads, uint32_t box_rows) {
  typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
    return e == cudaSuccess && found == cudaDriverEntryPointSuccess ? reinterpret_cast<Encode>(f) : nullptr;
  }();
  if (!encode) return false;
  // (one head's or one row's stride is never used)
  const uint64_t row = rows > 1 ? t.row_stride : std::max<int64_t>(t.row_stride, width);
  const uint64_t head = n_heads > 1 ? t.head_stride : (width + 7) / 8 * 8;
  const cuuint64_t dims[3] = {width, n_heads, rows}, strides[2] = {head * 2, row * 2};
  const cuuint32_t box[3] = {64, box_heads, box_rows}, steps[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(t.data), dims, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool NEG>
int launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& pe, const PromptParams& p, cudaStream_t st) {
  if (!p.direct) {
    plan_kernel<<<1, kPlanThreads, 0, st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return SMLA_ERR_CUDA;
  }
  cudaLaunchAttribute at{};  // set up while the plan is made
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * (p.direct ? p.max_blocks * p.units : p.pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes<D>;
  cfg.stream = st;
  cfg.attrs = &at, cfg.numAttrs = p.direct ? 0 : 1;
  if (cudaLaunchKernelEx(&cfg, prompt_kernel<D, NEG>, q, k, v, pe, p) != cudaSuccess) return SMLA_ERR_CUDA;
  if (!p.can_cut) return SMLA_OK;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(p.pairs, kBlock / (8 * kJoinThreads / 32));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_kernel, p) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

template <int D, bool NEG>
bool set_smem() {
  return cudaFuncSetAttribute(prompt_kernel<D, NEG>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes<D>)) == cudaSuccess;
}
template <int D, bool NEG>
int resident_pairs() {
  if (!set_smem<D, NEG>()) return 0;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = 2, at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * num_sms());
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes<D>;
  cfg.attrs = &at, cfg.numAttrs = 1;
  int n = 0;
  return cudaOccupancyMaxActiveClusters(&n, prompt_kernel<D, NEG>, &cfg) == cudaSuccess ? n : 0;
}
// CTA pairs that run at the same time (76 on a 152-SM part; fewer where a GPC has an odd number of
// SMs). Looked up once per device, with the kernels' shared memory limit set. 0: no device.
int pairs_of_device() {
  static std::mutex mutex;
  static int known[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mutex);
  if (known[dev] == 0)
    known[dev] = std::min({resident_pairs<192, false>(), resident_pairs<192, true>(), resident_pairs<128, false>(), resident_pairs<128, true>(), num_sms() / 2});
  return known[dev];
}

// Sizes that follow from the shape, and the workspace's parts; its bytes.
size_t layout(PromptParams& p, uint8_t* ws) {
  p.gshift = 0;
  while (p.gshift < 7 && p.group % (2 << p.gshift) == 0) ++p.gshift;
  p.units = p.n_heads >> p.gshift;
  p.max_blocks = p.total_q / (kBlock >> p.gshift) + p.n_seqs;
  p.pairs = std::max(1, pairs_of_device());
  p.can_cut = p.total_k > kLongTiles * kTile;
  // A small call needs no plan: 1 x 100 tokens of 16 heads, 9.5 us of device time against 14.3.
  p.direct = !p.can_cut && p.n_seqs <= kDirectSeqs && static_cast<int64_t>(p.max_blocks) * p.units <= p.pairs;
  const PromptParts w = prompt_parts(reinterpret_cast<uintptr_t>(ws), kStatusBytes, p.max_blocks, p.pairs, p.n_seqs, p.can_cut != 0);
  p.plan = reinterpret_cast<Plan*>(ws + w.plan);
  p.cuts = reinterpret_cast<Cut*>(ws + w.cuts);
  p.blocks = reinterpret_cast<Block*>(ws + w.blocks);
  p.line_at = reinterpret_cast<long long*>(ws + w.line_at);
  p.sorted = reinterpret_cast<Block*>(ws + w.sorted);
  p.block_at = reinterpret_cast<int32_t*>(ws + w.block_at);
  p.part_ml = reinterpret_cast<float2*>(ws + w.part_ml);
  p.part_o = reinterpret_cast<float4*>(ws + w.part_o);
  return w.bytes;
}

bool sizes_ok(const PromptParams& p) {  // 32-bit rows and counts
  return p.n_heads <= 1024 && p.n_seqs <= (1 << 24) && p.total_q <= INT_MAX / 2 && p.total_k <= INT_MAX - 1024;
}
bool heads_ok(const smla_heads* t, int64_t width, int32_t n) {
  return t && t->data && aligned_to(t->data, 16) && t->row_stride % 8 == 0 && t->head_stride % 8 == 0 && t->row_stride >= width &&
         t->row_stride < (1LL << 35) && t->head_stride < (1LL << 35) && (n == 1 || t->head_stride >= width);
}

}  // namespace
}  // namespace smla

using namespace smla;

extern "C" {

size_t smla_prompt_fwd_workspace_size(int32_t total_q, int32_t total_k, int32_t n_seqs, int32_t n_heads, int32_t n_kv_heads) {
  if (total_q <= 0 || total_k <= 0 || n_seqs <= 0 || n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads) return kStatusBytes;
  PromptParams p{};
  p.total_q = total_q, p.total_k = total_k, p.n_seqs = n_seqs, p.n_heads = n_heads, p.group = n_heads / n_kv_heads;
  if (!sizes_ok(p)) return kStatusBytes;
  return layout(p, nullptr);
}

int smla_prompt_fwd(const smla_heads* q, const smla_heads* k, const smla_heads* v, const void* k_pe,
                    int64_t k_pe_stride, int32_t total_q, int32_t total_k, int32_t n_seqs, const int32_t* cu_q,
                    const int32_t* cu_k, int32_t n_heads, int32_t n_kv_heads, int32_t d_qk, int32_t causal,
                    float sm_scale, const float* prev_out, const float* prev_lse, void* out, int32_t out_fp32,
                    float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (total_q <= 0 || total_k <= 0 || n_seqs <= 0 || n_heads <= 0 || n_kv_heads <= 0 || d_qk <= 0 || n_heads % n_kv_heads) return SMLA_ERR_INVALID_ARG;
  const int d_k = k_pe ? d_qk - kPe : d_qk;
  if (d_qk != 128 && d_qk != 192) return SMLA_ERR_UNSUPPORTED;
  PromptParams p{};
  p.total_q = total_q, p.total_k = total_k, p.n_seqs = n_seqs, p.n_heads = n_heads, p.group = n_heads / n_kv_heads;
  if (!sizes_ok(p)) return SMLA_ERR_UNSUPPORTED;
  if (!heads_ok(q, d_qk, n_heads) || !heads_ok(k, d_k, n_kv_heads) || !heads_ok(v, kVal, n_kv_heads)) return SMLA_ERR_INVALID_ARG;
  if (k_pe && (!aligned_to(k_pe, 16) || k_pe_stride % 8 || k_pe_stride < kPe || k_pe_stride >= (1LL << 35))) return SMLA_ERR_INVALID_ARG;
  if (!cu_q || !cu_k || !out || !aligned_to(cu_q, 4) || !aligned_to(cu_k, 4) || !aligned_to(out, 16) || !aligned_to(lse, 4)) return SMLA_ERR_INVALID_ARG;
  if ((prev_out == nullptr) != (prev_lse == nullptr) || !aligned_to(prev_out, 16) || !aligned_to(prev_lse, 4) || !std::isfinite(sm_scale))
    return SMLA_ERR_INVALID_ARG;
  if (static_cast<const void*>(prev_out) == out && out && !out_fp32) return SMLA_ERR_INVALID_ARG;
  if (!workspace || !aligned_to(workspace, 16) || workspace_bytes < layout(p, static_cast<uint8_t*>(workspace))) return SMLA_ERR_WORKSPACE;
  p.cu_q = cu_q, p.cu_k = cu_k, p.causal = causal != 0, p.d_k = d_k;
  // never 0: masked logits are infinities, and 0 times those is not
  const float s = sm_scale * 1.4426950408889634f;
  if (!std::isfinite(s)) return SMLA_ERR_INVALID_ARG;
  p.scale_log2 = s < 0.0f ? std::min(s, -1e-37f) : std::max(s, 1e-37f);
  p.prev_out = prev_out, p.prev_lse = prev_lse, p.out = out, p.out_fp32 = out_fp32, p.out_sectors = aligned_to(out, 32), p.lse = lse;
  p.status = static_cast<uint32_t*>(workspace);
  // heads worked on at a time: K and V of their keys in some 40 MB of L2 (16,384 tokens 3.00 / 2.99 / 3.02 ms with
  // 20 / 40 / 80 MB)
  const int64_t kv_bytes = static_cast<int64_t>(total_k) * (d_k + kVal) * 2, at_once = std::max<int64_t>(1, (40LL << 20) / kv_bytes);
  p.units_a = static_cast<int32_t>(std::min<int64_t>(p.units, at_once * (p.group >> p.gshift)));
  CUtensorMap q_map{}, k_map{}, v_map{}, pe_map{};
  const int g = 1 << p.gshift;
  const smla_heads pe{k_pe, k_pe_stride, kPe};
  if (!encode_heads(&q_map, *q, d_qk, n_heads, total_q, g, kTile / g) || !encode_heads(&k_map, *k, d_k, n_kv_heads, total_k, 1, kTile / 2) ||
      !encode_heads(&v_map, *v, kVal, n_kv_heads, total_k, 1, kTile) || (k_pe && !encode_heads(&pe_map, pe, kPe, 1, total_k, 1, kTile / 2)))
    return SMLA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const auto go = d_qk == 192 ? (p.scale_log2 < 0.0f ? launch<192, true> : launch<192, false>) : (p.scale_log2 < 0.0f ? launch<128, true> : launch<128, false>);
  return go(q_map, k_map, v_map, pe_map, p, st);
}

}  // extern "C"
