// Attention of a batch over a shared prompt and each request's own tokens
// (smla_shared_prefix_fwd): out = softmax(sm_scale q K^T) K[:, 0:512] over every
// key a token sees, in one pass over the keys with a running maximum and sum.
//
// Rows of the problem are (token, head) pairs: the latent row of a key serves
// every head of every token, so the shared prompt is ONE product with
// n_seqs * q_per_seq * n_heads rows, and a request's own tokens one with
// q_per_seq * n_heads rows. Both are cut into segments of 128 rows (row block)
// x a range of keys, walked in tiles of 128 keys (two pages).
//
// Why a CTA pair. A row's output has 512 fp32 values, so 128 rows fill all 512
// columns of an SM's tensor memory and leave none for the logits. A cluster of
// two CTAs therefore shares a block of 128 rows:
//   CTA c computes the logits of page c of each tile (QK over 576 values) and
//   the output values 256 c .. 256 c + 255 (PV over both pages of the tile).
// Every product is one M = 128 tcgen05.mma per 16 values, no logit is computed
// twice, and what crosses the pair per tile is the row maxima (512 B) and the
// probabilities of the other page (16 KB), both sent through distributed shared
// memory with their bytes counted on the receiver's barrier.
//
// Tensor memory (512 columns): O 256 | S 64 | six of Q's nine chunks (192). Shared
// memory (216 KB + barriers): Q's other chunks, the keys of one tile in flight
// in QK and one in PV as 17 slots of 64 keys x 64 values, and both halves of P:
//   KO  own page, the 5 chunks that only QK reads     (1 tile)
//   KV  own page, the 4 chunks of this CTA's output   (2 tiles)
//   VO  other page, the 4 chunks of this CTA's output (1 tile)
// Warp roles: 0 MMA issue, 1 TMA loads, 4-11 softmax and results (a thread per row
// and half of the page's keys); FP8 caches: 2-3 and 12-15 load and widen rows, two
// warps for each of KO, KV and VO. FP8 rows that several row blocks read (the shared
// part, where there are two row blocks or more) are widened once by widen_kernel and
// come by TMA like BF16 rows; the widening warps then only pass the tile on.
// The issue order QK(t + 1), PV(t) keeps the tensor pipe busy during softmax(t).
//
// The work is cut evenly: segment after segment on one line (each tile and each
// segment's start has a cost), and pair i of P walks the i-th of P equal stretches.
// A segment that is cut leaves several partial results (fp32 O with its maximum
// and sums) that merge_kernel joins; no pair waits for another. Rows whose keys are
// one uncut segment get their results at once.
//
// Bound by the tensor pipe: a tile's 44 MMAs take 2,376 cycles issued back to back,
// a tile here 2,900 (BF16), the rest being the row maxima's way across the pair and
// the starts of segments. 64 x 2 tokens of 64 heads on a 64K prompt: 735 us and 20 to
// join, 1,620 TFLOP/s in this kernel, 85% of cuBLAS's bf16 rate (the tensor pipe is
// active in 72% of the cycles of a call half that size). 1,024 tokens after 8K: 740 us and 20.
// Per-token FP8, 64 x 2 on 16K: 218 us, 8 to widen, 25 to join, 1,240 TFLOP/s in all:
// the requests' own keys, 6% of all, are 15% of the line's cost. A single request's
// FP8 rows have no copy: each of its row blocks widens them (1,024 tokens after 8K: 1.34
// ms with per-token scales, 2.27 ms with tile scales, 0.78 ms from BF16 rows). One token
// on 1,100 keys: 13 us, 17 on cold caches, a chain of latencies: Q, three tiles a pair,
// results, join.
#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "serve.h"

namespace smla {
namespace {

constexpr int kRows = 128;       // rows of a block (MMA M)
// Costs on the line of work, in quarters of a tile that comes by TMA (2,900 cycles
// with BF16 rows, 3,100 with the 16-bit copy): a segment's start (the pipeline
// drains, Q in, results out), a tile of the shared part, a tile of a request's own
// keys (FP8: widened on the way, 5,500 cycles with per-token scales, 7,800 with tile
// scales). Starts and own tiles weighed too lightly leave the pairs that walk short
// segments to end last. Measured over the start's cost: 64 x 2 tokens of 64 heads on
// a 64K prompt, BF16, 850 / 834 / 825 / 842 us at 12 / 16 / 20 / 24; on a 16K prompt,
// per-token FP8, 284 / 275 / 266 / 259 us at 20 / 26 / 32 / 38 with own tiles at 6, and
// 254 / 253 / 258 at 38 / 44 / 56 with own tiles at 7; later 255 at 40 and 7, 256 / 257 /
// 260 at 32 / 40 / 48 with own tiles at 8.
struct Costs {
  int32_t start, shared_tile, own_tile;
};
constexpr int kChunk = 64 * 128; // 64 keys x 64 values
constexpr int kQChunk = kRows * 128;
// Q chunks follow the key slots they meet (KO 0-4, KV 0-3, below): those of KO 0-3
// and KV 0-1 are in tensor memory, those of KO 4 and KV 2-3 in shared memory.
constexpr uint32_t kColO = 0, kColS = 256, kColQ = 320;
constexpr int kOffQ = 0, kOffKO = 3 * kQChunk, kOffKV = kOffKO + 5 * kChunk, kOffVO = kOffKV + 8 * kChunk,
              kOffP = kOffVO + 4 * kChunk, kOffMeta = kOffP + 2 * kQChunk;
constexpr float kRaise = 8.0f;   // log2: the reference maximum is raised only when exceeded by this much
constexpr int kMaxPairs = 128;
constexpr int kMaxPieces = kMaxPairs + 2;  // of a row: its two segments are walked by distinct pairs, but for one at each border
constexpr int kEnds = 768, kGroups = 512;
constexpr int kTileRowBytes = 656, kTileRope = 528;
constexpr int kSoftWarps = 8, kMmaWarp = 0, kTmaWarp = 1, kSoftWarp0 = 4;
constexpr int kPHalf = kRows * 64;  // P of half a page: 128 rows x 32 keys, 64-byte swizzled

enum { kBf16 = 0, kTokenFp8 = 1, kTileFp8 = 2 };

struct PrefixParams {
  const uint8_t* kv;
  const float* kv_scale;
  int32_t num_pages;
  const int32_t* page_tables;
  int32_t max_pages, n_seqs;
  const int32_t* seq_lens;
  int32_t max_seq_len, shared_len, q_per_seq, hshift;  // heads = 1 << hshift
  const uint16_t* q;
  float scale_log2;   // |sm_scale| log2 e, not 0
  uint32_t q_sign;    // flips the sign of Q where sm_scale is negative
  uint16_t* out;
  float* lse;
  uint32_t* status;
  int32_t n_rows;     // tokens * heads
  int32_t n_rb;       // row blocks of the shared part (0: nothing shared)
  int32_t end_shift;  // 2^end_shift row blocks form a group with one end of the shared part
  int32_t n_groups;   // (kGroups at most)
  int32_t rb_s;       // row blocks of one request
  int32_t n_seg, pairs;
  int32_t pair_slots; // where partial results lie: piece_slot
  Costs costs;
  int32_t q_tma;      // Q's chunks for shared memory come by TMA
  int32_t q_sectors;  // q starts on a 32-byte boundary
  int32_t wide;       // FP8: the shared rows are read from their 16-bit copy
  uint16_t* wide_rows;  // [shared pages * 64][576]
  long long* seg_off; // [s] where segment s starts on the line; -1: one piece walks it and writes the results itself
  long long* bounds;  // [pairs + 1] where each pair's stretch starts
  uint32_t* errors;   // [2 * pairs] status bits of each CTA
  uint4* wide_over;   // [shared pages] tile-scaled: which of each page's 4 x 16 keys hold a value outside f16's range
  float* part_m;      // [slot][128]
  float* part_l;      // [slot][4][128]: sums of each CTA's two halves
  float4* part_o;     // [slot][2][64][128]: four output values of a row
};

// ------------------------------------------------------------------ the line of work
__device__ __forceinline__ int length_of(const PrefixParams& p, int b) {
  return max(0, min(__ldg(p.seq_lens + b), p.max_seq_len));
}
// Keys of the shared part that some token of the row blocks of group g sees: a block of
// idle requests, or of requests that end before the shared part does, walks no more.
__device__ __forceinline__ int shared_end(const PrefixParams& p, int g) {
  const int n = (kRows >> p.hshift) << p.end_shift, first = g * n, last = min(first + n, p.n_rows >> p.hshift);  // its tokens
  int b = first / p.q_per_seq, j = first - b * p.q_per_seq, end = 0;
#pragma unroll 4
  for (int k = first; k < last; ++k) {
    end = max(end, length_of(p, b) - p.q_per_seq + j + 1);
    if (++j == p.q_per_seq) j = 0, ++b;
  }
  return min(end, p.shared_len);
}
// Keys that the last token of own segment i sees.
__device__ __forceinline__ int own_end(const PrefixParams& p, int i) {
  const int b = i / p.rb_s, rb = i - b * p.rb_s;
  const int j = min(p.q_per_seq - 1, (rb * kRows + kRows - 1) >> p.hshift);
  return length_of(p, b) - p.q_per_seq + j + 1;
}
__device__ __forceinline__ int own_tiles(const PrefixParams& p, int end) {
  if (end <= p.shared_len) return 0;
  return ((end + kPage - 1) / kPage - p.shared_len / kPage + 1) >> 1;
}
__device__ __forceinline__ int shared_tiles(int end) { return (end + 2 * kPage - 1) / (2 * kPage); }
// The same from the CTA's table: the groups' ends, then those of the own segments as far as it reaches.
__device__ __forceinline__ int seg_end(const PrefixParams& p, const int* ends, int s) {
  const int at = s < p.n_rb ? s >> p.end_shift : s - p.n_rb + p.n_groups;
  return at < kEnds ? ends[at] : own_end(p, s - p.n_rb);
}
__device__ __forceinline__ int seg_tiles(const PrefixParams& p, const int* ends, int s) {
  const int end = seg_end(p, ends, s);
  return s < p.n_rb ? shared_tiles(end) : own_tiles(p, end);
}
__device__ __forceinline__ int seg_cost(const PrefixParams& p, int s, int tiles) {
  return tiles > 0 ? p.costs.start + tiles * (s < p.n_rb ? p.costs.shared_tile : p.costs.own_tile) : 0;
}
// Tiles [t0, t1) of segment s, which starts at a, that begin inside the stretch [x, y).
__device__ __forceinline__ void stretch_tiles(const PrefixParams& p, int s, int tiles, long long a, long long x, long long y, int& t0,
                                              int& t1) {
  const uint32_t one = s < p.n_rb ? p.costs.shared_tile : p.costs.own_tile;
  const long long from = a + p.costs.start, most = static_cast<long long>(tiles) * one;  // (below 2^31: a tile has 128 keys)
  t0 = static_cast<int>((static_cast<uint32_t>(min(max(x - from, 0LL), most)) + one - 1) / one);
  t1 = static_cast<int>((static_cast<uint32_t>(min(max(y - from, 0LL), most)) + one - 1) / one);
}

struct Line {  // a pair's stretch [x, y) and where it stands: segment s starts at a
  long long x, y, a;
  int s;
};
struct Piece {
  int s, t0, t1;  // tiles [t0, t1) of segment s
  bool whole;     // all of them
};

__device__ __forceinline__ bool piece_after(const PrefixParams& p, const int* ends, Line& L, Piece& pc, bool writer) {
  while (L.s < p.n_seg && L.a < L.y) {
    const int s = L.s++;
    const int tiles = seg_tiles(p, ends, s), cost = seg_cost(p, s, tiles);
    const long long a = L.a;
    if (cost == 0) continue;
    L.a += cost;
    stretch_tiles(p, s, tiles, a, L.x, L.y, pc.t0, pc.t1);
    if (pc.t1 > pc.t0) {
      pc.s = s;
      pc.whole = pc.t0 == 0 && pc.t1 == tiles;
      // (the pair with the first tile writes it)
      if (writer && pc.t0 == 0) p.seg_off[s] = pc.whole && p.n_rb == 0 ? -1 : a;
      return true;
    }
  }
  return false;
}

// Slot of the partial results of a pair's piece of segment s that begins at tile t0. Along
// the line segment + pair grows with every piece, so it is a slot of the piece's own. With
// nothing shared uncut segments write no partial results, and a pair has two pieces at
// most that do: one that goes on from the pair before, one that goes on in the next. Two
// slots a pair are fewer where there are more segments than pairs (a chunk of 8,192
// tokens of 64 heads: 40 MB, against 1.1 GB with a slot a segment).
__device__ __forceinline__ int piece_slot(const PrefixParams& p, int s, int pair, int t0) {
  return (p.pair_slots ? pair + (t0 == 0) : s) + pair;
}

// Through copies, so that the caller's own stay in registers.
__device__ __forceinline__ bool next_piece(const PrefixParams& p, const int* ends, Line& L, Piece& pc, bool writer) {
  Line line = L;
  Piece piece;
  const bool more = piece_after(p, ends, line, piece, writer);
  L = line;
  if (more) pc = piece;
  return more;
}

// The tiles of a pair's pieces one after another, with the tile's page ids.
struct Tiles {
  Line line;
  Piece pc;
  int t;
  const int32_t* table;
  int first_page, end_page;  // of the segment
  int seen_page;             // end of the pages that some row of the segment sees
  int first_key, end_key;    // keys that some row sees
  int own_id, other_id;      // table entries of the tile's page `rank` and of the other one (kNoPage past the end);
                             // loaded a tile ahead and looked at when the tile is
  static constexpr int kNoPage = INT_MIN;

  __device__ __forceinline__ int entry(int i) const { return i < end_page ? __ldg(table + i) : kNoPage; }
  // pool page of an entry, -1: none
  static __device__ __forceinline__ int pool_page(const PrefixParams& p, int id) { return id >= 0 && id < p.num_pages ? id : -1; }
  // a page that a row sees is missing
  __device__ __forceinline__ bool bad(const PrefixParams& p, int rank) const {
    const int page = first_page + 2 * t;
    return (page + rank < seen_page && pool_page(p, own_id) < 0) || (page + (rank ^ 1) < seen_page && pool_page(p, other_id) < 0);
  }
  __device__ __forceinline__ bool next_segment(const PrefixParams& p, const int* ends) {
    if (!next_piece(p, ends, line, pc, false)) return false;
    t = pc.t0;
    const int end = seg_end(p, ends, pc.s);
    end_key = end;
    if (pc.s < p.n_rb) {
      table = p.page_tables;
      first_page = first_key = 0;
      end_page = (p.shared_len + kPage - 1) / kPage;
      seen_page = (end + kPage - 1) / kPage;
    } else {
      const int i = pc.s - p.n_rb;
      table = p.page_tables + static_cast<long long>(i / p.rb_s) * p.max_pages;
      first_page = p.shared_len / kPage;
      first_key = p.shared_len;
      end_page = seen_page = (end + kPage - 1) / kPage;
    }
    return true;
  }
  __device__ __forceinline__ bool next(const PrefixParams& p, const int* ends, int rank, bool fresh) {
    if ((fresh || ++t >= pc.t1) && !next_segment(p, ends)) return false;
    own_id = entry(first_page + 2 * t + rank);
    other_id = entry(first_page + 2 * t + (rank ^ 1));
    return true;
  }
};

// ------------------------------------------------------------------ cluster helpers
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// one float into the peer's shared memory, its 4 bytes counted on the peer's barrier
__device__ __forceinline__ void send_float(uint32_t dst, float v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(dst),
               "r"(__float_as_uint(v)), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void send_bulk(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(src), "r"(bytes), "r"(bar)
               : "memory");
}
// Bounded waits without calls: across a call the tile loops' values would go to local
// memory, and next to 225 KB of shared memory there is hardly any L1 to hold it.
// kCluster: also acquires what the other CTA sent.
template <bool kCluster>
__device__ __forceinline__ bool try_bar(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  if (kCluster)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  return ok != 0;
}
// Gives up after kWaitLimitCycles, or when another role has: false, and *abort is
// raised (the end of the kernel reports it). One thread.
template <bool kCluster>
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint32_t a = smem_u32(bar);
  long long t0 = 0;
  for (uint32_t it = 1; !try_bar<kCluster>(a, parity); ++it) {
    if ((it & 255u) != 0) continue;
    if (t0 == 0) t0 = clock64();
    if (*abort || clock64() - t0 > kWaitLimitCycles) {
      *abort = 2;
      return false;
    }
  }
  return true;
}
// The same by a whole warp: every lane sees the phase, all leave together.
template <bool kCluster>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint32_t a = smem_u32(bar);
  long long t0 = 0;
  for (uint32_t it = 1; !__all_sync(0xFFFFFFFFu, try_bar<kCluster>(a, parity)); ++it) {
    if ((it & 255u) != 0) continue;
    if (t0 == 0) t0 = clock64();
    if (__any_sync(0xFFFFFFFFu, *abort != 0 || clock64() - t0 > kWaitLimitCycles)) {
      *abort = 2;
      return false;
    }
  }
  return true;
}
// Bounded wait of the MMA warp, warp-uniform and without a call (a call takes the
// descriptors out of the uniform registers). It polls about 2^26 times at most
// (a second or so). Measured between batches of MMAs on a phase that is complete:
// 67 cycles; 163 with the loop left by each lane for itself, 300 with a try_wait
// that has a time hint, and there are six such waits in a tile's 2,400 cycles.
template <bool kCluster>
__device__ __forceinline__ bool wait_poll(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  auto done = [&] {
    uint32_t ok;
    if (kCluster)
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(a), "r"(parity)
          : "memory");
    else
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(a), "r"(parity)
          : "memory");
    return __all_sync(0xFFFFFFFFu, ok != 0) != 0;
  };
  bool ok = done();
  for (uint32_t it = 0; !ok && it < (1u << 26); ++it) ok = done();
  return ok;
}
// the same box into L2 only
__device__ __forceinline__ void prefetch_chunks(const CUtensorMap* map, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(0), "r"(y), "r"(z)
               : "memory");
}
// true in one thread of the (converged) warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
  return r != 0;
}
// chunks z .. of a page (box 64 values x 64 keys x chunks: one 8 KB slot per chunk)
__device__ __forceinline__ void tma_chunks(void* dst, const CUtensorMap* map, uint64_t* bar, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(y), "r"(z)
      : "memory");
}
// Shared-memory operand of an MMA: the low word of its descriptor holds the address
// (in 16 bytes), the high word is the same wherever the operand starts.
struct Operand {
  uint32_t lo, hi;
  __device__ __forceinline__ Operand operator+(int bytes) const { return {lo + static_cast<uint32_t>(bytes >> 4), hi}; }
};
__device__ __forceinline__ Operand operand(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t layout = kSwizzle128B) {
  const uint64_t d = smem_desc(saddr, lbo, sbo, layout);
  return {static_cast<uint32_t>(d), static_cast<uint32_t>(d >> 32)};
}
// A from tensor memory
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, Operand b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A from shared memory
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, Operand a, Operand b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %6, 0;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// arrives on the barrier at this address in both CTAs of the pair
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\t"
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
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
__device__ __forceinline__ uint32_t pack2(float a, float b, bool f16) {
  if (f16) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// two e4m3 codes -> two f16 values, exactly
__device__ __forceinline__ uint32_t e4m3x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
__device__ __forceinline__ uint32_t piece_off(int row, int j) {  // 16-byte piece j of a 128-byte swizzled row
  return static_cast<uint32_t>(row * 128 + ((j ^ (row & 7)) << 4));
}
// ... -> two bf16 values, exactly
__device__ __forceinline__ uint32_t e4m3x2_bf16(uint16_t c) {
  const uint32_t h = e4m3x2(c);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack2(f.x, f.y, false);
}
// bf16 pair -> f16 pair; `over`: a value outside f16's range
__device__ __forceinline__ uint32_t to_f16(uint32_t w, bool& over) {
  over |= ((w & 0x7FFFu) > 0x477Fu && (w & 0x7FFFu) < 0x7F80u) || ((w & 0x7FFF0000u) > 0x477F0000u && (w & 0x7FFF0000u) < 0x7F800000u);
  return pack2(bf_lo(w), bf_hi(w), true);
}

struct Meta {
  float mx[2][4][kRows];      // row maxima of this CTA's two halves and of the other's
  float4 ks[kSoftWarps][8];   // per softmax warp: the scales of its 32 keys (per-token FP8),
  float4 vs[kSoftWarps][8];   // and as they meet the probabilities
  uint64_t q_full, ko_full, kv_full[2], vo_full, ko_free, kv_free[2], vo_free;
  uint64_t s_full, s_free, p_own, pv_done, o_free;
  uint64_t mx_full[2][4];
  long long scan[34];
  int ends[kEnds];            // seg_end
  long long start_a;
  int start_s;
  uint32_t tmem_slot, status;
  int abort_flag;
};
constexpr size_t kSmemBytes = kOffMeta + sizeof(Meta);
static_assert(kSmemBytes <= 232448, "shared memory budget");

// Keys [lo, hi) that a row sees in its segment; over the block's rows that see
// any, the smallest and largest hi.
struct Limits {
  int lo, hi, min_hi, max_hi;
};
__device__ __forceinline__ Limits limits(const PrefixParams& p, int s, int row) {
  const int lane = threadIdx.x & 31;
  const bool shared = s < p.n_rb;
  const int i = s - p.n_rb, b0 = shared ? 0 : i / p.rb_s;
  const int r0 = (shared ? s : i - b0 * p.rb_s) * kRows;
  const int last = shared ? p.n_rows >> p.hshift : p.q_per_seq;  // tokens of the batch or of the request
  const int n = kRows >> p.hshift;  // tokens of the block (at most 8): one a lane
  Limits m;
  m.lo = shared ? 0 : p.shared_len;
  const int k = (r0 >> p.hshift) + lane;
  int hi = 0;
  if (lane < n && k < last) {
    const int b = shared ? k / p.q_per_seq : b0, j = shared ? k - b * p.q_per_seq : k;
    hi = max(0, length_of(p, b) - p.q_per_seq + j + 1);
    if (shared) hi = min(hi, p.shared_len);
  }
  m.min_hi = hi > m.lo ? hi : INT_MAX;
  m.max_hi = hi > m.lo ? hi : 0;
#pragma unroll
  for (int d = 4; d > 0; d >>= 1) {
    m.min_hi = min(m.min_hi, __shfl_xor_sync(0xFFFFFFFFu, m.min_hi, d));
    m.max_hi = max(m.max_hi, __shfl_xor_sync(0xFFFFFFFFu, m.max_hi, d));
  }
  m.min_hi = __shfl_sync(0xFFFFFFFFu, m.min_hi, 0);
  m.max_hi = __shfl_sync(0xFFFFFFFFu, m.max_hi, 0);
  m.hi = __shfl_sync(0xFFFFFFFFu, hi, row >> p.hshift);
  return m;
}

// First row of segment s in q, and how many of the rows from there on are its own.
__device__ __forceinline__ long long first_row(const PrefixParams& p, int s, int& rows) {
  if (s < p.n_rb) {
    rows = p.n_rows - s * kRows;
    return static_cast<long long>(s) * kRows;
  }
  const int i = s - p.n_rb, b = i / p.rb_s, in = (i - b * p.rb_s) * kRows;
  rows = (p.q_per_seq << p.hshift) - in;
  return (static_cast<long long>(b) * p.q_per_seq << p.hshift) + in;
}
// 32 bytes, a whole sector, at once (aligned to 32)
__device__ __forceinline__ void ldg32(const void* p, uint32_t* v) {
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "l"(p));
}
// Q of segment s, by one softmax warp (the logits of the previous piece are complete:
// all of Q's places are free). The six chunks for tensor memory: every lane reads its
// own row's 128 bytes a chunk in whole sectors. The three for shared memory come by
// TMA unless their values change on the way (f16, a negative scale): then eight lanes
// bring a row's chunk in 16-byte pieces. More chunks in flight push the tile
// loops' values into local memory, and next to 225 KB of shared memory there is
// hardly any L1 to hold that. Returns whether a value was outside f16's range. f16:
// rows that are not in `live` (they see no key of the segment) count as zeros, whatever
// they hold.
template <int FMT>
__device__ __forceinline__ bool load_q(const PrefixParams& p, int s, uint8_t* q_smem, uint32_t q_tmem, int rank, int quad, int half,
                                       uint32_t live) {
  constexpr bool F16 = FMT == kTileFp8;
  constexpr int kBatch = FMT == kBf16 ? 3 : 1;
  const int lane = threadIdx.x & 31;
  int rows;
  const uint16_t* src = p.q + (first_row(p, s, rows) + quad * 32) * kDqk;
  const int limit = rows - quad * 32;  // rows of the warp that exist
  float top = 0.0f;
  auto change = [&](uint32_t w) {
    if (F16) {
      const float a = bf_lo(w), b = bf_hi(w);
      top = fmaxf(top, fmaxf(fabsf(a), fabsf(b)));
      w = pack2(a, b, true);
    }
    return w ^ p.q_sign;
  };
  // chunk of values at place c: 0-5 in tensor memory (KO 0-3, KV 0-1), 6-8 in shared memory (KO 4, KV 2-3)
  auto chunk_of = [&](int c) { return c < 4 ? 4 * (rank ^ 1) + c : c < 6 ? 4 * rank + c - 4 : c == 6 ? 8 : 4 * rank + c - 5; };
  uint32_t v[kBatch][32];
#pragma unroll 1
  for (int c0 = 3 * half; c0 < 3 * half + 3; c0 += kBatch) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const uint16_t* at = src + lane * kDqk + chunk_of(c0 + u) * 64;
      if (lane >= limit || (F16 && !(live >> lane & 1))) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[u][j] = 0;
      } else if (p.q_sectors) {
#pragma unroll
        for (int j = 0; j < 4; ++j) ldg32(at + 16 * j, v[u] + 8 * j);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint4 w = __ldg(reinterpret_cast<const uint4*>(at) + j);
          v[u][4 * j] = w.x, v[u][4 * j + 1] = w.y, v[u][4 * j + 2] = w.z, v[u][4 * j + 3] = w.w;
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[u][j] = change(v[u][j]);
      tmem_st_32x32b_x32(q_tmem + 32 * (c0 + u), v[u]);
    }
  }
  if (!p.q_tma) {
    const int sub = lane >> 3, pcs = lane & 7;
#pragma unroll 1
    for (int c = 6; c < 9; ++c) {  // half of the warp's rows each
      uint4 w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 16 * half + 4 * j + sub;
        w[j] = r < limit && (!F16 || (live >> r & 1)) ? __ldg(reinterpret_cast<const uint4*>(src + r * kDqk + chunk_of(c) * 64 + pcs * 8)) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4*>(q_smem + (c - 6) * kQChunk + piece_off(quad * 32 + 16 * half + 4 * j + sub, pcs)) =
            make_uint4(change(w[j].x), change(w[j].y), change(w[j].z), change(w[j].w));
    }
    fence_proxy_async_smem();
  }
  tmem_wait_st();
  tc_fence_before();
  __syncwarp();
  return top > 65504.0f;
}
// the rows of a later segment's Q into L2
__device__ __forceinline__ void prefetch_q(const PrefixParams& p, int s, int row) {
  int rows;
  const long long first = first_row(p, s, rows);
  if (row < rows) prefetch_l2_lines(p.q + (first + row) * kDqk, 2 * kDqk);
}

template <int FMT>
constexpr int kThreadsOf = FMT == kBf16 ? 384 : 512;

template <int FMT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreadsOf<FMT>, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap rope_map,
                  const __grid_constant__ CUtensorMap q_map, const PrefixParams p) {
  constexpr bool F16 = FMT == kTileFp8;  // operand type of the MMAs: bf16 holds BF16 rows and e4m3 codes as they are
  constexpr uint32_t kFmt = F16 ? kFmtF16 : kFmtBF16;
  constexpr int kThreads = kThreadsOf<FMT>;
  constexpr uint32_t kFills = FMT == kBf16 ? 1 : 3;  // arrivals that fill a slot group: TMA and the widening warps
  extern __shared__ __align__(1024) uint8_t smem[];
  Meta& M = *reinterpret_cast<Meta*>(smem + kOffMeta);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int pair = blockIdx.x >> 1;
  const bool aligned = (smem_u32(smem) & 1023u) == 0;

  asm volatile("griddepcontrol.launch_dependents;");  // merge_kernel may take an SM as soon as there is room
  if (tid == 0) {
    mbar_init(&M.q_full, kSoftWarps + (p.q_tma ? 1 : 0));
    mbar_init(&M.ko_full, kFills);
    mbar_init(&M.vo_full, kFills);
    mbar_init(&M.ko_free, 1);
    mbar_init(&M.vo_free, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&M.kv_full[i], kFills);
      mbar_init(&M.kv_free[i], 1);
      for (int w = 0; w < 4; ++w) mbar_init(&M.mx_full[i][w], 1);
    }
    mbar_init(&M.s_full, 1);
    mbar_init(&M.s_free, kSoftWarps);
    mbar_init(&M.p_own, kSoftWarps);
    mbar_init(&M.pv_done, 2);
    mbar_init(&M.o_free, kSoftWarps);
    M.abort_flag = 0;
    M.status = 0;
    M.start_s = p.n_seg;
    M.start_a = 0;
    fence_mbar_init();
    if (!aligned) set_status(&M.status, kStatusSetup);
  }
  if (warp == kTmaWarp) {
    tmem_alloc(&M.tmem_slot, 512);
    tmem_relinquish();
  }

  // ---- the length of the line, this pair's stretch, and the segment it begins in
  Line line;
  {
    for (int i = tid; i < min(p.n_groups + p.n_seg - p.n_rb, kEnds); i += kThreads)
      M.ends[i] = i < p.n_groups ? shared_end(p, i) : own_end(p, i - p.n_groups);
    if (p.end_shift > 0) __syncthreads();  // (otherwise a thread reads the ends that it wrote)
    const long long first_cost = tid < p.n_seg ? seg_cost(p, tid, seg_tiles(p, M.ends, tid)) : 0;
    long long sum = first_cost;
    for (int i = tid + kThreads; i < p.n_seg; i += kThreads) sum += seg_cost(p, i, seg_tiles(p, M.ends, i));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    if (lane == 0) M.scan[warp] = sum;
    if (pair == 0 && rank == 0)
      for (int b = tid; b < p.n_seqs; b += kThreads)
        if (__ldg(p.seq_lens + b) > p.max_seq_len) set_status(&M.status, kStatusBounds);
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < kThreads / 32; ++w) total += M.scan[w];
    line.x = total * pair / p.pairs;
    line.y = total * (pair + 1) / p.pairs;
    if (rank == 0 && tid == 0) {
      p.bounds[pair] = line.x;
      if (pair == p.pairs - 1) p.bounds[p.pairs] = line.y;
    }
    if (line.x < line.y) {
      long long before = 0;
      for (int c0 = 0; c0 < p.n_seg && before <= line.x; c0 += kThreads) {
        const int i = c0 + tid;
        const long long cost = c0 == 0 ? first_cost : i < p.n_seg ? seg_cost(p, i, seg_tiles(p, M.ends, i)) : 0;
        long long v = cost;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const long long o = __shfl_up_sync(0xFFFFFFFFu, v, d);
          if (lane >= d) v += o;
        }
        __syncthreads();
        if (lane == 31) M.scan[warp] = v;
        __syncthreads();
        long long all = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
          if (w < warp) v += M.scan[w];
          all += M.scan[w];
        }
        if (before + v - cost <= line.x && line.x < before + v) {
          M.start_s = i;
          M.start_a = before + v - cost;
        }
        before += all;
      }
    }
  }
  if (FMT != kBf16) asm volatile("griddepcontrol.wait;" ::: "memory");  // widen_kernel's rows
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's barriers are set up before either CTA sends to the other
  tc_fence_after();
  line.s = aligned ? M.start_s : p.n_seg;
  line.a = M.start_a;
  const uint32_t tmem = M.tmem_slot;
  const uint32_t sbase = smem_u32(smem);
  volatile int* abort_v = &M.abort_flag;

  if (warp >= kSoftWarp0 && warp < kSoftWarp0 + kSoftWarps) {
    // -------------------------------------------------------------- softmax, results
    const int sw = warp - kSoftWarp0, quad = sw & 3, half = sw >> 2;
    const int row = quad * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t mx0 = smem_u32(&M.mx[0][0][0]), mxbar0 = smem_u32(&M.mx_full[0][0]);
    const uint32_t self_mx = peer_addr(mx0, rank), self_mxbar = peer_addr(mxbar0, rank);
    const uint32_t peer_mx = peer_addr(mx0, rank ^ 1), peer_mxbar = peer_addr(mxbar0, rank ^ 1);
    const uint32_t p_at = kOffP + half * kPHalf + quad * 2048;  // the warp's 32 rows of its half
    const uint32_t peer_p = peer_addr(sbase + kQChunk + p_at, rank ^ 1);
    const uint32_t peer_pbar = peer_addr(smem_u32(&M.vo_full), rank ^ 1);
    const bool writer = rank == 0 && sw == 0 && lane == 0;
    bool over = false;
    Line wline = line;
    Piece pc, nx;
    nx.s = 0;
    bool have = next_piece(p, M.ends, wline, nx, writer), started = false;
    if (have && half == 0) prefetch_q(p, nx.s, row);
    Tiles cur;  // one ahead of the tile that is worked on: its page ids have arrived when they are used
    cur.line = line;
    bool more = false;
    int own_next = -1;  // own page of the next tile to be worked on
    auto load_scale = [&] {  // scale of key 32 half + lane of the own page of tile `cur`
      const int own = Tiles::pool_page(p, cur.own_id);
      return own >= 0 ? __ldg(p.kv_scale + static_cast<long long>(own) * kPage + half * 32 + lane) : 0.0f;
    };
    float scale = 0.0f;
    uint32_t g = 0, sent = 0;  // tiles; exchanges between the warps of a row
    bool ok = true;
    Limits lim, next_lim;
    float m = 0.0f, l = 0.0f;
    // A value of a row from each of the four warps that hold the row (both halves,
    // both CTAs; own CTA's first), in the same order everywhere but for the CTA.
    auto exchange = [&](float value, float4& got) {
      const uint32_t par = sent & 1, bar = (par * 4 + quad) * 8;
      send_float(self_mx + ((par * 4 + half) * kRows + row) * 4, value, self_mxbar + bar);
      send_float(peer_mx + ((par * 4 + 2 + half) * kRows + row) * 4, value, peer_mxbar + bar);
      if (half == 0 && lane == 0) mbar_arrive_expect_tx(&M.mx_full[par][quad], 4 * 32 * 4);
      if (!wait_warp<true>(&M.mx_full[par][quad], (sent >> 1) & 1, abort_v)) return false;
      ++sent;
      const volatile float* v = &M.mx[par][0][row];
      got = make_float4(v[0], v[kRows], v[2 * kRows], v[3 * kRows]);
      return true;
    };
    while (ok) {
      // the next piece's Q while the last product of this one runs, then this one's results
      if (have) {
        if (F16 && !started) next_lim = limits(p, nx.s, row);
        const uint32_t live = F16 ? __ballot_sync(0xFFFFFFFFu, next_lim.hi > next_lim.lo) : 0;
        over |= load_q<FMT>(p, nx.s, smem + kOffQ, tmem + lanes + kColQ, rank, quad, half, live);
        if (lane == 0) mbar_arrive(&M.q_full);
      }
      if (started) {
        if (!wait_warp<true>(&M.pv_done, (g - 1) & 1, abort_v)) break;
        tc_fence_after();
        // a row that sees none of the segment's keys took part in the unmasked tiles: dropped here
        if (lim.hi <= lim.lo) l = 0.0f;
        const bool whole = pc.whole && p.n_rb == 0;  // no other piece has keys of these rows: their results
        if (whole) {
          float4 of;
          if (!exchange(l, of)) break;
          // summed in the same order by both CTAs
          const float sum = rank == 0 ? (of.x + of.y) + (of.z + of.w) : (of.z + of.w) + (of.x + of.y);
          const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
          const int i = pc.s, b = i / p.rb_s, r = (i - b * p.rb_s) * kRows + row;
          const bool exists = r < p.q_per_seq << p.hshift;
          const long long flat = (static_cast<long long>(b) * p.q_per_seq << p.hshift) + r;
          uint16_t* o = p.out + flat * kDv + 256 * rank + 128 * half;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float v[32];
            tmem_ld_32x32b_x32(tmem + lanes + kColO + 128 * half + 32 * c, reinterpret_cast<uint32_t*>(v));
            tmem_wait_ld();
            if (exists) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  w[k] = sum != 0.0f ? pack2(v[8 * j + 2 * k] * inv, v[8 * j + 2 * k + 1] * inv, false) : 0u;
                *reinterpret_cast<uint4*>(o + 32 * c + 8 * j) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
          if (exists && rank == 0 && half == 0 && p.lse) p.lse[flat] = sum != 0.0f ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
        } else {
          const int slot = piece_slot(p, pc.s, pair, pc.t0);
          float4* o = p.part_o + ((static_cast<long long>(slot) * 2 + rank) * 64 + half * 32) * kRows + row;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float v[32];
            tmem_ld_32x32b_x32(tmem + lanes + kColO + 128 * half + 32 * c, reinterpret_cast<uint32_t*>(v));
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j) o[(8 * c + j) * kRows] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          }
          if (rank == 0 && half == 0) p.part_m[static_cast<long long>(slot) * kRows + row] = m;
          p.part_l[(static_cast<long long>(slot) * 4 + 2 * rank + half) * kRows + row] = l;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&M.o_free);
      } else if (have) {
        if (!F16) next_lim = limits(p, nx.s, row);
        more = cur.next(p, M.ends, rank, true);
        own_next = Tiles::pool_page(p, cur.own_id);
        if (FMT == kTokenFp8) scale = load_scale();
        more = cur.next(p, M.ends, rank, false);
      }
      if (!have) break;
      started = true;
      pc = nx;
      lim = next_lim;
      const int first_page = pc.s < p.n_rb ? 0 : p.shared_len / kPage;
      m = -INFINITY, l = 0.0f;
      have = next_piece(p, M.ends, wline, nx, writer);
      if (have) {
        if (half == 0) prefetch_q(p, nx.s, row);
        next_lim = limits(p, nx.s, row);
      }
      for (int t = pc.t0; t < pc.t1; ++t, ++g) {
        const int tile_k = (first_page + 2 * t) * kPage, key0 = tile_k + rank * kPage + half * 32;
        const int own = own_next;
        if (FMT == kTokenFp8) {
          // Per-token scales multiply the logits, and the probabilities on their way to
          // V's codes, in fp32. A warp's 32 keys, loaded a tile ahead. (Keys that no row
          // of the block sees may have any scale: they count as 1. One that is not finite
          // reaches the rows that see its key through the logit alone: 0 * NaN.)
          const int key = key0 + lane;
          const float sc = key < lim.lo || key >= lim.max_hi ? 1.0f : scale;
          __syncwarp();
          reinterpret_cast<float*>(M.ks[sw])[lane] = sc;
          reinterpret_cast<float*>(M.vs[sw])[lane] = fabsf(sc) < INFINITY ? sc : 1.0f;
          __syncwarp();
          if (more) scale = load_scale();
        }
        own_next = more ? Tiles::pool_page(p, cur.own_id) : -1;
        if (more) more = cur.next(p, M.ends, rank, false);
        if (!wait_warp<false>(&M.s_full, g & 1, abort_v)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float x[32];
        tmem_ld_32x32b_x32(tmem + lanes + kColS + 32 * half, reinterpret_cast<uint32_t*>(x));
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&M.s_free);
        const bool edge = own < 0 || key0 < lim.lo || key0 + 32 > lim.min_hi;
        if (FMT == kTokenFp8) {
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 k = M.ks[sw][i >> 2];
            const float2 y = mul2(make_float2(x[i], x[i + 1]), make_float2(k.x, k.y));
            const float2 z = mul2(make_float2(x[i + 2], x[i + 3]), make_float2(k.z, k.w));
            x[i] = y.x, x[i + 1] = y.y, x[i + 2] = z.x, x[i + 3] = z.y;
          }
        }
        if (edge) {
          const int hi = own < 0 ? 0 : lim.hi;
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = key0 + i >= lim.lo && key0 + i < hi ? x[i] : -INFINITY;
        }
        float mine = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; i += 2) mine = max3(mine, x[i], x[i + 1]);
        mine *= p.scale_log2;
        // the row's maximum over both halves of both pages, which all scale P by the
        // same reference: every warp sends its rows' to both CTAs
        float4 of;
        if (!exchange(mine, of)) {
          ok = false;
          break;
        }
        const float top = fmaxf(fmaxf(of.x, of.y), fmaxf(of.z, of.w));
        const bool raise = top > m + kRaise || (m == -INFINITY && top > -INFINITY);
        float alpha = 1.0f;
        if (raise) {
          alpha = m == -INFINITY ? 0.0f : exp2_fast(m - top);
          m = top;
          l *= alpha;
        }
        const float ref = m == -INFINITY ? 0.0f : m;
        uint32_t pk[16];
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        const float2 factor = make_float2(p.scale_log2, p.scale_log2), minus = make_float2(-ref, -ref);
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 y = fma2(make_float2(x[i], x[i + 1]), factor, minus);
          float2 e = make_float2(exp2_fast(y.x), exp2_fast(y.y));
          sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], e);
          if (FMT == kTokenFp8) e = mul2(e, reinterpret_cast<const float2*>(M.vs[sw])[i >> 1]);
          // P is rounded to the operands' type (bf16: off by at most 2^-8 of a probability,
          // f16: 2^-11); the sum l is not
          pk[i >> 1] = pack2(e.x, e.y, F16);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        // both CTAs are done with the previous tile's P, and O holds it
        if (g > 0 && !wait_warp<true>(&M.pv_done, (g - 1) & 1, abort_v)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (t > pc.t0 && __any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(tmem + lanes + kColO + 128 * half + 32 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st_32x32b_x32(tmem + lanes + kColO + 128 * half + 32 * c, o);
          }
          tmem_wait_st();
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)  // 64-byte rows: piece j of row r sits at j ^ (r / 2 mod 4)
          *reinterpret_cast<uint4*>(smem + p_at + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
              make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
        // P goes to the other CTA first: the wait below is for its P as well
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) send_bulk(peer_p, sbase + p_at, 2048, peer_pbar);
        // 0 * NaN: V rows that no row of the block sees are zeroed, and rows that
        // only some see are zeroed if they hold a value that is not finite (those
        // that see it have a logit that is not finite either). Two chunks a half.
        if (tile_k < lim.lo || tile_k + 2 * kPage > lim.min_hi) {
          if (!wait_warp<false>(&M.kv_full[g & 1], (g >> 1) & 1, abort_v) || !wait_warp<true>(&M.vo_full, g & 1, abort_v)) {
            ok = false;
            break;
          }
          const bool oth = row >= kPage;
          const int r = row & (kPage - 1), key = tile_k + (oth ? rank ^ 1 : rank) * kPage + r;
          uint8_t* v = smem + (oth ? kOffVO : kOffKV + static_cast<int>(g & 1) * 4 * kChunk) + 2 * half * kChunk;
          bool zero = key < lim.lo || key >= lim.max_hi;
          if (!zero && key >= lim.min_hi) {
            constexpr uint32_t inf = F16 ? 0x7C00u : 0x7F80u;
            for (int j = 0; j < 16; ++j) {
              const uint4 u = *reinterpret_cast<const uint4*>(v + (j >> 3) * kChunk + piece_off(r, j & 7));
              const uint32_t e[4] = {u.x, u.y, u.z, u.w};
              for (int k = 0; k < 4; ++k) zero |= (e[k] & inf) == inf || (e[k] & (inf << 16)) == inf << 16;
            }
          }
          if (zero)
            for (int j = 0; j < 16; ++j)
              *reinterpret_cast<uint4*>(v + (j >> 3) * kChunk + piece_off(r, j & 7)) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&M.p_own);
        __syncwarp();
      }
    }
    if (over) set_status(&M.status, kStatusOverflow);
  } else if (warp == kTmaWarp) {
    // -------------------------------------------------------------- TMA loads
    if (elect_one()) {
      const int v0 = 4 * rank, k0 = 4 * (rank ^ 1);  // first chunk of this CTA's output values, of the others
      Tiles cur;
      cur.line = line;
      bool more = cur.next(p, M.ends, rank, true);
      // where a page's rows lie in the map: pool rows, or (FP8) rows of the shared part's
      // copy; -64 for a page that is missing: a box wholly before the rows reads as zeros
      auto place = [&](int id, int i) {
        if (FMT != kBf16) return id != Tiles::kNoPage ? (cur.first_page + 2 * cur.t + i) * kPage : -kPage;
        const int page = Tiles::pool_page(p, id);
        return page >= 0 ? page * kPage : -kPage;
      };
      auto load_vo = [&](uint32_t h, bool by_tma, int y) {
        if (h > 0 && !wait_one<false>(&M.vo_free, (h - 1) & 1, abort_v)) return false;
        if (FMT != kBf16 && !by_tma) {
          mbar_arrive(&M.vo_full);
          return true;
        }
        // V of the other page and (BF16; else a widening warp expects it) its P
        mbar_arrive_expect_tx(&M.vo_full, 4 * kChunk + (FMT == kBf16 ? kQChunk : 0));
        tma_chunks(smem + kOffVO, &kv_map, &M.vo_full, y, v0);
        return true;
      };
      uint32_t g = 0;
      bool ok = true, last_tma = false;
      int last_y = 0;
      if (FMT != kBf16) asm volatile("fence.proxy.async.global;" ::: "memory");  // the copy was written by plain stores
      if (more && p.q_tma) prefetch_tensormap(&q_map);
      for (; more && ok; ++g) {
        const bool by_tma = FMT == kBf16 || (p.wide && cur.pc.s < p.n_rb);
        const int y = place(cur.own_id, rank), other_y = place(cur.other_id, rank ^ 1);
        if (FMT == kBf16 && cur.bad(p, rank)) set_status(&M.status, kStatusBounds);
        const bool new_piece = cur.t == cur.pc.t0;
        int rows;
        const int q_row = static_cast<int>(first_row(p, cur.pc.s, rows));
        more = cur.next(p, M.ends, rank, false);
        if (g > 0 && !wait_one<false>(&M.ko_free, (g - 1) & 1, abort_v)) { ok = false; break; }
        if (by_tma) {
          mbar_arrive_expect_tx(&M.ko_full, 5 * kChunk);
          tma_chunks(smem + kOffKO, &kv_map, &M.ko_full, y, k0);
          tma_chunks(smem + kOffKO + 4 * kChunk, &rope_map, &M.ko_full, y, 8);
        } else {
          mbar_arrive(&M.ko_full);
        }
        const int buf = g & 1;
        if (g > 1 && !wait_one<false>(&M.kv_free[buf], ((g >> 1) - 1) & 1, abort_v)) { ok = false; break; }
        if (by_tma) {
          mbar_arrive_expect_tx(&M.kv_full[buf], 4 * kChunk);
          tma_chunks(smem + kOffKV + 4 * buf * kChunk, &kv_map, &M.kv_full[buf], y, v0);
        } else {
          mbar_arrive(&M.kv_full[buf]);
        }
        if (more && (FMT == kBf16 || (p.wide && cur.pc.s < p.n_rb))) {  // the next tile's own page into L2
          const int next = place(cur.own_id, rank);
          if (next >= 0) {
            prefetch_chunks(&kv_map, next, k0);
            prefetch_chunks(&rope_map, next, 8);
            prefetch_chunks(&kv_map, next, v0);
          }
        }
        if (g > 0) ok = load_vo(g - 1, last_tma, last_y);
        if (p.q_tma && new_piece) {  // its Q, once the logits of the piece before are complete
          if (g > 0 && !wait_one<false>(&M.s_full, (g - 1) & 1, abort_v)) { ok = false; break; }
          mbar_arrive_expect_tx(&M.q_full, 3 * kQChunk);
          tma_chunks(smem + kOffQ, &q_map, &M.q_full, q_row, 8);
          tma_chunks(smem + kOffQ + kQChunk, &q_map, &M.q_full, q_row, v0 + 2);
          tma_chunks(smem + kOffQ + 2 * kQChunk, &q_map, &M.q_full, q_row, v0 + 3);
        }
        last_tma = by_tma;
        last_y = other_y;
      }
      if (g > 0 && ok) load_vo(g - 1, last_tma, last_y);
    }
  } else if (warp == kMmaWarp) {
    // -------------------------------------------------------------- MMA issue
    // tcgen05.mma takes its descriptors from uniform registers. So the loop runs
    // warp-wide on warp-uniform values, each batch of MMAs is unrolled with constant
    // offsets and issued by one thread chosen with elect.sync (the compiler then
    // knows that one thread is active), and no call or wait stands inside a batch.
    // Measured on the issue alone, a tile's 44 MMAs: 2,376 cycles (back to back) in
    // this form; 4,185 under `if (lane == 0)`, where each MMA becomes a loop over
    // the active threads; about 3,300 with waits inside the batches.
    constexpr uint32_t id_qk = instr_desc(128, 64, kFmt, kFmt, false, false);
    constexpr uint32_t id_pv = instr_desc(128, 256, kFmt, kFmt, false, true);
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    const uint32_t sb = __shfl_sync(0xFFFFFFFFu, sbase, 0);
    const Operand q_desc = operand(sb + kOffQ, 16, 1024);
    const Operand ko_desc = operand(sb + kOffKO, 16, 1024);
    const Operand kv_desc = operand(sb + kOffKV, 16, 1024);
    const Operand v_desc = operand(sb + kOffKV, kChunk, 1024);   // the same chunks read as V: values x keys
    const Operand vo_desc = operand(sb + kOffVO, kChunk, 1024);
    const Operand p_desc = operand(sb + kOffP, 16, 512, kSwizzle64B);  // 32 keys a half: two K = 16 steps each
    const Operand po_desc = operand(sb + kOffP + kQChunk, 16, 512, kSwizzle64B);
    Line wline = line;
    Piece pc;
    uint32_t g = 0, n = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_poll<false>(bar, parity); };
    // logits of tile g
    auto qk = [&] {
      if (!wait(&M.ko_full, g & 1) || (g > 0 && !wait(&M.s_free, (g - 1) & 1))) return false;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts(tm + kColS, tm + kColQ + 32 * i + 8 * kk, ko_desc + (i * kChunk + 32 * kk), id_qk, i != 0 || kk != 0);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_ss(tm + kColS, q_desc + 32 * kk, ko_desc + (4 * kChunk + 32 * kk), id_qk, 1);
        mma_commit(&M.ko_free);
      }
      __syncwarp();
      if (!wait(&M.kv_full[g & 1], (g >> 1) & 1)) return false;
      tc_fence_after();
      if (elect_one()) {
        const Operand kd = kv_desc + static_cast<int>(g & 1) * 4 * kChunk;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_ts(tm + kColS, tm + kColQ + 128 + 32 * i + 8 * kk, kd + (i * kChunk + 32 * kk), id_qk, 1);
#pragma unroll
        for (int i = 2; i < 4; ++i)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss(tm + kColS, q_desc + ((i - 1) * kQChunk + 32 * kk), kd + (i * kChunk + 32 * kk), id_qk, 1);
        mma_commit(&M.s_full);
      }
      __syncwarp();
      ++g;
      return true;
    };
    // O (+)= P V of tile h, own page first: its V slots are the next to be refilled
    auto pv = [&](uint32_t h, uint32_t first) {
      if (!wait(&M.p_own, h & 1) || (first && n > 0 && !wait(&M.o_free, (n - 1) & 1))) return false;
      tc_fence_after();
      if (elect_one()) {
        const Operand v = v_desc + static_cast<int>(h & 1) * 4 * kChunk;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ss(tm + kColO, p_desc + ((kk >> 1) * kPHalf + 32 * (kk & 1)), v + kk * 2048, id_pv, kk != 0 ? 1 : first ^ 1);
        mma_commit(&M.kv_free[h & 1]);
      }
      __syncwarp();
      if (!wait_poll<true>(&M.vo_full, h & 1)) return false;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ss(tm + kColO, po_desc + ((kk >> 1) * kPHalf + 32 * (kk & 1)), vo_desc + kk * 2048, id_pv, 1);
        mma_commit(&M.vo_free);
        commit_pair(&M.pv_done);
      }
      __syncwarp();
      return true;
    };
    while (ok && next_piece(p, M.ends, wline, pc, false)) {
      if (!wait(&M.q_full, n & 1)) { ok = false; break; }
      const int t0 = __shfl_sync(0xFFFFFFFFu, pc.t0, 0), t1 = __shfl_sync(0xFFFFFFFFu, pc.t1, 0);
      // the logits of a tile are issued before the product of the tile before it
      ok = qk();
      for (int t = t0 + 1; ok && t < t1; ++t) ok = qk() && pv(g - 2, t - 1 == t0);
      ok = ok && pv(g - 1, t1 - 1 == t0);
      ++n;
    }
    if (!ok) *abort_v = 2;
  } else if (FMT != kBf16) {
    // -------------------------------------------------------------- FP8 rows: load, widen, store
    // Two warps for each of KO (2, 3), KV (12, 13) and VO (14, 15). Thread u takes
    // 16 codes of rows u / 4 + 16 i in every chunk (four lanes on a row's 64
    // contiguous bytes); a tile's pieces are loaded while the tile before is waited
    // for. Per-token codes are exact in bf16; tile-scaled values (code * scale) are
    // rounded to f16: off by at most 2^-11 of the value (at least 2^-25). Tile-scaled
    // rows that no row of the segment sees count as zeros: their values may be outside
    // f16's range.
    const int cw = warp < kSoftWarp0 ? warp - 2 : warp - 10;
    const int group = cw >> 1;  // 0 KO, 1 KV, 2 VO
    const int u = (cw & 1) * 32 + lane, r0 = u >> 2, pcs = u & 3;
    constexpr int kRowBytes = FMT == kTokenFp8 ? kDqk : kTileRowBytes;
    const int c0 = group == 0 ? 4 * (rank ^ 1) : 4 * rank;
    bool over = false;
    float top = 0.0f;
    uint4 v[5][4];   // chunks of four rows; the fifth (KO) is the rope (tile-scaled rows: loaded when it is stored)
    const uint8_t* rope = nullptr;
    float2 sc[4];    // scales of the two 128-value tiles that the four chunks cover
    uint32_t seen = 0;  // which of the four rows (tile-scaled)
    auto fetch = [&](int page, int key0, int first_key, int end_key) {
      const uint8_t* src = p.kv + (static_cast<long long>(max(page, 0)) * kPage + r0) * kRowBytes;
      const uint4 none = make_uint4(0, 0, 0, 0);
      seen = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key0 + r0 + 16 * i;
        const bool live = page >= 0 && (FMT != kTileFp8 || (key >= first_key && key < end_key));
        const uint8_t* row = src + i * 16 * kRowBytes;
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c][i] = live ? __ldg(reinterpret_cast<const uint4*>(row + (c0 + c) * 64 + pcs * 16)) : none;
        if (FMT == kTileFp8) sc[i] = live ? __ldg(reinterpret_cast<const float2*>(row + kDv) + (c0 >> 2)) : make_float2(0, 0);
        if (FMT == kTokenFp8 && group == 0) v[4][i] = live ? __ldg(reinterpret_cast<const uint4*>(row + kDv + pcs * 16)) : none;
        if (FMT == kTileFp8 && live) {
          seen |= 1u << i;
          if (group == 0 && pcs == 0) prefetch_l2_lines(row + kTileRope, 128);
        }
      }
      if (FMT == kTileFp8 && group == 0) rope = src + kTileRope + pcs * 32;
    };
    auto store = [&](int off) {
#pragma unroll
      for (int c = 0; c < 5; ++c) {
        if (c == 4 && group != 0) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = r0 + 16 * i;
          uint8_t* dst = smem + off + c * kChunk;
          uint32_t o[8];
          if (FMT == kTileFp8 && c == 4) {  // bf16 rope -> f16
            const uint4 none = make_uint4(0, 0, 0, 0);
            const bool live = seen >> i & 1;
            const uint4 a = live ? __ldg(reinterpret_cast<const uint4*>(rope + i * 16 * kRowBytes)) : none;
            const uint4 b = live ? __ldg(reinterpret_cast<const uint4*>(rope + i * 16 * kRowBytes + 16)) : none;
            o[0] = to_f16(a.x, over), o[1] = to_f16(a.y, over), o[2] = to_f16(a.z, over), o[3] = to_f16(a.w, over);
            o[4] = to_f16(b.x, over), o[5] = to_f16(b.y, over), o[6] = to_f16(b.z, over), o[7] = to_f16(b.w, over);
          } else {
            const uint32_t w[4] = {v[c][i].x, v[c][i].y, v[c][i].z, v[c][i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint16_t lo = static_cast<uint16_t>(w[k]), hi = static_cast<uint16_t>(w[k] >> 16);
              o[2 * k] = F16 ? e4m3x2(lo) : e4m3x2_bf16(lo);
              o[2 * k + 1] = F16 ? e4m3x2(hi) : e4m3x2_bf16(hi);
            }
            if (FMT == kTileFp8) {
              const float s = c < 2 ? sc[i].x : sc[i].y;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&o[k]));
                const float a = f.x * s, b = f.y * s;
                top = fmaxf(top, fmaxf(fabsf(a), fabsf(b)));
                o[k] = pack2(a, b, true);
              }
            }
          }
          *reinterpret_cast<uint4*>(dst + piece_off(r, 2 * pcs)) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(dst + piece_off(r, 2 * pcs + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
    };
    Tiles cur;
    cur.line = line;
    bool more = cur.next(p, M.ends, rank, true);
    auto mine = [&] { return !(p.wide && cur.pc.s < p.n_rb); };  // not a tile of the copy
    bool here = more && mine();
    auto fetch_tile = [&] {
      const int side = group == 2 ? rank ^ 1 : rank;
      fetch(Tiles::pool_page(p, group == 2 ? cur.other_id : cur.own_id), (cur.first_page + 2 * cur.t + side) * kPage, cur.first_key, cur.end_key);
    };
    if (here) fetch_tile();
    for (uint32_t g = 0; more; ++g) {
      const bool stores = here;
      if (group == 0 && cur.bad(p, rank) && lane == 0) set_status(&M.status, kStatusBounds);
      more = cur.next(p, M.ends, rank, false);
      here = more && mine();
      // the slots' previous tile: g - 1, or g - 2 for KV's two buffers
      const uint32_t back = group == 1 ? 2 : 1;
      if (g >= back) {
        uint64_t* bar = group == 0 ? &M.ko_free : group == 1 ? &M.kv_free[g & 1] : &M.vo_free;
        if (!wait_warp<false>(bar, group == 1 ? ((g >> 1) - 1) & 1 : (g - 1) & 1, abort_v)) break;
      }
      if (stores) {
        store(group == 0 ? kOffKO : group == 1 ? kOffKV + static_cast<int>(g & 1) * 4 * kChunk : kOffVO);
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) {
        if (cw == 4) mbar_arrive_expect_tx(&M.vo_full, kQChunk);  // and the other page's P
        else mbar_arrive(group == 0 ? &M.ko_full : group == 1 ? &M.kv_full[g & 1] : &M.vo_full);
      }
      if (here) fetch_tile();
    }
    if (over || top > 65504.0f) set_status(&M.status, kStatusOverflow);
  }

  __syncwarp();
  if (*abort_v == 2) set_status(&M.status, kStatusTimeout);
  if (*abort_v) {  // a wait gave up: let copies that are still under way land before the memory goes
    const long long t0 = clock64();
    while (clock64() - t0 < 4000000) __nanosleep(1000);
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0) p.errors[blockIdx.x] = M.status;
  cluster_sync();  // the peer may still read or signal this CTA's shared memory until here
  if (warp == kTmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ the shared rows, widened
// The shared pages' rows in logical order, as the MMAs take them: per-token codes in
// bf16, exactly; tile-scaled values (code * scale) in f16, rounded (off by at most
// 2^-11 of the value). Four blocks a page, which read 37 or 42 KB and write 74 KB:
// bound by memory and, for short prompts, by latency (7.5 us for 16K tokens, 29 MB,
// 3.8 TB/s; 4.2 us for 5K). Each row block of the batch would widen them again
// otherwise: 64 x 2 tokens of 64 heads on 16K per-token rows (64 row blocks), 382 us
// against 253 with the copy; 37 x 2 of 16 heads on 5K tile-scaled rows (10 row
// blocks) 72 against 69.
template <int FMT>
__global__ void __launch_bounds__(256) widen_kernel(const PrefixParams p) {
  constexpr int kRowBytes = FMT == kTokenFp8 ? kDqk : kTileRowBytes;
  constexpr int kPieces = FMT == kTokenFp8 ? kDqk / 16 : kDv / 16 + 8;  // 16 codes each, then (tile-scaled) 8 rope values
  asm volatile("griddepcontrol.launch_dependents;");  // prefix_kernel may set up; it waits for the rows
  const int id = p.page_tables[blockIdx.x];
  const bool live = id >= 0 && id < p.num_pages;
  constexpr int kPart = kPage / 4;
  const uint8_t* src = p.kv + (static_cast<long long>(live ? id : 0) * kPage + blockIdx.y * kPart) * kRowBytes;
  uint16_t* dst = p.wide_rows + (static_cast<long long>(blockIdx.x) * kPage + blockIdx.y * kPart) * kDqk;
  __shared__ uint32_t over_keys;
  if (FMT == kTileFp8) {
    if (threadIdx.x == 0) over_keys = 0;
    __syncthreads();
  }
#pragma unroll 4
  for (int u = threadIdx.x; u < kPart * kPieces; u += 256) {
    const int r = u / kPieces, j = u - r * kPieces;
    const uint8_t* row = src + r * kRowBytes;
    uint16_t* out = dst + r * kDqk;
    bool over = false;
    float top = 0.0f;
    if (FMT == kTileFp8 && j >= kDv / 16) {
      const int i = j - kDv / 16;
      const uint4 w = live ? __ldg(reinterpret_cast<const uint4*>(row + kTileRope + 16 * i)) : make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(out + kDv + 8 * i) = make_uint4(to_f16(w.x, over), to_f16(w.y, over), to_f16(w.z, over), to_f16(w.w, over));
      if (over) atomicOr(&over_keys, 1u << r);
      continue;
    }
    const uint4 c = live ? __ldg(reinterpret_cast<const uint4*>(row + 16 * j)) : make_uint4(0, 0, 0, 0);
    const float s = FMT == kTileFp8 && live ? __ldg(reinterpret_cast<const float*>(row + kDv) + (j >> 3)) : 1.0f;
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint16_t pair = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
      o[k] = FMT == kTileFp8 ? e4m3x2(pair) : e4m3x2_bf16(pair);
      if (FMT == kTileFp8) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&o[k]));
        top = fmaxf(top, fmaxf(fabsf(f.x * s), fabsf(f.y * s)));
        o[k] = pack2(f.x * s, f.y * s, true);
      }
    }
    *reinterpret_cast<uint4*>(out + 16 * j) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(out + 16 * j + 8) = make_uint4(o[4], o[5], o[6], o[7]);
    if (FMT == kTileFp8 && top > 65504.0f) atomicOr(&over_keys, 1u << r);
  }
  if (FMT == kTileFp8) {
    __syncthreads();
    if (threadIdx.x == 0) reinterpret_cast<uint32_t*>(p.wide_over)[4 * blockIdx.x + blockIdx.y] = over_keys;
  }
}

// ------------------------------------------------------------------ joining the pieces
// A block joins 128 output values of 16 rows (one token's heads or part of them):
// the pieces of the rows' shared segment and of their own one, weighted by
// 2^(m - largest m). Reading fp32 partials that were just written, it is bound by
// L2 and, for few rows, by latency: up to four blocks share a row's values, and each
// thread keeps eight 16-byte loads in flight. It ends 20 us after prefix_kernel for
// 8,192 rows of three or four pieces, 9 us after it for 1,184 rows, 5 us for 64.
__device__ __forceinline__ float piece_sum(const PrefixParams& p, int slot, int at) {
  const float* l = p.part_l + static_cast<long long>(slot) * 4 * kRows + at;
  return (l[0] + l[kRows]) + (l[2 * kRows] + l[3 * kRows]);
}

constexpr int kMergeRows = 16, kMergeCols = 128, kMergeThreads = 256;

__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const PrefixParams p) {
  __shared__ int slots[kMaxPieces];       // slot * 128 + the rows' place in the block
  __shared__ float wgt[kMaxPieces][kMergeRows], sums[kMaxPieces][kMergeRows];
  __shared__ float inv[kMergeRows];
  __shared__ long long bounds[kMaxPairs + 1];
  __shared__ uint32_t warp_bits[kMergeThreads / 32];
  __shared__ __align__(16) uint16_t o[kMergeRows][kMergeCols];
  __shared__ int s_n;
  const int tid = threadIdx.x, lane = tid & 31;
  const int r0 = blockIdx.x * kMergeRows;
  // what does not depend on the pieces, then wait until they are written
  int seg[2], at[2], tiles[2];  // the rows' shared and own segment
  {
    const int per = p.q_per_seq << p.hshift, b = r0 / per, in = r0 - b * per;
    seg[0] = r0 / kRows, at[0] = r0 % kRows;
    seg[1] = p.n_rb + b * p.rb_s + in / kRows, at[1] = in % kRows;
    tiles[0] = p.n_rb > 0 ? shared_tiles(shared_end(p, seg[0] >> p.end_shift)) : 0;
    tiles[1] = own_tiles(p, own_end(p, seg[1] - p.n_rb));
  }
  const bool reports = blockIdx.x == 0 && blockIdx.y == 0;  // the call's status
  int seen = 0;  // keys of the shared part that some row sees
  if (reports && p.wide_over) {
#pragma unroll 4
    for (int b = tid; b < p.n_seqs; b += kMergeThreads) seen = max(seen, length_of(p, b));
    seen = __reduce_max_sync(0xFFFFFFFFu, seen);
    if (lane == 0) warp_bits[tid >> 5] = seen;
    __syncthreads();
    for (int w = 0; w < kMergeThreads / 32; ++w) seen = max(seen, static_cast<int>(warp_bits[w]));
    seen = min(seen, p.shared_len);
    __syncthreads();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long own_at = tiles[1] > 0 ? p.seg_off[seg[1]] : 0, shared_at = tiles[0] > 0 ? p.seg_off[seg[0]] : 0;
  const bool done = own_at < 0;
  if (done && blockIdx.x != 0) return;
  for (int q = tid; q <= p.pairs; q += kMergeThreads) bounds[q] = p.bounds[q];
  if (reports) {
    uint32_t bits = 0;
    for (int q = tid; q < 2 * p.pairs; q += kMergeThreads) bits |= p.errors[q];
    if (p.wide_over) {
#pragma unroll 4
      for (int i = tid; i < 4 * ((seen + kPage - 1) / kPage); i += kMergeThreads) {  // 16 keys each
        const uint32_t over = reinterpret_cast<const uint32_t*>(p.wide_over)[i];
        const int n = seen - 16 * i;
        if (n > 0 && (over & ((1u << min(n, 16)) - 1))) bits |= kStatusOverflow;
      }
    }
    bits = __reduce_or_sync(0xFFFFFFFFu, bits);
    if (lane == 0) warp_bits[tid >> 5] = bits;
  }
  __syncthreads();
  if (reports && tid == 0) {
    uint32_t bits = 0;
    for (int w = 0; w < kMergeThreads / 32; ++w) bits |= warp_bits[w];
    *p.status = bits;
  }
  if (done) return;
  if (tid < 32) {
    int n = 0;
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      if (tiles[part] == 0) continue;
      const int s = seg[part];
      const long long a = part == 1 ? own_at : shared_at;
      for (int base = 0; base < p.pairs; base += 32) {
        const int q = base + lane;
        int t0 = 0, t1 = 0;
        if (q < p.pairs) stretch_tiles(p, s, tiles[part], a, bounds[q], bounds[q + 1], t0, t1);
        const bool in = t1 > t0;
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, in);
        const int at_n = n + __popc(mask & ((1u << lane) - 1));
        if (in && at_n < kMaxPieces) slots[at_n] = piece_slot(p, s, q, t0) * kRows + at[part];
        n += __popc(mask);
      }
    }
    if (lane == 0) s_n = min(n, kMaxPieces);
  }
  __syncthreads();
  const int n = s_n;
  {  // 16 threads per row
    const int row = tid >> 4, k = tid & 15;
    float top = -INFINITY;
    for (int i = k; i < n; i += 16) {
      const int slot = slots[i] / kRows, at = slots[i] % kRows + row;
      const float l = piece_sum(p, slot, at);
      const float m = p.part_m[static_cast<long long>(slot) * kRows + at];
      // a row that saw nothing in a piece (l = 0) has nothing there, whatever its O holds
      wgt[i][row] = m;
      sums[i][row] = l;
      if (l != 0.0f) top = fmaxf(top, m);
    }
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    float sum = 0.0f;
    for (int i = k; i < n; i += 16) {
      const float l = sums[i][row];
      const float w = l != 0.0f ? exp2_fast(wgt[i][row] - top) : -1.0f;  // -1: nothing to add
      wgt[i][row] = w;
      if (l != 0.0f) sum += w * l;
    }
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    if (k == 0) {
      inv[row] = sum != 0.0f ? 1.0f / sum : 0.0f;
      if (p.lse && blockIdx.y == 0) p.lse[r0 + row] = sum != 0.0f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
    }
  }
  __syncthreads();
  const int row = tid & 15, c0 = tid >> 4;  // two groups of four values: c0 and c0 + 16 of the 32
#pragma unroll 1
  for (int cols = blockIdx.y * kMergeCols; cols < kDv; cols += gridDim.y * kMergeCols) {
    float4 acc[2] = {make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0)};
    const float4* part = p.part_o + static_cast<long long>(cols / 4 + c0) * kRows + row;
    for (int i0 = 0; i0 < n; i0 += 4) {
      float4 v[4][2];
      float w[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        w[u] = i0 + u < n ? wgt[i0 + u][row] : -1.0f;
        if (w[u] != -1.0f) {
          const int slot = slots[i0 + u] / kRows, at = slots[i0 + u] % kRows;
          const float4* src = part + static_cast<long long>(slot) * 2 * 64 * kRows + at;
          v[u][0] = src[0];
          v[u][1] = src[16 * kRows];
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (w[u] != -1.0f) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[j].x += w[u] * v[u][j].x, acc[j].y += w[u] * v[u][j].y, acc[j].z += w[u] * v[u][j].z, acc[j].w += w[u] * v[u][j].w;
        }
    }
    const float f = inv[row];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      *reinterpret_cast<uint2*>(&o[row][4 * (c0 + 16 * j)]) =
          make_uint2(pack2(acc[j].x * f, acc[j].y * f, false), pack2(acc[j].z * f, acc[j].w * f, false));
    __syncthreads();
    {
      const int r = tid >> 4, j = tid & 15;
      *reinterpret_cast<uint4*>(p.out + static_cast<long long>(r0 + r) * kDv + cols + 8 * j) = *reinterpret_cast<const uint4*>(&o[r][8 * j]);
    }
    __syncthreads();
  }
}

template <int FMT>
bool set_smem() {
  return cudaFuncSetAttribute(prefix_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes)) == cudaSuccess;
}

template <int FMT>
int launch(const CUtensorMap& map, const CUtensorMap& rope, const CUtensorMap& q, const PrefixParams& p, cudaStream_t st) {
  // each kernel but the call's first is set up while the one before runs, and waits for it itself
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * p.pairs);
  cfg.blockDim = dim3(kThreadsOf<FMT>);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cfg.attrs = &at, cfg.numAttrs = p.wide ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, prefix_kernel<FMT>, map, rope, q, p) != cudaSuccess) return SMLA_ERR_CUDA;
  cfg = cudaLaunchConfig_t{};
  // few rows: four blocks share a row's values; from 1,024 blocks on the GPU is full without
  cfg.gridDim = dim3(p.n_rows / kMergeRows, p.n_rows / kMergeRows < 1024 ? kDv / kMergeCols : 1);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = st;
  cfg.attrs = &at, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, merge_kernel, p) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

template <int FMT>
int resident_pairs() {
  if (!set_smem<FMT>()) return 0;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = 2, at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * num_sms());
  cfg.blockDim = dim3(kThreadsOf<FMT>);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.attrs = &at, cfg.numAttrs = 1;
  int n = 0;
  return cudaOccupancyMaxActiveClusters(&n, prefix_kernel<FMT>, &cfg) == cudaSuccess ? n : 0;
}

// CTA pairs that run at the same time (76 on a 152-SM part; fewer than half of the
// SMs where a GPC has an odd number of them: a pair too many would start when the
// others end). Looked up once per device, with the kernels' shared memory limit set.
int pairs_of_device() {
  static std::mutex mutex;
  static int known[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  std::lock_guard<std::mutex> lock(mutex);
  if (known[dev] == 0) {
    const int n = std::min({resident_pairs<kBf16>(), resident_pairs<kTokenFp8>(), resident_pairs<kTileFp8>()});
    known[dev] = std::max(1, std::min(n > 0 ? n : num_sms() / 2, kMaxPairs));
  }
  return known[dev];
}

// Rows of 576 16-bit values as [9 chunks][rows][64 values], loaded in boxes of
// `box_rows` rows and `chunks` chunks, each chunk 128-byte swizzled.
bool encode_chunks(CUtensorMap* map, const void* base, uint64_t rows, uint32_t box_rows, uint32_t chunks) {
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
  const cuuint64_t dims[3] = {64, rows, kDqk / 64}, strides[2] = {kDqk * 2, 128};
  const cuuint32_t box[3] = {64, box_rows, chunks}, steps[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

Costs costs_of(int32_t kv_dtype, bool wide) {
  if (kv_dtype == SMLA_BF16) return {20, 4, 4};
  const int own = kv_dtype == SMLA_FP8_E4M3 ? 7 : 10;
  return {kv_dtype == SMLA_FP8_E4M3 ? 40 : 34, wide ? 4 : own, own};
}

// Row blocks and segments; false: more than 32-bit counts hold.
bool plan(PrefixParams& p) {
  if (p.n_seqs == 1) p.shared_len = 0;  // its table is row 0: one segment per row block instead of two
  const int64_t rows = static_cast<int64_t>(p.n_seqs) * p.q_per_seq << p.hshift;
  const int64_t rb_s = ((static_cast<int64_t>(p.q_per_seq) << p.hshift) + kRows - 1) / kRows;
  const int64_t n_rb = p.shared_len > 0 ? (rows + kRows - 1) / kRows : 0;
  const int64_t n_seg = n_rb + rb_s * p.n_seqs;
  if (rows > INT32_MAX - kRows || (n_seg + kMaxPieces) * kRows > INT32_MAX) return false;
  p.n_rows = static_cast<int32_t>(rows);
  p.rb_s = static_cast<int32_t>(rb_s);
  p.n_rb = static_cast<int32_t>(n_rb);
  p.end_shift = 0;
  while (((n_rb - 1) >> p.end_shift) >= kGroups) ++p.end_shift;
  p.n_groups = n_rb > 0 ? static_cast<int32_t>((n_rb - 1) >> p.end_shift) + 1 : 0;
  p.n_seg = static_cast<int32_t>(n_seg);
  p.pairs = pairs_of_device();
  return true;
}

size_t layout(PrefixParams& p, uint8_t* ws, int32_t kv_dtype) {
  p.pair_slots = p.n_rb == 0 && p.n_seg > p.pairs;
  const size_t slots = static_cast<size_t>(p.pair_slots ? p.pairs : p.n_seg) + p.pairs;
  size_t at = kStatusBytes;
  p.bounds = reinterpret_cast<long long*>(ws + at);
  at += up256((static_cast<size_t>(p.pairs) + 1) * 8);
  p.errors = reinterpret_cast<uint32_t*>(ws + at);
  at += up256(static_cast<size_t>(p.pairs) * 2 * 4);
  p.seg_off = reinterpret_cast<long long*>(ws + at);
  at += up256(static_cast<size_t>(p.n_seg) * 8);
  p.part_m = reinterpret_cast<float*>(ws + at);
  at += slots * kRows * 4;
  p.part_l = reinterpret_cast<float*>(ws + at);
  at += slots * 4 * kRows * 4;
  p.part_o = reinterpret_cast<float4*>(ws + at);
  at += slots * 2 * 64 * kRows * 16;
  p.wide = kv_dtype != SMLA_BF16 && p.n_rb >= 2;
  p.costs = costs_of(kv_dtype, p.wide);
  if (p.wide) {
    p.wide_rows = reinterpret_cast<uint16_t*>(ws + at);
    const size_t pages = (static_cast<size_t>(p.shared_len) + kPage - 1) / kPage;
    at += pages * kPage * kDqk * 2;
    if (kv_dtype == SMLA_FP8_DS_MLA) p.wide_over = reinterpret_cast<uint4*>(ws + at);
    at += pages * sizeof(uint4);
  }
  return at;
}

}  // namespace
}  // namespace smla

using namespace smla;

extern "C" {

size_t smla_shared_prefix_fwd_workspace_size(int32_t n_seqs, int32_t max_seq_len, int32_t shared_len,
                                             int32_t q_per_seq, int32_t n_heads, int32_t kv_dtype) {
  if (n_seqs <= 0 || q_per_seq <= 0 || max_seq_len <= 0 || shared_len < 0 || (n_heads != 16 && n_heads != 64)) return kStatusBytes;
  PrefixParams p{};
  p.n_seqs = n_seqs, p.q_per_seq = q_per_seq, p.shared_len = shared_len, p.hshift = n_heads == 64 ? 6 : 4;
  if (!plan(p)) return kStatusBytes;
  return layout(p, nullptr, kv_dtype);
}

int smla_shared_prefix_fwd(const smla_paged_cache* cache, const int32_t* page_tables, int32_t max_pages,
                           int32_t n_seqs, const int32_t* seq_lens, int32_t max_seq_len, int32_t shared_len,
                           int32_t q_per_seq, const void* q, int32_t n_heads, float sm_scale, void* out, float* lse,
                           void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_serve_cache(cache, true, false);
  if (rc) return rc;
  if (!page_tables || !seq_lens || !q || !out || !aligned_to(page_tables, 4) || !aligned_to(seq_lens, 4) || !aligned_to(q, 16) || !aligned_to(out, 16) || !aligned_to(lse, 4))
    return SMLA_ERR_INVALID_ARG;
  if (n_seqs <= 0 || q_per_seq <= 0 || max_pages <= 0 || max_seq_len <= 0 || shared_len < 0 || shared_len > max_seq_len)
    return SMLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(max_pages) * kPage < max_seq_len || !(sm_scale == sm_scale)) return SMLA_ERR_INVALID_ARG;
  if (n_heads != 16 && n_heads != 64) return SMLA_ERR_UNSUPPORTED;
  if (max_seq_len > INT32_MAX - 4 * kPage) return SMLA_ERR_UNSUPPORTED;  // key positions of a tile are int32
  PrefixParams p{};
  p.n_seqs = n_seqs, p.q_per_seq = q_per_seq, p.shared_len = shared_len, p.hshift = n_heads == 64 ? 6 : 4;
  if (!plan(p)) return SMLA_ERR_UNSUPPORTED;
  if (!workspace || !aligned_to(workspace, 16) || workspace_bytes < layout(p, static_cast<uint8_t*>(workspace), cache->kv_dtype)) return SMLA_ERR_WORKSPACE;
  p.kv = static_cast<const uint8_t*>(cache->kv), p.kv_scale = cache->kv_scale, p.num_pages = cache->num_pages;
  p.page_tables = page_tables, p.max_pages = max_pages, p.seq_lens = seq_lens, p.max_seq_len = max_seq_len;
  p.q = static_cast<const uint16_t*>(q);
  // the logits' scale as a positive factor: the maximum can be taken before it
  p.scale_log2 = std::max(std::fabs(sm_scale) * 1.4426950408889634f, 1e-37f);
  p.q_sign = sm_scale < 0.0f ? 0x80008000u : 0u;
  p.out = static_cast<uint16_t*>(out), p.lse = lse;
  p.status = static_cast<uint32_t*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  CUtensorMap map{}, rope{}, q_map{};
  const bool bf16 = cache->kv_dtype == SMLA_BF16, token = cache->kv_dtype == SMLA_FP8_E4M3;
  if (bf16 || p.wide) {  // (16-bit values of either type)
    const int pages = (p.shared_len + kPage - 1) / kPage;
    const void* base = bf16 ? cache->kv : p.wide_rows;
    const uint64_t rows = static_cast<uint64_t>(bf16 ? cache->num_pages : pages) * kPage;
    if (!encode_chunks(&map, base, rows, kPage, 4) || !encode_chunks(&rope, base, rows, kPage, 1)) return SMLA_ERR_CUDA;
    if (!bf16) {
      if (token) widen_kernel<kTokenFp8><<<dim3(pages, 4), 256, 0, st>>>(p);
      else widen_kernel<kTileFp8><<<dim3(pages, 4), 256, 0, st>>>(p);
      if (cudaGetLastError() != cudaSuccess) return SMLA_ERR_CUDA;
    }
  }
  p.q_tma = cache->kv_dtype != SMLA_FP8_DS_MLA && p.q_sign == 0;
  p.q_sectors = aligned_to(q, 32);
  if (p.q_tma && !encode_chunks(&q_map, q, static_cast<uint64_t>(p.n_rows), kRows, 1)) return SMLA_ERR_CUDA;
  if (bf16) return launch<kBf16>(map, rope, q_map, p, st);
  return token ? launch<kTokenFp8>(map, rope, q_map, p, st) : launch<kTileFp8>(map, rope, q_map, p, st);
}

}  // extern "C"
