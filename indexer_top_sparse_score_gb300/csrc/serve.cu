// Serving steps around the paged cache: block tables and slot maps
// (smla_build_tables), new rows into the cache (smla_cache_append), queries
// (smla_query_prep). All three move little or stream their data once, so their
// floors are launch latency (decode-sized calls) and memory bandwidth
// (prefill-sized calls).
#include <cfloat>
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/smla_serve.h"
#include "common.cuh"
#include "internal.h"

namespace smla {
namespace {

// ---------------------------------------------------------------------------- tables
constexpr int kTabThreads = 256;

struct TablesParams {
  const int32_t* ctx;
  const int32_t* add;
  int32_t n_seqs, max_pages;
  int32_t* tables;
  const int32_t* free_pages;
  int32_t n_free, max_new;
  int32_t *seq_lens, *cu, *positions, *slots, *row_seq, *pages_used;
  uint32_t* status;
  int32_t rows_per_block;
};

// Inclusive sum over the block's threads; every thread also gets the total.
__device__ __forceinline__ long long block_scan(long long v, long long* warp_sums, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();  // the previous use of warp_sums is over
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kTabThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  return v + before;
}

// Every block scans all requests' lengths (a few KB that stay in L2; no block
// waits for another, so one launch does the whole job) and writes the rows
// [first, last) of the per-token outputs that are its share; block 0 also
// writes the per-request outputs and the status word, which needs no clearing
// launch because block 0 sees every condition that can set it.
__global__ void __launch_bounds__(kTabThreads) build_tables_kernel(const TablesParams p) {
  __shared__ long long warp_sums[kTabThreads / 32];
  __shared__ int s_cu[kTabThreads + 1];   // first row of each request of the chunk
  __shared__ int s_ctx[kTabThreads];      // its tokens so far
  __shared__ int s_got[kTabThreads];      // new tokens that have a slot
  __shared__ long long s_free[kTabThreads];  // where its pages begin in the free list
  const int tid = threadIdx.x;
  const bool lead = blockIdx.x == 0;
  const long long first_row = static_cast<long long>(blockIdx.x) * p.rows_per_block;
  const long long last_row = min(first_row + p.rows_per_block, static_cast<long long>(p.max_new));
  long long rows_before = 0, pages_before = 0;  // of the chunks before this one
  uint32_t bad = 0;
  for (int c0 = 0; c0 < p.n_seqs; c0 += kTabThreads) {
    const int b = c0 + tid;
    long long ctx = 0, add = 0;
    bool valid = true;
    if (b < p.n_seqs) {
      ctx = p.ctx[b];
      add = p.add[b];
      valid = ctx >= 0 && add >= 0 && ctx + add <= static_cast<long long>(p.max_pages) * kPage;
      if (!valid) ctx = add = 0;
    }
    long long rows_total, pages_total;
    const long long upto = rows_before + block_scan(add, warp_sums, rows_total);
    const int cu1 = static_cast<int>(min(upto, static_cast<long long>(p.max_new)));
    const int cu0 = static_cast<int>(min(upto - add, static_cast<long long>(p.max_new)));
    if (cu1 - cu0 < add) bad = kStatusBounds;
    add = cu1 - cu0;
    const long long held = (ctx + kPage - 1) / kPage;
    const long long need = (ctx + add + kPage - 1) / kPage - held;
    const long long pages_to = pages_before + block_scan(need, warp_sums, pages_total);
    const long long at = pages_to - need;
    const long long given = max(0LL, min(need, static_cast<long long>(p.n_free) - at));
    long long got = min(add, (held + given) * kPage - ctx);
    if (!valid || got < add) bad = kStatusBounds;
    s_cu[tid] = cu0;
    if (tid == kTabThreads - 1) s_cu[kTabThreads] = cu1;
    s_ctx[tid] = static_cast<int>(ctx);
    s_got[tid] = static_cast<int>(got);
    s_free[tid] = at;
    if (lead && b < p.n_seqs) {
      p.seq_lens[b] = static_cast<int>(ctx + got);
      p.cu[b] = cu0;
      if (b == p.n_seqs - 1) p.cu[p.n_seqs] = cu1;
      if (got > 0 && ctx % kPage && p.tables[static_cast<long long>(b) * p.max_pages + ctx / kPage] < 0)
        bad = kStatusBounds;
    }
    __syncthreads();
    const int chunk_first = s_cu[0], chunk_last = s_cu[kTabThreads];
    for (long long r = max(first_row, static_cast<long long>(chunk_first)) + tid; r < min(last_row, static_cast<long long>(chunk_last));
         r += kTabThreads) {
      int lo = 0, hi = kTabThreads;  // s_cu[lo] <= r < s_cu[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= r) lo = mid; else hi = mid;
      }
      const int k = static_cast<int>(r) - s_cu[lo];
      const int ctx_b = s_ctx[lo], pos = ctx_b + k, page = pos / kPage, held_b = (ctx_b + kPage - 1) / kPage;
      int slot = -1;
      if (k < s_got[lo]) {
        int32_t* row = p.tables + static_cast<long long>(c0 + lo) * p.max_pages;
        // a new page's id comes from the free list (its table entry is being
        // written by the row that opens it), a continued page's from the table
        const int id = page < held_b ? row[page] : p.free_pages[s_free[lo] + page - held_b];
        if (page >= held_b && pos % kPage == 0) row[page] = id;
        if (id >= 0) slot = id * kPage + pos % kPage;
      }
      p.slots[r] = slot;
      if (p.positions) p.positions[r] = pos;
      if (p.row_seq) p.row_seq[r] = c0 + lo;
    }
    rows_before += rows_total;
    pages_before += pages_total;
  }
  const long long used = min(rows_before, static_cast<long long>(p.max_new));
  for (long long r = max(first_row, used) + tid; r < last_row; r += kTabThreads) {
    p.slots[r] = -1;
    if (p.positions) p.positions[r] = -1;
    if (p.row_seq) p.row_seq[r] = -1;
  }
  if (lead) {
    const int any = __syncthreads_or(bad != 0);
    if (tid == 0) {
      *p.status = any ? kStatusBounds : 0u;
      *p.pages_used = static_cast<int>(min(pages_before, static_cast<long long>(p.n_free)));
    }
  }
}

// ---------------------------------------------------------------------------- rows
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf_pack(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// two values -> two e4m3 codes (nearest even, saturating), the first in the low byte
__device__ __forceinline__ uint32_t e4m3_pack(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
template <int N>
__device__ __forceinline__ void unpack(const void* p, float* v) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    v[2 * i] = bf_lo(w[i]);
    v[2 * i + 1] = bf_hi(w[i]);
  }
}
template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int d = W / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}
template <int W>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int d = W / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
  return v;
}
__device__ __forceinline__ float scale_of(float top) { return top > 0.0f ? top / 448.0f : 1.0f; }

// Rotation of 8 neighbouring values (first value's index i0 within the 64) held
// by a lane; the other half of a half-split pair sits 4 lanes away.
__device__ __forceinline__ void load_turn8(const float* cs, int i0, bool inter, float* c, float* s) {
  if (inter) {  // pairs i0/2 .. i0/2 + 3
    const float4 a = *reinterpret_cast<const float4*>(cs + i0 / 2), b = *reinterpret_cast<const float4*>(cs + 32 + i0 / 2);
    c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w;
    s[0] = b.x, s[1] = b.y, s[2] = b.z, s[3] = b.w;
  } else {
    const int j = i0 & 31;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 a = *reinterpret_cast<const float4*>(cs + j + 4 * h), b = *reinterpret_cast<const float4*>(cs + 32 + j + 4 * h);
      c[4 * h] = a.x, c[4 * h + 1] = a.y, c[4 * h + 2] = a.z, c[4 * h + 3] = a.w;
      s[4 * h] = b.x, s[4 * h + 1] = b.y, s[4 * h + 2] = b.z, s[4 * h + 3] = b.w;
    }
  }
}
// (a, b) -> (a c - b s, a s + b c); `act`: the lane holds rotated values (the
// whole warp takes part in the exchange)
__device__ __forceinline__ void turn8(float* v, const float* c, const float* s, int i0, bool inter, bool act) {
  if (inter) {
    if (act) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = v[2 * i], b = v[2 * i + 1];
        v[2 * i] = a * c[i] - b * s[i];
        v[2 * i + 1] = a * s[i] + b * c[i];
      }
    }
  } else {
    const float sign = i0 < 32 ? -1.0f : 1.0f;  // first half: a c - b s; second: b c + a s
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_xor_sync(0xFFFFFFFFu, v[i], 4);
      if (act) v[i] = v[i] * c[i] + sign * o * s[i];
    }
  }
}

struct AppendParams {
  uint8_t* kv;
  float* kv_scale;
  uint8_t* k_idx;
  float* k_idx_scale;
  long long pool_rows;
  int32_t kv_dtype, idx_fp8, rows;
  const int32_t *slots, *positions;
  const uint16_t* ckv;
  long long ckv_stride;
  const float* kv_norm;
  const uint16_t* k_raw;
  long long k_stride;
  const float *idx_norm, *idx_bias;
  float eps;
  const float* cos_sin;
  int32_t max_pos, kv_inter, idx_inter;
  uint32_t* status;
};

// The row's slot, or -1 to skip it; what is out of range is reported.
__device__ __forceinline__ int row_slot(const AppendParams& p, int row, int& pos) {
  const int slot = p.slots[row];
  pos = p.positions[row];
  if (slot == -1) return -1;
  if (slot < 0 || slot >= p.pool_rows || pos < 0 || pos >= p.max_pos) {
    if ((threadIdx.x & 31) == 0) set_status(p.status, kStatusBounds);
    return -1;
  }
  return slot;
}

// One warp per latent row and one per four indexer keys (a key takes 8 or 16
// lanes of 8 values): a row is read once in 16-byte pieces, reduced in
// registers and written once.
constexpr int kRowThreads = 128;

__device__ __forceinline__ void append_latent(const AppendParams& p, int row) {
  const int lane = threadIdx.x & 31;
  int pos;
  const int slot = row_slot(p, row, pos);
  if (slot < 0) return;
  const uint16_t* x = p.ckv + row * p.ckv_stride;
  // values 8 lane .. 8 lane + 7 and 256 + 8 lane .. of the latent part, two rope values
  const uint4 w0 = *reinterpret_cast<const uint4*>(x + 8 * lane);
  const uint4 w1 = *reinterpret_cast<const uint4*>(x + 256 + 8 * lane);
  const float* cs = p.cos_sin + static_cast<long long>(pos) * 64;
  const float c = cs[lane], s = cs[32 + lane];
  const int ia = p.kv_inter ? 2 * lane : lane, ib = p.kv_inter ? 2 * lane + 1 : lane + 32;
  const float a = __uint_as_float(static_cast<uint32_t>(x[kDv + ia]) << 16);
  const float b = __uint_as_float(static_cast<uint32_t>(x[kDv + ib]) << 16);
  const float ra = a * c - b * s, rb = a * s + b * c;
  float v[16];
  unpack<8>(&w0, v);
  unpack<8>(&w1, v + 8);
  if (p.kv_norm) {
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sq += v[i] * v[i];
    const float r = 1.0f / sqrtf(lanes_sum<32>(sq) / kDv + p.eps);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * h + i] = v[8 * h + i] * r * p.kv_norm[256 * h + 8 * lane + i];
  }
  if (p.kv_dtype == SMLA_BF16) {
    uint16_t* o = reinterpret_cast<uint16_t*>(p.kv) + static_cast<long long>(slot) * kDqk;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<uint4*>(o + 256 * h + 8 * lane) =
          make_uint4(bf_pack(v[8 * h], v[8 * h + 1]), bf_pack(v[8 * h + 2], v[8 * h + 3]),
                     bf_pack(v[8 * h + 4], v[8 * h + 5]), bf_pack(v[8 * h + 6], v[8 * h + 7]));
    const uint32_t pr = bf_pack(ra, rb);
    o[kDv + ia] = static_cast<uint16_t>(pr);
    o[kDv + ib] = static_cast<uint16_t>(pr >> 16);
    return;
  }
  const bool tile = p.kv_dtype == SMLA_FP8_DS_MLA;
  float top[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 16; ++i) top[i >> 3] = fmaxf(top[i >> 3], fabsf(v[i]));
  float sc[2];
  if (tile) {  // 16 lanes hold a tile of 128 values
    sc[0] = scale_of(lanes_max<16>(top[0]));
    sc[1] = scale_of(lanes_max<16>(top[1]));
  } else {
    sc[0] = sc[1] = scale_of(lanes_max<32>(fmaxf(fmaxf(top[0], top[1]), fmaxf(fabsf(ra), fabsf(rb)))));
  }
  uint8_t* o = p.kv + static_cast<long long>(slot) * (tile ? 656 : kDqk);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = e4m3_pack(v[8 * h + 2 * i] / sc[h], v[8 * h + 2 * i + 1] / sc[h]);
    *reinterpret_cast<uint2*>(o + 256 * h + 8 * lane) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
  }
  if (tile) {
    if ((lane & 15) == 0) {
      reinterpret_cast<float*>(o + kDv)[lane >> 4] = sc[0];
      reinterpret_cast<float*>(o + kDv)[2 + (lane >> 4)] = sc[1];
    }
    uint16_t* ro = reinterpret_cast<uint16_t*>(o + kDv + 16);
    const uint32_t pr = bf_pack(ra, rb);
    ro[ia] = static_cast<uint16_t>(pr);
    ro[ib] = static_cast<uint16_t>(pr >> 16);
  } else {
    const uint32_t q = e4m3_pack(ra / sc[0], rb / sc[0]);
    o[kDv + ia] = static_cast<uint8_t>(q);
    o[kDv + ib] = static_cast<uint8_t>(q >> 8);
    if (lane == 0) p.kv_scale[slot] = sc[0];
  }
}

// Norm of 8 values a lane over the L lanes of one head or key of 8 L values.
template <int L>
__device__ __forceinline__ void head_norm(float* v, const float* w, const float* bias, float eps, int sub) {
  if (!w) return;
  if (bias) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += v[i];
    const float mean = lanes_sum<L>(sum) / (8 * L);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] -= mean;
  }
  float sq = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) sq += v[i] * v[i];
  const float r = 1.0f / sqrtf(lanes_sum<L>(sq) / (8 * L) + eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] * r * w[8 * sub + i] + (bias ? bias[8 * sub + i] : 0.0f);
}

// L lanes of 8 values a key: 16 (e4m3, 128 values) or 8 (bf16, 64 values).
template <int L>
__device__ __forceinline__ void append_keys(const AppendParams& p, int unit) {
  const int lane = threadIdx.x & 31, sub = lane % L;
  const int row = unit * (32 / L) + lane / L;
  int pos = 0, slot = -1;
  if (row < p.rows) {
    slot = p.slots[row];
    pos = p.positions[row];
    if (slot != -1 && (slot < 0 || slot >= p.pool_rows || pos < 0 || pos >= p.max_pos)) {
      set_status(p.status, kStatusBounds);
      slot = -1;
    }
  }
  const bool live = slot >= 0;
  if (!live) pos = 0;
  uint4 w = make_uint4(0, 0, 0, 0);
  if (live) w = *reinterpret_cast<const uint4*>(p.k_raw + row * p.k_stride + 8 * sub);
  float c[8], s[8], v[8];
  const bool act = sub < 8;
  const int i0 = 8 * (sub & 7);
  load_turn8(p.cos_sin + static_cast<long long>(pos) * 64, i0, p.idx_inter, c, s);
  unpack<8>(&w, v);
  head_norm<L>(v, p.idx_norm, p.idx_bias, p.eps, sub);
  turn8(v, c, s, i0, p.idx_inter, act);
  if (L == 8) {
    if (live)
      *reinterpret_cast<uint4*>(p.k_idx + static_cast<long long>(slot) * 128 + 16 * sub) =
          make_uint4(bf_pack(v[0], v[1]), bf_pack(v[2], v[3]), bf_pack(v[4], v[5]), bf_pack(v[6], v[7]));
    return;
  }
  float sc = 1.0f;
  if (p.k_idx_scale) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
    sc = scale_of(lanes_max<L>(top));
    if (live && sub == 0) p.k_idx_scale[slot] = sc;
  }
  if (live) {
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = e4m3_pack(v[2 * i] / sc, v[2 * i + 1] / sc);
    *reinterpret_cast<uint2*>(p.k_idx + static_cast<long long>(slot) * 128 + 8 * sub) =
        make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
  }
}

__global__ void __launch_bounds__(kRowThreads) cache_append_kernel(const AppendParams p, int latent_warps) {
  const int warp = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (warp < latent_warps) {
    append_latent(p, warp);
  } else if (p.k_raw) {
    const int unit = warp - latent_warps;
    if (p.idx_fp8) {
      if (unit * 2 < p.rows) append_keys<16>(p, unit);
    } else {
      if (unit * 4 < p.rows) append_keys<8>(p, unit);
    }
  }
}

struct QueryParams {
  const float* cos_sin;
  int32_t max_pos, kv_inter, idx_inter, rows;
  const int32_t* positions;
  const uint16_t* q_pe;
  long long pe_row, pe_head;
  int32_t n_heads;
  uint16_t* q;
  const uint16_t* q_raw;
  long long raw_stride;
  int32_t h_idx, idx_fp8;
  const float* idx_norm;
  float eps;
  const float* w;
  float w_scale;
  uint8_t* q_idx;
  float* w_out;
  uint32_t* status;
  int32_t pe_units, units;  // warps per row: 16 attention heads or 8 (fp8) / 16 (bf16) indexer heads each
};

template <int L>
__device__ __forceinline__ void query_heads(const QueryParams& p, int row, int pos, int unit) {
  constexpr int kPer = 32 / L;  // heads per step
  const int lane = threadIdx.x & 31, sub = lane % L;
  const int i0 = 8 * (sub & 7);
  float c[8], s[8];
  load_turn8(p.cos_sin + static_cast<long long>(pos) * 64, i0, p.idx_inter, c, s);
  uint4 w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int h = (unit * 4 + j) * kPer + lane / L;
    if (h < p.h_idx) w[j] = *reinterpret_cast<const uint4*>(p.q_raw + row * p.raw_stride + h * (8 * L) + 8 * sub);
    else w[j] = make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int h = (unit * 4 + j) * kPer + lane / L;
    const bool live = h < p.h_idx;
    const long long at = static_cast<long long>(row) * p.h_idx + h;
    float v[8];
    unpack<8>(&w[j], v);
    head_norm<L>(v, p.idx_norm, nullptr, p.eps, sub);
    turn8(v, c, s, i0, p.idx_inter, sub < 8);
    float sc = 1.0f;
    if (L == 8) {
      if (live)
        *reinterpret_cast<uint4*>(p.q_idx + at * 128 + 16 * sub) =
            make_uint4(bf_pack(v[0], v[1]), bf_pack(v[2], v[3]), bf_pack(v[4], v[5]), bf_pack(v[6], v[7]));
    } else {
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
      sc = scale_of(lanes_max<L>(top));
      uint32_t q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = e4m3_pack(v[2 * i] / sc, v[2 * i + 1] / sc);
      if (live) *reinterpret_cast<uint2*>(p.q_idx + at * 128 + 8 * sub) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
    }
    if (live && sub == 0) p.w_out[at] = p.w[at] * (sc * p.w_scale);
  }
}

__global__ void __launch_bounds__(kRowThreads) query_prep_kernel(const QueryParams p) {
  const long long warp = static_cast<long long>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int row = static_cast<int>(warp / p.units), unit = static_cast<int>(warp - static_cast<long long>(row) * p.units);
  if (row >= p.rows) return;
  const int lane = threadIdx.x & 31;
  const int pos = p.positions[row];
  if (pos < 0 || pos >= p.max_pos) {
    if (lane == 0) set_status(p.status, kStatusBounds);
    return;
  }
  if (unit >= p.pe_units) {
    if (p.idx_fp8) query_heads<16>(p, row, pos, unit - p.pe_units);
    else query_heads<8>(p, row, pos, unit - p.pe_units);
    return;
  }
  const int sub = lane & 7, i0 = 8 * sub;
  float c[8], s[8];
  load_turn8(p.cos_sin + static_cast<long long>(pos) * 64, i0, p.kv_inter, c, s);
  uint4 w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int h = unit * 16 + j * 4 + (lane >> 3);
    w[j] = *reinterpret_cast<const uint4*>(p.q_pe + row * p.pe_row + h * p.pe_head + i0);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int h = unit * 16 + j * 4 + (lane >> 3);
    float v[8];
    unpack<8>(&w[j], v);
    turn8(v, c, s, i0, p.kv_inter, true);
    *reinterpret_cast<uint4*>(p.q + (static_cast<long long>(row) * p.n_heads + h) * kDqk + kDv + i0) =
        make_uint4(bf_pack(v[0], v[1]), bf_pack(v[2], v[3]), bf_pack(v[4], v[5]), bf_pack(v[6], v[7]));
  }
}

bool al(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_rope(const smla_rope* r) {
  if (!r || !r->cos_sin || !al(r->cos_sin, 16) || r->max_pos <= 0) return SMLA_ERR_INVALID_ARG;
  return SMLA_OK;
}

int check_ws(void* workspace, size_t bytes) {
  return !workspace || !al(workspace, 16) || bytes < kStatusBytes ? SMLA_ERR_WORKSPACE : SMLA_OK;
}

int launched() { return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA; }

}  // namespace
}  // namespace smla

using namespace smla;

extern "C" {

int smla_build_tables(const int32_t* ctx_lens, const int32_t* new_lens, int32_t n_seqs, int32_t* page_tables,
                      int32_t max_pages, const int32_t* free_pages, int32_t n_free, int32_t max_new,
                      int32_t* seq_lens, int32_t* cu_new, int32_t* positions, int32_t* slots, int32_t* row_seq,
                      int32_t* pages_used, void* workspace, size_t workspace_bytes, void* stream) {
  if (!ctx_lens || !new_lens || !page_tables || !seq_lens || !cu_new || !slots || !pages_used) return SMLA_ERR_INVALID_ARG;
  if (n_seqs <= 0 || max_pages <= 0 || n_free < 0 || max_new <= 0 || (n_free > 0 && !free_pages)) return SMLA_ERR_INVALID_ARG;
  if (max_pages > (1 << 25)) return SMLA_ERR_UNSUPPORTED;  // positions are int32
  for (const void* a : {static_cast<const void*>(ctx_lens), static_cast<const void*>(new_lens), static_cast<const void*>(page_tables),
                        static_cast<const void*>(free_pages), static_cast<const void*>(seq_lens), static_cast<const void*>(cu_new),
                        static_cast<const void*>(positions), static_cast<const void*>(slots), static_cast<const void*>(row_seq),
                        static_cast<const void*>(pages_used)})
    if (!al(a, 4)) return SMLA_ERR_INVALID_ARG;
  if (seq_lens == ctx_lens || seq_lens == new_lens) return SMLA_ERR_INVALID_ARG;  // other blocks still read the lengths
  if (const int rc = check_ws(workspace, workspace_bytes)) return rc;
  const int rows_per_block = 2 * kTabThreads;
  TablesParams p{ctx_lens, new_lens, n_seqs, max_pages, page_tables, free_pages, n_free, max_new, seq_lens, cu_new, positions,
                 slots, row_seq, pages_used, static_cast<uint32_t*>(workspace), rows_per_block};
  const unsigned blocks = static_cast<unsigned>((static_cast<long long>(max_new) + rows_per_block - 1) / rows_per_block);
  build_tables_kernel<<<blocks, kTabThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return launched();
}

int smla_cache_append(const smla_paged_cache* cache, const smla_rope* rope, int32_t rows, const int32_t* slots,
                      const int32_t* positions, const void* ckv, int64_t ckv_stride, const float* kv_norm,
                      const void* k_raw, int64_t k_stride, const float* idx_norm, const float* idx_bias, float eps,
                      void* workspace, size_t workspace_bytes, void* stream) {
  if (!ckv && !k_raw) return SMLA_ERR_INVALID_ARG;
  int rc = check_cache(cache, ckv != nullptr, k_raw != nullptr);
  if (rc) return rc;
  if ((rc = check_rope(rope))) return rc;
  if (rows <= 0 || !slots || !positions || !al(slots, 4) || !al(positions, 4) || !(eps >= 0.0f)) return SMLA_ERR_INVALID_ARG;
  if (ckv && (!al(ckv, 16) || ckv_stride < kDqk || ckv_stride % 8 || !al(kv_norm, 4))) return SMLA_ERR_INVALID_ARG;
  if (k_raw && (!al(k_raw, 16) || k_stride < cache->d_idx || k_stride % 8 || !al(idx_norm, 4) || !al(idx_bias, 4) ||
                (idx_bias && !idx_norm)))
    return SMLA_ERR_INVALID_ARG;
  if ((rc = check_ws(workspace, workspace_bytes))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, 4, st) != cudaSuccess) return SMLA_ERR_CUDA;
  AppendParams p{};
  p.kv = static_cast<uint8_t*>(const_cast<void*>(cache->kv));
  p.kv_scale = const_cast<float*>(cache->kv_scale);
  p.k_idx = static_cast<uint8_t*>(const_cast<void*>(cache->k_idx));
  p.k_idx_scale = const_cast<float*>(cache->k_idx_scale);
  p.pool_rows = static_cast<long long>(cache->num_pages) * kPage;
  p.kv_dtype = cache->kv_dtype;
  p.idx_fp8 = cache->idx_dtype == SMLA_FP8_E4M3;
  p.rows = rows;
  p.slots = slots, p.positions = positions;
  p.ckv = static_cast<const uint16_t*>(ckv), p.ckv_stride = ckv_stride, p.kv_norm = kv_norm;
  p.k_raw = static_cast<const uint16_t*>(k_raw), p.k_stride = k_stride, p.idx_norm = idx_norm, p.idx_bias = idx_bias;
  p.eps = eps;
  p.cos_sin = rope->cos_sin, p.max_pos = rope->max_pos;
  p.kv_inter = rope->kv_interleaved, p.idx_inter = rope->idx_interleaved;
  p.status = static_cast<uint32_t*>(workspace);
  const int latent = ckv ? rows : 0;
  const long long warps = latent + (k_raw ? (static_cast<long long>(rows) + 1) / (p.idx_fp8 ? 2 : 4) + 1 : 0);
  const unsigned blocks = static_cast<unsigned>((warps + kRowThreads / 32 - 1) / (kRowThreads / 32));
  cache_append_kernel<<<blocks, kRowThreads, 0, st>>>(p, latent);
  return launched();
}

int smla_query_prep(const smla_rope* rope, int32_t rows, const int32_t* positions, const void* q_pe,
                    int64_t pe_row_stride, int64_t pe_head_stride, int32_t n_heads, void* q, const void* q_raw,
                    int64_t q_raw_stride, int32_t h_idx, int32_t d_idx, int32_t idx_dtype, const float* idx_norm,
                    float eps, const float* w, float w_scale, void* q_idx, float* w_out, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!q_pe && !q_raw) return SMLA_ERR_INVALID_ARG;
  int rc = check_rope(rope);
  if (rc) return rc;
  if (rows <= 0 || !positions || !al(positions, 4)) return SMLA_ERR_INVALID_ARG;
  if (q_pe) {
    if (!q || !al(q, 16) || !al(q_pe, 16) || pe_row_stride % 8 || pe_head_stride % 8 || pe_head_stride < 64 || pe_row_stride < 0)
      return SMLA_ERR_INVALID_ARG;
    if (n_heads != 16 && n_heads != 64) return SMLA_ERR_UNSUPPORTED;
  }
  if (q_raw) {
    if (!w || !q_idx || !w_out || !al(q_raw, 16) || !al(q_idx, 16) || !al(w, 4) || !al(w_out, 4) || !al(idx_norm, 4) ||
        q_raw_stride % 8 || d_idx <= 0 || h_idx <= 0 || q_raw_stride < static_cast<int64_t>(h_idx) * d_idx || !(eps >= 0.0f))
      return SMLA_ERR_INVALID_ARG;
    if (idx_dtype != SMLA_BF16 && idx_dtype != SMLA_FP8_E4M3) return SMLA_ERR_INVALID_ARG;
    if (d_idx != (idx_dtype == SMLA_BF16 ? 64 : 128)) return SMLA_ERR_UNSUPPORTED;
    if (h_idx != 4 && h_idx != 8 && h_idx != 16 && h_idx != 32 && h_idx != 64) return SMLA_ERR_UNSUPPORTED;
  }
  if ((rc = check_ws(workspace, workspace_bytes))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, 4, st) != cudaSuccess) return SMLA_ERR_CUDA;
  QueryParams p{};
  p.cos_sin = rope->cos_sin, p.max_pos = rope->max_pos;
  p.kv_inter = rope->kv_interleaved, p.idx_inter = rope->idx_interleaved;
  p.rows = rows, p.positions = positions;
  p.q_pe = static_cast<const uint16_t*>(q_pe), p.pe_row = pe_row_stride, p.pe_head = pe_head_stride;
  p.n_heads = n_heads, p.q = static_cast<uint16_t*>(q);
  p.q_raw = static_cast<const uint16_t*>(q_raw), p.raw_stride = q_raw_stride, p.h_idx = h_idx;
  p.idx_fp8 = idx_dtype == SMLA_FP8_E4M3, p.idx_norm = idx_norm, p.eps = eps;
  p.w = w, p.w_scale = w_scale, p.q_idx = static_cast<uint8_t*>(q_idx), p.w_out = w_out;
  p.status = static_cast<uint32_t*>(workspace);
  p.pe_units = q_pe ? n_heads / 16 : 0;
  const int per = p.idx_fp8 ? 8 : 16;
  p.units = p.pe_units + (q_raw ? (h_idx + per - 1) / per : 0);
  const long long warps = static_cast<long long>(rows) * p.units;
  const unsigned blocks = static_cast<unsigned>((warps + kRowThreads / 32 - 1) / (kRowThreads / 32));
  query_prep_kernel<<<blocks, kRowThreads, 0, st>>>(p);
  return launched();
}

}  // extern "C"
