// Serving steps around the paged cache: block tables and slot maps
// (smla_build_tables), new rows into the cache (smla_cache_append), queries
// (smla_query_prep). All three move little or stream their data once, so their
// floors are launch latency (decode-sized calls) and memory bandwidth
// (prefill-sized calls).
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "serve.h"

namespace smla {
namespace {

// ---------------------------------------------------------------------------- tables
constexpr int kTabThreads = 1024;

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

// A page id that a pool can have (pool rows are int32).
__device__ __forceinline__ bool page_id(int id) { return id >= 0 && id < (1 << 25); }

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
  long long w = warp_sums[lane];  // as many warps as lanes: every warp scans the warps' sums
  static_assert(kTabThreads == 1024, "32 warps");
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xFFFFFFFFu, w, d);
    if (lane >= d) w += o;
  }
  total = __shfl_sync(0xFFFFFFFFu, w, 31);
  const long long before = __shfl_sync(0xFFFFFFFFu, w, (warp + 31) & 31);
  return v + (warp ? before : 0);
}

// Every block scans all requests' lengths, 1,024 at a time (a few KB that stay in
// L2; no block waits for another, so one launch does the whole job), and writes
// the rows [first, last) of the per-token outputs that are its share; block 0
// also writes the per-request outputs and the status word, which needs no clearing
// launch because block 0 sees every condition that can set it. Bound by latency:
// a load, two block scans and a search per 1,024 requests, and block 0's look at the
// ids that were taken. 1,000 requests with up to 257 new tokens: 7.4 us on cold
// caches; 64 requests: 5.5 us, within the launch of a call.
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
  const long long most = min(static_cast<long long>(p.max_pages) * kPage, static_cast<long long>(INT_MAX) - (kPage - 1));
  long long rows_before = 0, pages_before = 0;  // of the chunks before this one
  uint32_t bad = 0;
  for (int c0 = 0; c0 < p.n_seqs; c0 += kTabThreads) {
    const int b = c0 + tid;
    long long ctx = 0, add = 0;
    bool valid = true;
    if (b < p.n_seqs) {
      ctx = p.ctx[b];
      add = p.add[b];
      valid = ctx >= 0 && add >= 0 && ctx + add <= most;
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
      if (got > 0 && ctx % kPage && !page_id(p.tables[static_cast<long long>(b) * p.max_pages + ctx / kPage]))
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
        if (page_id(id)) slot = id * kPage + pos % kPage;
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
    const int taken = static_cast<int>(min(pages_before, static_cast<long long>(p.n_free)));
#pragma unroll 4
    for (int i = tid; i < taken; i += kTabThreads)
      if (!page_id(p.free_pages[i])) bad = kStatusBounds;
    const int any = __syncthreads_or(bad != 0);
    if (tid == 0) {
      *p.status = any ? kStatusBounds : 0u;
      *p.pages_used = taken;
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
__device__ __forceinline__ void load8(const float* p, float* v) {  // 16-byte aligned
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
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
// scale = amax / 448 (at least 2^-126; 1 where all are zero), and codes of the fp32
// quotients value / scale. Each division is the product with the rounded reciprocal
// and one step of correction, q + (x - q s) / s, whose remainder an fma gives exactly
// (Markstein's division): no branch and no call. Rows under 2^-80 go up by 2^64
// first, where remainders stay inside fp32's range. An infinite amax gives finite
// values the code 0, as the division does. (NaN does not show in amax: its code is
// NaN.) 8,192 rows of queries: 52 us; 56 with division instructions, and 49 without
// the step of correction, where scales are a few 2^-24 off and values next to a tie
// land on the other code.
struct Scale {
  float s, d, inv, up;  // the scale; what the (raised) values are divided by
  __device__ __forceinline__ explicit Scale(float top) : s(1.0f), d(1.0f), inv(1.0f), up(1.0f) {
    if (top > 0.0f) {
      constexpr float k = 1.0f / 448.0f;
      up = top < 0x1p-80f ? 0x1p64f : 1.0f;
      const float t = top * up, q = t * k;
      d = t < INFINITY ? fmaxf(fmaf(fmaf(-q, 448.0f, t), k, q), FLT_MIN * up) : t;
      inv = __frcp_rn(d);
      s = top < 0x1p-80f ? d * 0x1p-64f : d;
      if (!(d < INFINITY)) d = 0.0f;
    }
  }
  // codes of two values, the first in the low byte
  __device__ __forceinline__ uint32_t pack(float a, float b) const {
    const float2 v = mul2(make_float2(a, b), make_float2(up, up)), by = make_float2(inv, inv);
    const float2 q = mul2(v, by), rest = fma2(make_float2(-q.x, -q.y), make_float2(d, d), v), y = fma2(rest, by, q);
    return e4m3_pack(y.x, y.y);
  }
  __device__ __forceinline__ uint32_t pack4(const float* v) const { return pack(v[0], v[1]) | (pack(v[2], v[3]) << 16); }
};

// How a head's or key's values lie in its lanes: eight a lane in two groups of four,
// so that both values of every rotated pair are in one lane under either pairing.
// Rotated lanes (sub < 8): pairs 4 sub .. 4 sub + 3.
struct Places {
  int a, b;  // first value of each group
  __device__ __forceinline__ Places(int sub, bool inter) {
    const bool halves = !inter && sub < 8;
    a = halves ? 4 * sub : 8 * sub;
    b = halves ? 32 + 4 * sub : 8 * sub + 4;
  }
};
struct Turn {  // cosines and sines of a lane's four pairs
  float4 c, s;
  __device__ __forceinline__ Turn(const float* cos_sin, int pos, int sub) {
    const float* at = cos_sin + static_cast<long long>(pos) * 64 + 4 * (sub & 7);
    c = __ldg(reinterpret_cast<const float4*>(at));
    s = __ldg(reinterpret_cast<const float4*>(at + 32));
  }
  static __device__ __forceinline__ void pair(float& a, float& b, float c, float s) {
    const float x = a, y = b;
    a = x * c - y * s;
    b = x * s + y * c;
  }
  __device__ __forceinline__ void apply(float* v, bool inter) const {
    if (inter) {
      pair(v[0], v[1], c.x, s.x), pair(v[2], v[3], c.y, s.y), pair(v[4], v[5], c.z, s.z), pair(v[6], v[7], c.w, s.w);
    } else {
      pair(v[0], v[4], c.x, s.x), pair(v[1], v[5], c.y, s.y), pair(v[2], v[6], c.z, s.z), pair(v[3], v[7], c.w, s.w);
    }
  }
};
// the lane's eight bf16 values of a head at p, and the way back
__device__ __forceinline__ uint4 load_groups(const uint16_t* p, const Places& at) {
  const uint2 a = __ldg(reinterpret_cast<const uint2*>(p + at.a)), b = __ldg(reinterpret_cast<const uint2*>(p + at.b));
  return make_uint4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store_groups(uint16_t* p, const Places& at, const float* v) {
  *reinterpret_cast<uint2*>(p + at.a) = make_uint2(bf_pack(v[0], v[1]), bf_pack(v[2], v[3]));
  *reinterpret_cast<uint2*>(p + at.b) = make_uint2(bf_pack(v[4], v[5]), bf_pack(v[6], v[7]));
}
__device__ __forceinline__ void load_weights(const float* p, const Places& at, float* w) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p + at.a)), b = __ldg(reinterpret_cast<const float4*>(p + at.b));
  w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
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
  int32_t max_pos, kv_inter, idx_inter, first_reports;
  uint32_t* status;
};

// The row's slot, or -1 to skip it (a row that is not written, or out of range).
__device__ __forceinline__ int usable_slot(const AppendParams& p, int slot, int pos) {
  const bool ok = slot >= 0 && slot < p.pool_rows && pos >= 0 && pos < p.max_pos;
  if (!ok && slot != -1 && !p.first_reports) set_status(p.status, kStatusBounds);
  return ok ? slot : -1;
}
// How a launch reports rows that it skips as out of range. Up to kReportRows rows
// its first block only looks all of them over and writes the status word, so that
// the call needs no launch to clear it (about 2 us of an 8 us call); with more rows
// that block would end last, the word is cleared by a memset, and the warps report.
constexpr int kReportRows = 4096;

template <typename Bad>
__device__ __forceinline__ void report_rows(int rows, uint32_t* status, Bad bad) {
  bool any = false;
  for (int r0 = threadIdx.x; r0 < rows; r0 += 8 * blockDim.x) {
    bool b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = bad(min(r0 + i * static_cast<int>(blockDim.x), rows - 1));  // loads of all eight in flight
#pragma unroll
    for (int i = 0; i < 8; ++i) any |= b[i];
  }
  const int found = __syncthreads_or(any);
  if (threadIdx.x == 0) *status = found ? kStatusBounds : 0u;
}

// One warp per latent row and one per two or four indexer keys (a key takes 16 or 8
// lanes of 8 values): a row is read once in 16-byte pieces, reduced in registers
// and written once. Its values are requested before the slot and position are
// looked at, so a row costs two memory latencies (position, then its angles)
// and not three. Cold caches: 128 rows 3.3 us; 8,192 BF16 rows with FP8 keys 8.7 us,
// 24 MB, 2.8 TB/s; 5,003 tile-scaled rows 6.7 us: two to four times what the bytes
// take, in one or two waves of warps. (More rows a warp have not been measured.)
constexpr int kRowThreads = 128;

__device__ __forceinline__ void append_latent(const AppendParams& p, int row) {
  const int lane = threadIdx.x & 31;
  const uint16_t* x = p.ckv + row * p.ckv_stride;
  const int pos = __ldg(p.positions + row), id = __ldg(p.slots + row);
  // values 8 lane .. 8 lane + 7 and 256 + 8 lane .. of the latent part, two rope values
  const uint4 w0 = __ldg(reinterpret_cast<const uint4*>(x + 8 * lane));
  const uint4 w1 = __ldg(reinterpret_cast<const uint4*>(x + 256 + 8 * lane));
  const int ia = p.kv_inter ? 2 * lane : lane, ib = p.kv_inter ? 2 * lane + 1 : lane + 32;
  const uint16_t xa = __ldg(x + kDv + ia), xb = __ldg(x + kDv + ib);
  const int slot = usable_slot(p, id, pos);
  if (slot < 0) return;
  const float* cs = p.cos_sin + static_cast<long long>(pos) * 64;
  const float c = __ldg(cs + lane), s = __ldg(cs + 32 + lane);
  const float a = __uint_as_float(static_cast<uint32_t>(xa) << 16);
  const float b = __uint_as_float(static_cast<uint32_t>(xb) << 16);
  const float ra = a * c - b * s, rb = a * s + b * c;
  float v[16];
  unpack<8>(&w0, v);
  unpack<8>(&w1, v + 8);
  if (p.kv_norm) {
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sq += v[i] * v[i];
    const float r = rsqrtf(lanes_sum<32>(sq) / kDv + p.eps);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float w[8];
      load8(p.kv_norm + 256 * h + 8 * lane, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * h + i] = v[8 * h + i] * r * w[i];
    }
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
  if (tile) {  // 16 lanes hold a tile of 128 values
    top[0] = lanes_max<16>(top[0]);
    top[1] = lanes_max<16>(top[1]);
  } else {
    top[0] = top[1] = lanes_max<32>(fmaxf(fmaxf(top[0], top[1]), fmaxf(fabsf(ra), fabsf(rb))));
  }
  const Scale by[2] = {Scale(top[0]), Scale(top[1])};
  uint8_t* o = p.kv + static_cast<long long>(slot) * (tile ? 656 : kDqk);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    *reinterpret_cast<uint2*>(o + 256 * h + 8 * lane) = make_uint2(by[h].pack4(v + 8 * h), by[h].pack4(v + 8 * h + 4));
  }
  if (tile) {
    if ((lane & 15) == 0) {
      reinterpret_cast<float*>(o + kDv)[lane >> 4] = by[0].s;
      reinterpret_cast<float*>(o + kDv)[2 + (lane >> 4)] = by[1].s;
    }
    uint16_t* ro = reinterpret_cast<uint16_t*>(o + kDv + 16);
    const uint32_t pr = bf_pack(ra, rb);
    ro[ia] = static_cast<uint16_t>(pr);
    ro[ib] = static_cast<uint16_t>(pr >> 16);
  } else {
    const uint32_t q = by[0].pack(ra, rb);
    o[kDv + ia] = static_cast<uint8_t>(q);
    o[kDv + ib] = static_cast<uint8_t>(q >> 8);
    if (lane == 0) p.kv_scale[slot] = by[0].s;
  }
}

// Norm of 8 values a lane over the L lanes of one head or key of 8 L values; w and b:
// the lane's weights and biases.
template <int L>
__device__ __forceinline__ void head_norm(float* v, bool norm, const float* w, bool bias, const float* b, float eps) {
  if (!norm) return;
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
  const float r = rsqrtf(lanes_sum<L>(sq) / (8 * L) + eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] * r * w[i] + (bias ? b[i] : 0.0f);
}

// L lanes of 8 values a key: 16 (e4m3, 128 values) or 8 (bf16, 64 values).
template <int L>
__device__ __forceinline__ void append_keys(const AppendParams& p, int unit) {
  const int lane = threadIdx.x & 31, sub = lane % L;
  const int row = unit * (32 / L) + lane / L;
  const Places at(sub, p.idx_inter);
  int pos = 0, slot = -1;
  uint4 w = make_uint4(0, 0, 0, 0);
  if (row < p.rows) {
    w = load_groups(p.k_raw + row * p.k_stride, at);
    pos = __ldg(p.positions + row);
    slot = usable_slot(p, __ldg(p.slots + row), pos);
  }
  const bool live = slot >= 0;
  const Turn turn(p.cos_sin, live ? pos : 0, sub);
  float v[8], nw[8], nb[8];
  if (p.idx_norm) load_weights(p.idx_norm, at, nw);
  if (p.idx_bias) load_weights(p.idx_bias, at, nb);
  unpack<8>(&w, v);
  head_norm<L>(v, p.idx_norm != nullptr, nw, p.idx_bias != nullptr, nb, p.eps);
  if (sub < 8) turn.apply(v, p.idx_inter);
  uint8_t* o = p.k_idx + static_cast<long long>(max(slot, 0)) * 128;
  if (L == 8) {
    if (live) store_groups(reinterpret_cast<uint16_t*>(o), at, v);
    return;
  }
  if (!p.k_idx_scale) {  // as they are
    if (live) {
      *reinterpret_cast<uint32_t*>(o + at.a) = e4m3_pack(v[0], v[1]) | (e4m3_pack(v[2], v[3]) << 16);
      *reinterpret_cast<uint32_t*>(o + at.b) = e4m3_pack(v[4], v[5]) | (e4m3_pack(v[6], v[7]) << 16);
    }
    return;
  }
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
  const Scale by(lanes_max<L>(top));
  if (live) {
    if (sub == 0) p.k_idx_scale[slot] = by.s;
    *reinterpret_cast<uint32_t*>(o + at.a) = by.pack4(v);
    *reinterpret_cast<uint32_t*>(o + at.b) = by.pack4(v + 4);
  }
}

__global__ void __launch_bounds__(kRowThreads) cache_append_kernel(const AppendParams p, int latent_warps) {
  if (p.first_reports && blockIdx.x == 0) {
    report_rows(p.rows, p.status, [&](int r) {
      const int slot = __ldg(p.slots + r), pos = __ldg(p.positions + r);
      return slot != -1 && (slot < 0 || slot >= p.pool_rows || pos < 0 || pos >= p.max_pos);
    });
    return;
  }
  const int warp = (blockIdx.x - p.first_reports) * (kRowThreads / 32) + (threadIdx.x >> 5);
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
  int32_t pe_units, units;  // warps per row: up to 32 attention heads or 16 (fp8) / 32 (bf16) indexer heads each
  int32_t first_reports;
};

// A warp takes four steps of 4 (8 lanes a head) or 2 (16 lanes) heads of one row,
// all loaded before the row's position and angles, which are two latencies away.
// Bound by memory and instructions: 8,192 rows of 64 attention and 32 indexer heads
// move 239 MB in 51.4 us, 4.7 TB/s or 69% of a plain copy's rate (the rope values are
// written as 128 bytes of every 1,152); 128 rows take 4.7 us. Measured when codes were
// products without a step of correction and four steps took 48.6 us: two or eight
// steps 58 us, blocks of 256 threads 53, 51 or 42 registers (more warps) 53 or 55.
constexpr int kSteps = 4;

template <int L>
__device__ __forceinline__ void query_heads(const QueryParams& p, int row, int unit) {
  constexpr int kPer = 32 / L;  // heads per step
  const int lane = threadIdx.x & 31, sub = lane % L;
  const Places at(sub, p.idx_inter);
  uint4 w[kSteps];
  float head_w[kSteps];
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    const int h = (unit * kSteps + j) * kPer + lane / L;
    const bool live = h < p.h_idx;
    w[j] = live ? load_groups(p.q_raw + row * p.raw_stride + h * (8 * L), at) : make_uint4(0, 0, 0, 0);
    head_w[j] = live && sub == 0 ? p.w[static_cast<long long>(row) * p.h_idx + h] : 0.0f;  // (w_out may be w)
  }
  float nw[8];
  if (p.idx_norm) load_weights(p.idx_norm, at, nw);
  const int pos = __ldg(p.positions + row);
  if (pos < 0 || pos >= p.max_pos) {
    if (pos != -1 && !p.first_reports) set_status(p.status, kStatusBounds);
    return;
  }
  const Turn turn(p.cos_sin, pos, sub);
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    const int h = (unit * kSteps + j) * kPer + lane / L;
    const bool live = h < p.h_idx;
    if (j > 0 && (unit * kSteps + j) * kPer >= p.h_idx) break;
    const long long head = static_cast<long long>(row) * p.h_idx + h;
    float v[8];
    unpack<8>(&w[j], v);
    head_norm<L>(v, p.idx_norm != nullptr, nw, false, nw, p.eps);
    if (sub < 8) turn.apply(v, p.idx_inter);
    float top = 0.0f;
    if (L == 16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
      top = lanes_max<L>(top);
    }
    const Scale by(top);  // (bf16: 1)
    if (live) {
      uint8_t* o = p.q_idx + head * 128;
      if (L == 8) {
        store_groups(reinterpret_cast<uint16_t*>(o), at, v);
      } else {
        *reinterpret_cast<uint32_t*>(o + at.a) = by.pack4(v);
        *reinterpret_cast<uint32_t*>(o + at.b) = by.pack4(v + 4);
      }
      if (sub == 0) p.w_out[head] = head_w[j] * (by.s * p.w_scale);
    }
  }
}

__global__ void __launch_bounds__(kRowThreads) query_prep_kernel(const QueryParams p) {
  if (p.first_reports && blockIdx.x == 0) {
    report_rows(p.rows, p.status, [&](int r) {
      const int pos = __ldg(p.positions + r);
      return pos != -1 && (pos < 0 || pos >= p.max_pos);
    });
    return;
  }
  const long long warp = static_cast<long long>(blockIdx.x - p.first_reports) * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int row = static_cast<int>(warp / p.units), unit = static_cast<int>(warp - static_cast<long long>(row) * p.units);
  if (row >= p.rows) return;
  const int lane = threadIdx.x & 31;
  if (unit >= p.pe_units) {
    if (p.idx_fp8) query_heads<16>(p, row, unit - p.pe_units);
    else query_heads<8>(p, row, unit - p.pe_units);
    return;
  }
  const int sub = lane & 7;
  const Places at(sub, p.kv_inter);
  uint4 w[kSteps];
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    const int h = (unit * kSteps + j) * 4 + (lane >> 3);
    if (h < p.n_heads) w[j] = load_groups(p.q_pe + row * p.pe_row + h * p.pe_head, at);
  }
  const int pos = __ldg(p.positions + row);
  if (pos < 0 || pos >= p.max_pos) {
    if (pos != -1 && !p.first_reports) set_status(p.status, kStatusBounds);
    return;
  }
  const Turn turn(p.cos_sin, pos, sub);
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    const int h = (unit * kSteps + j) * 4 + (lane >> 3);
    if (h >= p.n_heads) break;  // (heads are a multiple of 4: the whole warp)
    float v[8];
    unpack<8>(&w[j], v);
    turn.apply(v, p.kv_inter);
    store_groups(p.q + (static_cast<long long>(row) * p.n_heads + h) * kDqk + kDv, at, v);
  }
}

int check_rope(const smla_rope* r) {
  if (!r || !r->cos_sin || !aligned_to(r->cos_sin, 16) || r->max_pos <= 0) return SMLA_ERR_INVALID_ARG;
  return SMLA_OK;
}

int check_ws(void* workspace, size_t bytes) {
  return !workspace || !aligned_to(workspace, 16) || bytes < kStatusBytes ? SMLA_ERR_WORKSPACE : SMLA_OK;
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
    if (!aligned_to(a, 4)) return SMLA_ERR_INVALID_ARG;
  if (seq_lens == ctx_lens || seq_lens == new_lens) return SMLA_ERR_INVALID_ARG;  // other blocks still read the lengths
  if (const int rc = check_ws(workspace, workspace_bytes)) return rc;
  const int rows_per_block = std::max(kTabThreads, static_cast<int>((max_new + 2LL * num_sms() - 1) / (2 * num_sms())));
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
  int rc = check_serve_cache(cache, ckv != nullptr, k_raw != nullptr);
  if (rc) return rc;
  if ((rc = check_rope(rope))) return rc;
  if (rows <= 0 || !slots || !positions || !aligned_to(slots, 4) || !aligned_to(positions, 4) || !(eps >= 0.0f)) return SMLA_ERR_INVALID_ARG;
  if (ckv && (!aligned_to(ckv, 16) || ckv_stride < kDqk || ckv_stride % 8 || !aligned_to(kv_norm, 16))) return SMLA_ERR_INVALID_ARG;
  if (k_raw && (!aligned_to(k_raw, 16) || k_stride < cache->d_idx || k_stride % 8 || !aligned_to(idx_norm, 16) || !aligned_to(idx_bias, 16) ||
                (idx_bias && !idx_norm)))
    return SMLA_ERR_INVALID_ARG;
  if ((rc = check_ws(workspace, workspace_bytes))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
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
  p.first_reports = rows <= kReportRows;
  if (!p.first_reports && cudaMemsetAsync(workspace, 0, 4, st) != cudaSuccess) return SMLA_ERR_CUDA;
  const int latent = ckv ? rows : 0;
  const long long warps = latent + (k_raw ? (static_cast<long long>(rows) + 1) / (p.idx_fp8 ? 2 : 4) + 1 : 0);
  const unsigned blocks = static_cast<unsigned>((warps + kRowThreads / 32 - 1) / (kRowThreads / 32)) + p.first_reports;
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
  if (rows <= 0 || !positions || !aligned_to(positions, 4)) return SMLA_ERR_INVALID_ARG;
  if (q_pe) {
    if (!q || !aligned_to(q, 16) || !aligned_to(q_pe, 16) || pe_row_stride % 8 || pe_head_stride % 8 || pe_head_stride < 64 || pe_row_stride < 0)
      return SMLA_ERR_INVALID_ARG;
    if (n_heads != 16 && n_heads != 64) return SMLA_ERR_UNSUPPORTED;
  }
  if (q_raw) {
    if (!w || !q_idx || !w_out || !aligned_to(q_raw, 16) || !aligned_to(q_idx, 16) || !aligned_to(w, 4) || !aligned_to(w_out, 4) || !aligned_to(idx_norm, 16) ||
        q_raw_stride % 8 || d_idx <= 0 || h_idx <= 0 || q_raw_stride < static_cast<int64_t>(h_idx) * d_idx || !(eps >= 0.0f))
      return SMLA_ERR_INVALID_ARG;
    if (idx_dtype != SMLA_BF16 && idx_dtype != SMLA_FP8_E4M3) return SMLA_ERR_INVALID_ARG;
    if (d_idx != (idx_dtype == SMLA_BF16 ? 64 : 128)) return SMLA_ERR_UNSUPPORTED;
    if (h_idx != 4 && h_idx != 8 && h_idx != 16 && h_idx != 32 && h_idx != 64) return SMLA_ERR_UNSUPPORTED;
  }
  if ((rc = check_ws(workspace, workspace_bytes))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
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
  p.pe_units = q_pe ? (n_heads + 4 * kSteps - 1) / (4 * kSteps) : 0;
  const int per = (p.idx_fp8 ? 2 : 4) * kSteps;
  p.units = p.pe_units + (q_raw ? (h_idx + per - 1) / per : 0);
  p.first_reports = rows <= kReportRows;
  if (!p.first_reports && cudaMemsetAsync(workspace, 0, 4, st) != cudaSuccess) return SMLA_ERR_CUDA;
  const long long warps = static_cast<long long>(rows) * p.units;
  const unsigned blocks = static_cast<unsigned>((warps + kRowThreads / 32 - 1) / (kRowThreads / 32)) + p.first_reports;
  query_prep_kernel<<<blocks, kRowThreads, 0, st>>>(p);
  return launched();
}

}  // extern "C"
