// Rows around the expanded form of latent attention: rotation tables
// (smla_rope_table), rotation of a part of each head (smla_rope_apply), rows of the
// paged cache back as bf16 values (smla_cache_read). Each value is read and written
// once: bound by memory, and by latency for few rows.
#include <algorithm>
#include <climits>
#include <cmath>

#include "../../include/smla_prompt.h"
#include "rows.cuh"

namespace smla {
namespace {

// ---------------------------------------------------------------------------- rotation tables
constexpr int kMaxDim = 256;
constexpr int kTableThreads = 256;

struct TableParams {
  float* out;
  uint64_t first;
  int32_t n, dim;
  float magnitude;
  uint64_t turns[kMaxDim / 2];  // of each pair per position, in 2^-64 turns
};

// cos and sin of angle / 2^64 turns. The nearest quarter of a turn is taken off, exactly; what is left, at most
// an eighth, becomes a float (three roundings) and goes into the Taylor series of sin and cos
// up to x^9 and x^10, which are off by 2^-29 there: 2.4 * 2^-24 altogether at most (1.8 * 2^-24 over 80 million angles).
__device__ __forceinline__ void cos_sin_of(uint64_t angle, float& c, float& s) {
  const uint64_t up = angle + (1ull << 61);
  const int32_t rest = static_cast<int32_t>(static_cast<uint32_t>((up << 2) >> 32) ^ 0x80000000u);  // - 1/8 .. 1/8 turn in 2^-34 turns
  const float x = static_cast<float>(rest) * (0x1p-34f * 6.28318530717958648f), t = x * x;
  const float sn = x * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), 1.0f);
  const float cs = fmaf(t, fmaf(t, fmaf(t, fmaf(t, fmaf(t, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
  const uint32_t quarter = static_cast<uint32_t>(up >> 62);
  const float a = quarter & 1 ? sn : cs, b = quarter & 1 ? cs : sn;
  c = __uint_as_float(__float_as_uint(a) ^ ((quarter + 1 & 2) << 30));  // quarters 1 and 2
  s = __uint_as_float(__float_as_uint(b) ^ ((quarter & 2) << 30));      // quarters 2 and 3
}

// A thread keeps four pairs and walks the rows: position * turns wraps at whole
// turns by itself in 64-bit integers, so the angle needs no reduction and goes on by additions.
// Bound by memory: 1,048,576 positions of 64 values, 268 MB written in 45 us, 6.0 TB/s (55 us with
// sincospif, by instructions); 8,192 positions in 2.4 us.
__global__ void __launch_bounds__(kTableThreads) rope_table_kernel(const __grid_constant__ TableParams p) {
  const int groups = p.dim / 8, half = p.dim / 2;  // groups of four pairs
  const int g = threadIdx.x % groups, r0 = threadIdx.x / groups, per = kTableThreads / groups;
  if (r0 >= per) return;
  const long long step = static_cast<long long>(gridDim.x) * per;
  long long r = static_cast<long long>(blockIdx.x) * per + r0;
  uint64_t w[4], at[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t turns = p.turns[4 * g + i];
    at[i] = (p.first + static_cast<uint64_t>(r)) * turns;
    w[i] = static_cast<uint64_t>(step) * turns;
  }
  float* o = p.out + r * p.dim + 4 * g;
#pragma unroll 2
  for (; r < p.n; r += step, o += step * p.dim) {
    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cos_sin_of(at[i], c[i], s[i]);
      at[i] += w[i];
      c[i] *= p.magnitude;
      s[i] *= p.magnitude;
    }
    *reinterpret_cast<float4*>(o) = make_float4(c[0], c[1], c[2], c[3]);
    *reinterpret_cast<float4*>(o + half) = make_float4(s[0], s[1], s[2], s[3]);
  }
}

// ---------------------------------------------------------------------------- rotation
constexpr int kRopeThreads = 128;
constexpr int kRopeSteps = 4;  // heads a thread

struct RopeParams {
  const float* cos_sin;
  int32_t max_pos, dim, inter, rows;
  const int32_t* positions;
  const uint16_t* x;
  long long x_row, x_head;
  uint16_t* out;
  long long o_row, o_head;
  int32_t n_heads, subs, heads_a;  // threads a head, heads a step
  uint32_t* status;
  int32_t first_reports;
};

// A thread takes eight values (four pairs) of up to four heads of one row, all requested
// before the row's position and angles, which are two latencies away. Bound by memory: 8,192 rows of 64
// heads (64 of 192 values each), 136 MB in 26.7 us, 5.1 TB/s. On cold caches with two / four / eight heads
// a thread 32.4 / 28.3 / 28.3 us, in blocks of 256 threads 29.3; 128 rows 2.4 us.
__global__ void __launch_bounds__(kRopeThreads) rope_apply_kernel(const RopeParams p) {
  if (p.first_reports && blockIdx.x == 0) {
    report_rows(p.rows, p.status, [&](int r) {
      const int pos = __ldg(p.positions + r);
      return pos != -1 && (pos < 0 || pos >= p.max_pos);
    });
    return;
  }
  const long long id = static_cast<long long>(blockIdx.x - p.first_reports) * kRopeThreads + threadIdx.x;
  const int per_row = p.subs * p.heads_a;
  const long long row = id / per_row;
  if (row >= p.rows) return;
  const int in = static_cast<int>(id - row * per_row), h0 = in / p.subs, sub = in - h0 * p.subs;
  const int a = p.inter ? 8 * sub : 4 * sub, b = p.inter ? 8 * sub + 4 : p.dim / 2 + 4 * sub;
  const uint16_t* x = p.x + row * p.x_row;
  uint2 wa[kRopeSteps], wb[kRopeSteps];
#pragma unroll
  for (int j = 0; j < kRopeSteps; ++j) {
    const int h = h0 + j * p.heads_a;
    if (h < p.n_heads) {
      wa[j] = *reinterpret_cast<const uint2*>(x + h * p.x_head + a);
      wb[j] = *reinterpret_cast<const uint2*>(x + h * p.x_head + b);
    }
  }
  const int pos = __ldg(p.positions + row);
  if (pos < 0 || pos >= p.max_pos) {
    if (pos != -1 && !p.first_reports) set_status(p.status, kStatusBounds);
    return;
  }
  const float* cs = p.cos_sin + static_cast<long long>(pos) * p.dim + 4 * sub;
  const float4 c = __ldg(reinterpret_cast<const float4*>(cs)), s = __ldg(reinterpret_cast<const float4*>(cs + p.dim / 2));
  auto turn = [](float& u, float& v, float co, float si) {
    const float t = u * co - v * si;
    v = u * si + v * co;
    u = t;
  };
#pragma unroll
  for (int j = 0; j < kRopeSteps; ++j) {
    const int h = h0 + j * p.heads_a;
    if (h >= p.n_heads) break;
    float v[8] = {bf_lo(wa[j].x), bf_hi(wa[j].x), bf_lo(wa[j].y), bf_hi(wa[j].y),
                  bf_lo(wb[j].x), bf_hi(wb[j].x), bf_lo(wb[j].y), bf_hi(wb[j].y)};
    if (p.inter) {
      turn(v[0], v[1], c.x, s.x), turn(v[2], v[3], c.y, s.y), turn(v[4], v[5], c.z, s.z), turn(v[6], v[7], c.w, s.w);
    } else {
      turn(v[0], v[4], c.x, s.x), turn(v[1], v[5], c.y, s.y), turn(v[2], v[6], c.z, s.z), turn(v[3], v[7], c.w, s.w);
    }
    uint16_t* o = p.out + row * p.o_row + h * p.o_head;
    *reinterpret_cast<uint2*>(o + a) = make_uint2(bf_pack(v[0], v[1]), bf_pack(v[2], v[3]));
    *reinterpret_cast<uint2*>(o + b) = make_uint2(bf_pack(v[4], v[5]), bf_pack(v[6], v[7]));
  }
}

// ---------------------------------------------------------------------------- cache rows
constexpr int kReadThreads = 256, kReadRows = 32;
constexpr int kTileRow = 656, kTileRopeAt = 528;

struct ReadParams {
  const uint8_t* kv;
  const float* kv_scale;
  const uint8_t* k_idx;
  const float* k_idx_scale;
  int32_t num_pages, kv_dtype, idx_fp8, d_idx;
  const int32_t* tables;
  int32_t max_pages, n_seqs;
  const int32_t* cu;
  int32_t rows;
  const int32_t* starts;
  uint16_t* latent;
  long long latent_stride;
  uint16_t* pe;
  long long pe_stride;
  uint16_t* keys;
  long long keys_stride;
  uint32_t* status;
  int32_t first_reports;
};

// eight e4m3 codes times a scale, as bf16
__device__ __forceinline__ uint4 widen8(uint2 c, float s) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t pair = static_cast<uint16_t>((i < 2 ? c.x : c.y) >> (16 * (i & 1)));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(pair));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    o[i] = bf_pack(f.x * s, f.y * s);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// A block finds the pool rows of 32 output rows: every request's first row is loaded once
// and counted against them (one latency up to 255 requests, whose work is requests x rows / 32 loads; a search would
// be eight latencies one after the other), then the rows' pieces of 16 bytes of the pool
// go round the block's threads, each thread's requested together. Bound by memory: 131,072 FP8 rows, 227 MB in
// 41 us, 5.6 TB/s; 37 ragged requests of BF16 rows and keys, 102 MB in 22.6 us (1,184 blocks, each a chain of bounds,
// table, place and data, and the keys a second round); few rows by those latencies (600 rows: 4.5 us).
// Batches of two / three / five / nine pieces a thread, 131,072 rows on the device: BF16 50.2 / 49.3 / 49.2 / 68.7 us,
// FP8 38.9 / 38.9 / 47.1 / 47.1, tile-scaled 40.6 / 45.5 / 56.9 / 56.9 (registers); blocks of 16 rows took the FP8
// rows 46.8 us on cold caches, of 128 threads 44.7 (both with batches of five, which took 51.9).
// Programmatic launch after clear_kernel: who reports waits for it, and the first block does, so that the launch is not
// over before the word is cleared (what comes next on the stream may write it).
__global__ void clear_kernel(uint32_t* status) {
  asm volatile("griddepcontrol.launch_dependents;");
  *status = 0;
}
__device__ __forceinline__ void report(uint32_t* status) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  set_status(status, kStatusBounds);
}

// Pool row of token t of request b; -1: there is none.
__device__ __forceinline__ long long pool_row(const ReadParams& p, int b, long long t) {
  if (t < 0 || t / kPage >= p.max_pages) return -1;
  const int id = __ldg(p.tables + static_cast<long long>(b) * p.max_pages + t / kPage);
  return id >= 0 && id < p.num_pages ? static_cast<long long>(id) * kPage + t % kPage : -1;
}

// What no row shows: the list's order and its end.
__device__ __forceinline__ bool bad_bounds(const ReadParams& p) {
  bool bad = false;
  for (int i = threadIdx.x; i <= p.n_seqs; i += kReadThreads) {
    const int c = __ldg(p.cu + i);
    bad |= c < 0 || c > p.rows || (i > 0 && c < __ldg(p.cu + i - 1));
  }
  return bad;
}

// Up to kReportedRows rows of kReportedSeqs requests the first block only looks all of them over and writes the
// status word: no launch to clear it (about 2 us of a 12 us call).
constexpr int kReportedRows = 1024, kReportedSeqs = 1023;

__device__ __forceinline__ void report_all(const ReadParams& p) {
  __shared__ int cu[kReportedSeqs + 1];
  bool bad = bad_bounds(p);
  for (int i = threadIdx.x; i <= p.n_seqs; i += kReadThreads) cu[i] = __ldg(p.cu + i);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kReportedRows / kReadThreads; ++i) {
    const int r = threadIdx.x + i * kReadThreads;
    if (r >= p.rows || r < cu[0] || r >= cu[p.n_seqs]) continue;
    int lo = 0, hi = p.n_seqs;  // cu[lo] <= r < cu[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] <= r) lo = mid; else hi = mid;
    }
    bad |= pool_row(p, lo, static_cast<long long>(p.starts ? __ldg(p.starts + lo) : 0) + (r - cu[lo])) < 0;
  }
  const int found = __syncthreads_or(bad);
  if (threadIdx.x == 0) *p.status = found ? kStatusBounds : 0u;
}

// `pieces` pieces a row of the block's rows: load(place, piece) -> T, store(row, piece, T)
template <int BATCH, typename T, typename Load, typename Store>
__device__ __forceinline__ void each_piece(int pieces, const long long* place, Load load, Store store) {
  const int total = kReadRows * pieces;
  for (int u0 = threadIdx.x; u0 < total; u0 += BATCH * kReadThreads) {
    T v[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int u = u0 + i * kReadThreads, r = u / pieces;
      if (u < total && place[r] >= 0) v[i] = load(place[r], u - r * pieces);
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int u = u0 + i * kReadThreads, r = u / pieces;
      if (u < total && place[r] != -2) store(r, u - r * pieces, v[i], place[r] >= 0);
    }
  }
}

template <int FMT>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const ReadParams p) {
  __shared__ int begun[kReadRows + 1];      // requests that begin at or before the block's first row, then at each row
  __shared__ long long place[kReadRows];    // pool row; -1: zeros; -2: left as it is
  const int tid = threadIdx.x, lane = tid & 31;
  if (p.first_reports && blockIdx.x == 0) {
    report_all(p);
    return;
  }
  const int r0 = (blockIdx.x - p.first_reports) * kReadRows;
  for (int i = tid; i <= kReadRows; i += kReadThreads) begun[i] = 0;
  __syncthreads();
  int before = 0;
  for (int i = tid; i <= p.n_seqs; i += kReadThreads) {
    const int c = __ldg(p.cu + i);
    if (c <= r0) ++before;
    else if (c - r0 < kReadRows) atomicAdd(&begun[1 + c - r0], 1);
  }
  before = __reduce_add_sync(0xFFFFFFFFu, before);
  if (lane == 0 && before) atomicAdd(&begun[0], before);
  __syncthreads();
  if (tid < kReadRows) {
    const int r = r0 + tid;
    int n = begun[1 + tid];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, n, d);
      if (tid >= d) n += o;
    }
    const int b = begun[0] + n - 1;
    long long at = -2;
    bool bad = false;
    if (r < p.rows && b >= 0 && b < p.n_seqs) {
      const int first = __ldg(p.cu + b), last = __ldg(p.cu + b + 1);
      if (r < first || r >= last) {  // (an order that runs backwards: the counts do not fit)
        bad = true;
      } else {
        at = pool_row(p, b, static_cast<long long>(p.starts ? __ldg(p.starts + b) : 0) + (r - first));
        bad = at < 0;
      }
    }
    place[tid] = at;
    if (bad && !p.first_reports) report(p.status);
  }
  if (!p.first_reports && blockIdx.x == 0) {
    if (bad_bounds(p)) report(p.status);
    asm volatile("griddepcontrol.wait;" ::: "memory");
  }
  __syncthreads();
  const uint4 none = make_uint4(0, 0, 0, 0);
  auto to_latent = [&](int r, int j, uint4 v) { *reinterpret_cast<uint4*>(p.latent + (r0 + r) * p.latent_stride + 8 * j) = v; };
  auto to_pe = [&](int r, int j, uint4 v) { *reinterpret_cast<uint4*>(p.pe + (r0 + r) * p.pe_stride + 8 * j) = v; };
  if (FMT == SMLA_BF16) {
    const int first = p.latent ? 0 : 64, pieces = (p.pe ? 72 : 64) - first;  // of those that are wanted
    if (pieces > 0)
      each_piece<3, uint4>(pieces, place, [&](long long at, int j) { return __ldg(reinterpret_cast<const uint4*>(p.kv + at * (2 * kDqk)) + first + j); },
                           [&](int r, int j, uint4 v, bool there) {
                             j += first;
                             if (j < 64) to_latent(r, j, there ? v : none);
                             else to_pe(r, j - 64, there ? v : none);
                           });
  } else if (FMT == SMLA_FP8_E4M3) {
    const int first = p.latent ? 0 : 32, pieces = (p.pe ? 36 : 32) - first;  // sixteen codes each
    struct Got {
      uint4 c;
      float s;
    };
    if (pieces > 0)
      each_piece<3, Got>(pieces, place,
                         [&](long long at, int j) {
                           return Got{__ldg(reinterpret_cast<const uint4*>(p.kv + at * kDqk) + first + j), __ldg(p.kv_scale + at)};
                         },
                         [&](int r, int j, Got v, bool there) {
                           j += first;
                           const uint4 a = there ? widen8(make_uint2(v.c.x, v.c.y), v.s) : none, b = there ? widen8(make_uint2(v.c.z, v.c.w), v.s) : none;
                           if (j < 32) to_latent(r, 2 * j, a), to_latent(r, 2 * j + 1, b);
                           else to_pe(r, 2 * (j - 32), a), to_pe(r, 2 * (j - 32) + 1, b);
                         });
  } else if (FMT == SMLA_FP8_DS_MLA) {
    struct Got {
      uint4 c;
      float s;
    };
    const int first = p.latent ? 0 : 32, pieces = (p.pe ? 40 : 32) - first;  // sixteen codes or eight rope values each
    if (pieces > 0)
      each_piece<3, Got>(pieces, place,
                         [&](long long at, int j) {
                           const uint8_t* row = p.kv + at * kTileRow;
                           j += first;
                           return Got{__ldg(reinterpret_cast<const uint4*>(row + (j < 32 ? 0 : kTileRopeAt - kDv)) + j),
                                      j < 32 ? __ldg(reinterpret_cast<const float*>(row + kDv) + (j >> 3)) : 1.0f};
                         },
                         [&](int r, int j, Got v, bool there) {
                           j += first;
                           if (j < 32) {
                             to_latent(r, 2 * j, there ? widen8(make_uint2(v.c.x, v.c.y), v.s) : none);
                             to_latent(r, 2 * j + 1, there ? widen8(make_uint2(v.c.z, v.c.w), v.s) : none);
                           } else {
                             to_pe(r, j - 32, there ? v.c : none);
                           }
                         });
  }
  if (!p.keys) return;
  auto to_keys = [&](int r, int j, uint4 v) { *reinterpret_cast<uint4*>(p.keys + (r0 + r) * p.keys_stride + 8 * j) = v; };
  struct Got {
    uint4 c;
    float s;
  };
  each_piece<2, Got>(8, place,
                     [&](long long at, int j) {
                       return Got{__ldg(reinterpret_cast<const uint4*>(p.k_idx + at * kIdxRowBytes) + j), p.k_idx_scale ? __ldg(p.k_idx_scale + at) : 1.0f};
                     },
                     [&](int r, int j, Got v, bool there) {
                       if (p.idx_fp8) {
                         to_keys(r, 2 * j, there ? widen8(make_uint2(v.c.x, v.c.y), v.s) : none);
                         to_keys(r, 2 * j + 1, there ? widen8(make_uint2(v.c.z, v.c.w), v.s) : none);
                         return;
                       }
                       uint32_t w[4] = {v.c.x, v.c.y, v.c.z, v.c.w};
                       if (p.k_idx_scale)
#pragma unroll
                         for (int i = 0; i < 4; ++i) w[i] = bf_pack(bf_lo(w[i]) * v.s, bf_hi(w[i]) * v.s);
                       to_keys(r, j, there ? make_uint4(w[0], w[1], w[2], w[3]) : none);
                     });
}

// Whether two of the places of `dim` values at i * row + h * head (both strides at least dim where they are used) overlap.
bool places_overlap(int64_t rows, int64_t row, int64_t heads, int64_t head, int64_t dim) {
  typedef __int128 Wide;
  if (rows == 1 || heads == 1) return false;
  const Wide all_rows = static_cast<Wide>(rows - 1) * row, all_heads = static_cast<Wide>(heads - 1) * head;
  if (row >= all_heads + dim || head >= all_rows + dim) return false;  // heads inside a row, rows inside a head
  for (int64_t h = 1; h < heads; ++h) {  // the rows on both sides of a head's distance
    const Wide at = static_cast<Wide>(h) * head, below = at / row, rest = at % row;
    if (at >= all_rows + dim) break;
    if ((below < rows && rest < dim) || (below + 1 < rows && row - rest < dim)) return true;
  }
  return false;
}

bool strided(const void* p, int64_t stride, int64_t width) { return aligned_to(p, 16) && stride % 8 == 0 && stride >= width; }

}  // namespace
}  // namespace smla

using namespace smla;

extern "C" {

int smla_rope_table(float* cos_sin, int64_t first, int32_t n, int32_t dim, double base, double factor,
                    int32_t original, double beta_fast, double beta_slow, float magnitude, void* stream) {
  if (!cos_sin || !aligned_to(cos_sin, 16) || n <= 0 || first < 0 || dim <= 0 || original < 0) return SMLA_ERR_INVALID_ARG;
  if (!(base > 1.0) || !(factor >= 1.0) || !std::isfinite(base) || !std::isfinite(factor) || !std::isfinite(magnitude)) return SMLA_ERR_INVALID_ARG;
  if (original > 0 && (!(beta_slow > 0.0) || !(beta_fast >= beta_slow) || !std::isfinite(beta_fast))) return SMLA_ERR_INVALID_ARG;
  if (dim % 8 || dim > kMaxDim || first > (1LL << 31) - n) return SMLA_ERR_UNSUPPORTED;
  TableParams p{};
  p.out = cos_sin, p.first = static_cast<uint64_t>(first), p.n = n, p.dim = dim, p.magnitude = magnitude;
  const double two_pi = 6.283185307179586476925;
  double low = 0.0, high = 0.0;
  if (original > 0) {
    const double at_fast = dim * std::log(original / (beta_fast * two_pi)) / (2.0 * std::log(base));
    const double at_slow = dim * std::log(original / (beta_slow * two_pi)) / (2.0 * std::log(base));
    low = std::max(std::floor(at_fast), 0.0);
    high = std::min(std::ceil(at_slow), dim - 1.0);
  }
  for (int i = 0; i < dim / 2; ++i) {
    double w = std::pow(base, -2.0 * i / dim);
    if (original > 0) {
      const double r = std::min(1.0, std::max(0.0, (i - low) / std::max(high - low, 0.001)));
      w = w * (1.0 - r) + w / factor * r;
    } else {
      w /= factor;
    }
    // w / (2 pi) < 1/6 of a turn; off by 2^-52 of it, as w itself may be
    p.turns[i] = static_cast<uint64_t>(w * (0.15915494309189533577 * 0x1p64));
  }
  const int per = kTableThreads / (dim / 8);
  const long long blocks = (static_cast<long long>(n) + per - 1) / per;
  const unsigned grid = static_cast<unsigned>(std::min<long long>(blocks, 8LL * num_sms()));
  rope_table_kernel<<<grid, kTableThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return launched();
}

int smla_rope_apply(const float* cos_sin, int32_t max_pos, int32_t dim, int32_t interleaved, int32_t rows,
                    const int32_t* positions, const void* x, int64_t x_row, int64_t x_head, int32_t n_heads,
                    void* out, int64_t out_row, int64_t out_head, void* workspace, size_t workspace_bytes, void* stream) {
  if (!cos_sin || !positions || !x || !out || !aligned_to(cos_sin, 16) || !aligned_to(positions, 4) || !aligned_to(x, 16) || !aligned_to(out, 16))
    return SMLA_ERR_INVALID_ARG;
  if (max_pos <= 0 || rows <= 0 || n_heads <= 0 || dim <= 0) return SMLA_ERR_INVALID_ARG;
  if (dim % 8 || dim > kMaxDim) return SMLA_ERR_UNSUPPORTED;
  if (x_row % 8 || x_head % 8 || out_row % 8 || out_head % 8 || x_row < 0 || out_row < 0) return SMLA_ERR_INVALID_ARG;
  if (n_heads > 1 && (x_head < dim || out_head < dim)) return SMLA_ERR_INVALID_ARG;
  if (rows > 1 && out_row < dim) return SMLA_ERR_INVALID_ARG;
  if (places_overlap(rows, out_row, n_heads, out_head, dim)) return SMLA_ERR_INVALID_ARG;
  if (out == x && (x_row != out_row || x_head != out_head)) return SMLA_ERR_INVALID_ARG;
  if (const int rc = check_ws(workspace, workspace_bytes)) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  RopeParams p{};
  p.cos_sin = cos_sin, p.max_pos = max_pos, p.dim = dim, p.inter = interleaved, p.rows = rows, p.positions = positions;
  p.x = static_cast<const uint16_t*>(x), p.x_row = x_row, p.x_head = x_head;
  p.out = static_cast<uint16_t*>(out), p.o_row = out_row, p.o_head = out_head;
  p.n_heads = n_heads, p.subs = dim / 8, p.heads_a = (n_heads + kRopeSteps - 1) / kRopeSteps;
  p.status = static_cast<uint32_t*>(workspace);
  p.first_reports = rows <= kReportRows;
  if (static_cast<long long>(p.subs) * p.heads_a > INT_MAX) return SMLA_ERR_UNSUPPORTED;
  const long long threads = static_cast<long long>(rows) * p.subs * p.heads_a;
  const long long blocks = (threads + kRopeThreads - 1) / kRopeThreads + p.first_reports;
  if (blocks > INT_MAX) return SMLA_ERR_UNSUPPORTED;
  if (!p.first_reports && cudaMemsetAsync(workspace, 0, 4, st) != cudaSuccess) return SMLA_ERR_CUDA;
  rope_apply_kernel<<<static_cast<unsigned>(blocks), kRopeThreads, 0, st>>>(p);
  return launched();
}

int smla_cache_read(const smla_paged_cache* cache, const int32_t* page_tables, int32_t max_pages, int32_t n_seqs,
                    const int32_t* cu_rows, int32_t rows, const int32_t* starts, void* latent, int64_t latent_stride,
                    void* pe, int64_t pe_stride, void* keys, int64_t keys_stride, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!latent && !pe && !keys) return SMLA_ERR_INVALID_ARG;
  int rc = check_serve_cache(cache, latent || pe, keys != nullptr);
  if (rc) return rc;
  if (!page_tables || !cu_rows || !aligned_to(page_tables, 4) || !aligned_to(cu_rows, 4) || !aligned_to(starts, 4)) return SMLA_ERR_INVALID_ARG;
  if (max_pages <= 0 || n_seqs <= 0 || rows <= 0) return SMLA_ERR_INVALID_ARG;
  if ((latent && !strided(latent, latent_stride, kDv)) || (pe && !strided(pe, pe_stride, kDqk - kDv)) ||
      (keys && !strided(keys, keys_stride, cache->d_idx)))
    return SMLA_ERR_INVALID_ARG;
  if (rows > INT_MAX - kReadRows || n_seqs == INT_MAX) return SMLA_ERR_UNSUPPORTED;
  if ((rc = check_ws(workspace, workspace_bytes))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  ReadParams p{};
  p.kv = static_cast<const uint8_t*>(cache->kv), p.kv_scale = cache->kv_scale;
  p.k_idx = static_cast<const uint8_t*>(cache->k_idx), p.k_idx_scale = cache->k_idx_scale;
  p.num_pages = cache->num_pages, p.kv_dtype = cache->kv_dtype, p.idx_fp8 = cache->idx_dtype == SMLA_FP8_E4M3, p.d_idx = cache->d_idx;
  p.tables = page_tables, p.max_pages = max_pages, p.n_seqs = n_seqs, p.cu = cu_rows, p.rows = rows, p.starts = starts;
  p.latent = static_cast<uint16_t*>(latent), p.latent_stride = latent_stride;
  p.pe = static_cast<uint16_t*>(pe), p.pe_stride = pe_stride;
  p.keys = static_cast<uint16_t*>(keys), p.keys_stride = keys_stride;
  p.status = static_cast<uint32_t*>(workspace);
  p.first_reports = rows <= kReportedRows && n_seqs <= kReportedSeqs;
  if (!p.first_reports) {
    clear_kernel<<<1, 1, 0, st>>>(p.status);
    if (launched()) return SMLA_ERR_CUDA;
  }
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kReadRows - 1) / kReadRows) + p.first_reports);
  cfg.blockDim = dim3(kReadThreads);
  cfg.stream = st;
  cfg.attrs = &at, cfg.numAttrs = p.first_reports ? 0 : 1;
  const int fmt = latent || pe ? cache->kv_dtype : SMLA_BF16;  // (keys alone: no latent pieces)
  const auto kernel = fmt == SMLA_BF16 ? cache_read_kernel<SMLA_BF16> : fmt == SMLA_FP8_E4M3 ? cache_read_kernel<SMLA_FP8_E4M3> : cache_read_kernel<SMLA_FP8_DS_MLA>;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

}  // extern "C"
