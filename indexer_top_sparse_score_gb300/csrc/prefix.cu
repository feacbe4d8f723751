// Attention of a batch over a shared prompt and each request's own tokens
// (smla_shared_prefix_fwd).
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/smla_serve.h"
#include "common.cuh"
#include "internal.h"

namespace smla {
namespace {

struct PrefixParams {
  const uint8_t* kv;
  const float* kv_scale;
  int32_t kv_dtype, num_pages;
  const int32_t* page_tables;
  int32_t max_pages, n_seqs;
  const int32_t* seq_lens;
  int32_t max_seq_len, shared_len, q_per_seq;
  const uint16_t* q;
  float sm_scale;
  uint16_t* out;
  float* lse;
  uint32_t* status;
};

constexpr int kTile = 32;
constexpr int kThreads = 256;

__device__ __forceinline__ float e4m3_value(uint8_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(c)));
  return __half2float(__ushort_as_half(static_cast<uint16_t>(r)));
}

__device__ __forceinline__ float kv_value(const PrefixParams& p, long long row, int d) {
  if (p.kv_dtype == SMLA_BF16)
    return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p.kv)[row * kDqk + d]) << 16);
  if (p.kv_dtype == SMLA_FP8_E4M3) return e4m3_value(p.kv[row * kDqk + d]) * p.kv_scale[row];
  const uint8_t* r = p.kv + row * 656;
  if (d < kDv) return e4m3_value(r[d]) * reinterpret_cast<const float*>(r + kDv)[d >> 7];
  return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(r + 528)[d - kDv]) << 16);
}

// One block per new token: its heads' queries and 32 keys at a time in shared
// memory, running maximum and sum per head, two output columns per thread.
template <int H>
__global__ void __launch_bounds__(kThreads) prefix_simple_kernel(const PrefixParams p) {
  extern __shared__ float sm[];
  float* sq = sm;                   // [H][576]
  float* sk = sq + H * kDqk;        // [32][577]
  float* sp = sk + kTile * (kDqk + 1);  // [H][32]
  float* sa = sp + H * kTile;       // [H] rescale
  const int t = threadIdx.x, row = blockIdx.x, b = row / p.q_per_seq;
  int len = p.seq_lens[b];
  if (len > p.max_seq_len) {
    len = p.max_seq_len;
    if (t == 0) set_status(p.status, kStatusBounds);
  }
  const int n = max(0, len - p.q_per_seq + row - b * p.q_per_seq + 1);
  for (int i = t; i < H * kDqk; i += kThreads)
    sq[i] = __uint_as_float(static_cast<uint32_t>(p.q[static_cast<long long>(row) * H * kDqk + i]) << 16) * p.sm_scale;
  float acc[2 * H];
#pragma unroll
  for (int i = 0; i < 2 * H; ++i) acc[i] = 0.0f;
  float m = -INFINITY, l = 0.0f;  // of head t (t < H)
  for (int k0 = 0; k0 < n; k0 += kTile) {
    __syncthreads();
    for (int i = t; i < kTile * kDqk; i += kThreads) {
      const int k = i / kDqk, d = i - k * kDqk, key = k0 + k;
      float v = 0.0f;
      if (key < n) {
        const int page = p.page_tables[static_cast<long long>(key < p.shared_len ? 0 : b) * p.max_pages + key / kPage];
        if (page >= 0 && page < p.num_pages) v = kv_value(p, static_cast<long long>(page) * kPage + key % kPage, d);
        else if (d == 0) set_status(p.status, kStatusBounds);
      }
      sk[k * (kDqk + 1) + d] = v;
    }
    __syncthreads();
    for (int i = t; i < H * kTile; i += kThreads) {
      const int h = i / kTile, k = i % kTile, key = k0 + k;
      float s = -INFINITY;
      if (key < n) {
        const int page = p.page_tables[static_cast<long long>(key < p.shared_len ? 0 : b) * p.max_pages + key / kPage];
        if (page >= 0 && page < p.num_pages) {
          s = 0.0f;
          for (int d = 0; d < kDqk; ++d) s += sq[h * kDqk + d] * sk[k * (kDqk + 1) + d];
        }
      }
      sp[i] = s;
    }
    __syncthreads();
    if (t < H) {
      float top = m;
      for (int k = 0; k < kTile; ++k) top = fmaxf(top, sp[t * kTile + k]);
      const float ref = top == -INFINITY ? 0.0f : top;
      const float a = expf(m - ref);
      l *= a;
      for (int k = 0; k < kTile; ++k) {
        const float e = expf(sp[t * kTile + k] - ref);
        sp[t * kTile + k] = e;
        l += e;
      }
      m = top;
      sa[t] = a;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < H; ++h) {
      float a0 = acc[2 * h] * sa[h], a1 = acc[2 * h + 1] * sa[h];
#pragma unroll 4
      for (int k = 0; k < kTile; ++k) {
        const float e = sp[h * kTile + k];
        a0 += e * sk[k * (kDqk + 1) + t];
        a1 += e * sk[k * (kDqk + 1) + 256 + t];
      }
      acc[2 * h] = a0, acc[2 * h + 1] = a1;
    }
  }
  __syncthreads();
  if (t < H) {
    sa[t] = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    if (p.lse) p.lse[static_cast<long long>(row) * H + t] = l == 0.0f ? -INFINITY : m + logf(l);
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const __nv_bfloat16 o = __float2bfloat16(sa[h] == 0.0f ? 0.0f : acc[2 * h + j] * sa[h]);
      p.out[(static_cast<long long>(row) * H + h) * kDv + 256 * j + t] = *reinterpret_cast<const uint16_t*>(&o);
    }
}

template <int H>
int launch_simple(const PrefixParams& p, cudaStream_t st) {
  const size_t smem = (static_cast<size_t>(H) * kDqk + kTile * (kDqk + 1) + H * kTile + H) * 4;
  if (cudaFuncSetAttribute(prefix_simple_kernel<H>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
    return SMLA_ERR_CUDA;
  prefix_simple_kernel<H><<<p.n_seqs * p.q_per_seq, kThreads, smem, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

}  // namespace
}  // namespace smla

using namespace smla;

extern "C" {

size_t smla_shared_prefix_fwd_workspace_size(int32_t, int32_t, int32_t, int32_t, int32_t) { return kStatusBytes; }

int smla_shared_prefix_fwd(const smla_paged_cache* cache, const int32_t* page_tables, int32_t max_pages,
                           int32_t n_seqs, const int32_t* seq_lens, int32_t max_seq_len, int32_t shared_len,
                           int32_t q_per_seq, const void* q, int32_t n_heads, float sm_scale, void* out, float* lse,
                           void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_cache(cache, true, false);
  if (rc) return rc;
  auto al = [](const void* a, uintptr_t n) { return (reinterpret_cast<uintptr_t>(a) & (n - 1)) == 0; };
  if (!page_tables || !seq_lens || !q || !out || !al(page_tables, 4) || !al(seq_lens, 4) || !al(q, 16) || !al(out, 16) || !al(lse, 4))
    return SMLA_ERR_INVALID_ARG;
  if (n_seqs <= 0 || q_per_seq <= 0 || max_pages <= 0 || max_seq_len <= 0 || shared_len < 0 || shared_len > max_seq_len)
    return SMLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(max_pages) * kPage < max_seq_len || !(sm_scale == sm_scale)) return SMLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(n_seqs) * q_per_seq * n_heads > INT32_MAX) return SMLA_ERR_UNSUPPORTED;
  if (n_heads != 16 && n_heads != 64) return SMLA_ERR_UNSUPPORTED;
  if (!workspace || !al(workspace, 16) || workspace_bytes < kStatusBytes) return SMLA_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, 4, st) != cudaSuccess) return SMLA_ERR_CUDA;
  PrefixParams p{static_cast<const uint8_t*>(cache->kv), cache->kv_scale, cache->kv_dtype, cache->num_pages, page_tables, max_pages,
                 n_seqs, seq_lens, max_seq_len, shared_len, q_per_seq, static_cast<const uint16_t*>(q), sm_scale,
                 static_cast<uint16_t*>(out), lse, static_cast<uint32_t*>(workspace)};
  return n_heads == 64 ? launch_simple<64>(p, st) : launch_simple<16>(p, st);
}

}  // extern "C"
