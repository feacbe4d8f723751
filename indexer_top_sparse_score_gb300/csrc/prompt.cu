// Attention over packed prompts in the expanded form (smla_prompt_fwd):
//   o = softmax(sm_scale q K^T) V,  lse = ln sum exp(sm_scale q k)
// a warp for each (token, head), which walks the token's keys with a running maximum and sum.
#include <algorithm>
#include <climits>
#include <cmath>

#include "../../include/smla_prompt.h"
#include "rows.cuh"

namespace smla {
namespace {

constexpr int kVal = 128;   // values of a head's v
constexpr int kPe = 64;

struct PromptParams {
  const uint16_t *q, *k, *v, *pe;
  long long q_row, q_head, k_row, k_head, v_row, v_head, pe_row;
  int32_t total_q, total_k, n_seqs;
  const int32_t *cu_q, *cu_k;
  int32_t n_heads, group, d_qk, d_k, causal;
  float sm_scale;
  const float *prev_out, *prev_lse;
  void* out;
  int32_t out_fp32;
  float* lse;
  uint32_t* status;
};

__device__ __forceinline__ float bf_at(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }

__global__ void __launch_bounds__(128) prompt_kernel(const PromptParams p) {
  const int lane = threadIdx.x & 31;
  const long long id = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const long long rows = static_cast<long long>(p.total_q) * p.n_heads;
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < p.n_seqs; b += 128) {
      const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], k0 = p.cu_k[b], k1 = p.cu_k[b + 1];
      if (q0 < 0 || q1 < q0 || q1 > p.total_q || k0 < 0 || k1 < k0 || k1 > p.total_k) set_status(p.status, kStatusBounds);
    }
  }
  if (id >= rows) return;
  const int token = static_cast<int>(id / p.n_heads), h = static_cast<int>(id - static_cast<long long>(token) * p.n_heads);
  int b = -1, q0 = 0, q1 = 0, k0 = 0, k1 = 0;
  for (int i = 0; i < p.n_seqs; ++i) {
    q0 = p.cu_q[i], q1 = p.cu_q[i + 1], k0 = p.cu_k[i], k1 = p.cu_k[i + 1];
    if (q0 < 0 || q1 < q0 || q1 > p.total_q || k0 < 0 || k1 < k0 || k1 > p.total_k) continue;
    if (token >= q0 && token < q1) {
      b = i;
      break;
    }
  }
  if (b < 0) return;
  const int seen = p.causal ? max(0, k1 - k0 - (q1 - q0) + token - q0 + 1) : k1 - k0;
  const int g = h / p.group;
  float x[6];
#pragma unroll
  for (int i = 0; i < 6; ++i) x[i] = 32 * i + lane < p.d_qk ? bf_at(p.q + token * p.q_row + h * p.q_head + 32 * i + lane) : 0.0f;
  float m = -INFINITY, l = 0.0f, o[4] = {0, 0, 0, 0};
  for (int j = 0; j < seen; ++j) {
    const long long kj = k0 + j;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      const int d = 32 * i + lane;
      if (d < p.d_k) dot += x[i] * bf_at(p.k + kj * p.k_row + g * p.k_head + d);
      else if (d < p.d_qk) dot += x[i] * bf_at(p.pe + kj * p.pe_row + d - p.d_k);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, s);
    dot *= p.sm_scale;
    const float top = fmaxf(m, dot);
    const float alpha = m == -INFINITY ? 0.0f : expf(m - top), w = top == -INFINITY ? 0.0f : expf(dot - top);
    m = top;
    l = l * alpha + w;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = o[i] * alpha + w * bf_at(p.v + kj * p.v_row + g * p.v_head + 32 * i + lane);
  }
  float lse = l != 0.0f ? m + logf(l) : -INFINITY, f = l != 0.0f ? 1.0f / l : 0.0f, fp = 0.0f;
  if (p.prev_lse) {
    const float was = p.prev_lse[id], top = fmaxf(was, lse);
    if (was != -INFINITY) {
      const float both = l != 0.0f ? top + logf(expf(was - top) + expf(lse - top)) : was;
      f *= expf(lse - both);
      fp = expf(was - both);
      lse = both;
    }
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long at = id * kVal + 32 * i + lane;
    float y = l != 0.0f ? o[i] * f : 0.0f;
    if (fp != 0.0f) y += fp * p.prev_out[at];
    if (p.out_fp32) static_cast<float*>(p.out)[at] = y;
    else static_cast<uint16_t*>(p.out)[at] = static_cast<uint16_t>(bf_pack(y, 0.0f));
  }
  if (lane == 0 && p.lse) p.lse[id] = lse;
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
  (void)total_q, (void)total_k, (void)n_seqs, (void)n_heads, (void)n_kv_heads;
  return kStatusBytes;
}

int smla_prompt_fwd(const smla_heads* q, const smla_heads* k, const smla_heads* v, const void* k_pe,
                    int64_t k_pe_stride, int32_t total_q, int32_t total_k, int32_t n_seqs, const int32_t* cu_q,
                    const int32_t* cu_k, int32_t n_heads, int32_t n_kv_heads, int32_t d_qk, int32_t causal,
                    float sm_scale, const float* prev_out, const float* prev_lse, void* out, int32_t out_fp32,
                    float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (total_q <= 0 || total_k <= 0 || n_seqs <= 0 || n_heads <= 0 || n_kv_heads <= 0 || d_qk <= 0 || n_heads % n_kv_heads) return SMLA_ERR_INVALID_ARG;
  const int d_k = k_pe ? d_qk - kPe : d_qk;
  if (d_qk != 128 && d_qk != 192) return SMLA_ERR_UNSUPPORTED;
  if (n_heads > 1024 || n_seqs > (1 << 24) || total_q > INT_MAX - 1024 || total_k > INT_MAX - 1024) return SMLA_ERR_UNSUPPORTED;
  if (!heads_ok(q, d_qk, n_heads) || !heads_ok(k, d_k, n_kv_heads) || !heads_ok(v, kVal, n_kv_heads)) return SMLA_ERR_INVALID_ARG;
  if (k_pe && (!aligned_to(k_pe, 16) || k_pe_stride % 8 || k_pe_stride < kPe || k_pe_stride >= (1LL << 35))) return SMLA_ERR_INVALID_ARG;
  if (!cu_q || !cu_k || !out || !aligned_to(cu_q, 4) || !aligned_to(cu_k, 4) || !aligned_to(out, 16) || !aligned_to(lse, 4)) return SMLA_ERR_INVALID_ARG;
  if ((prev_out == nullptr) != (prev_lse == nullptr) || !aligned_to(prev_out, 16) || !aligned_to(prev_lse, 4) || !std::isfinite(sm_scale))
    return SMLA_ERR_INVALID_ARG;
  if (static_cast<const void*>(prev_out) == out && out && !out_fp32) return SMLA_ERR_INVALID_ARG;
  if (const int rc = check_ws(workspace, workspace_bytes)) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  PromptParams p{};
  p.q = static_cast<const uint16_t*>(q->data), p.q_row = q->row_stride, p.q_head = q->head_stride;
  p.k = static_cast<const uint16_t*>(k->data), p.k_row = k->row_stride, p.k_head = k->head_stride;
  p.v = static_cast<const uint16_t*>(v->data), p.v_row = v->row_stride, p.v_head = v->head_stride;
  p.pe = static_cast<const uint16_t*>(k_pe), p.pe_row = k_pe_stride;
  p.total_q = total_q, p.total_k = total_k, p.n_seqs = n_seqs, p.cu_q = cu_q, p.cu_k = cu_k;
  p.n_heads = n_heads, p.group = n_heads / n_kv_heads, p.d_qk = d_qk, p.d_k = d_k, p.causal = causal, p.sm_scale = sm_scale;
  p.prev_out = prev_out, p.prev_lse = prev_lse, p.out = out, p.out_fp32 = out_fp32, p.lse = lse;
  p.status = static_cast<uint32_t*>(workspace);
  if (cudaMemsetAsync(workspace, 0, 4, st) != cudaSuccess) return SMLA_ERR_CUDA;
  const long long warps = static_cast<long long>(total_q) * n_heads;
  if ((warps + 3) / 4 > INT_MAX) return SMLA_ERR_UNSUPPORTED;
  prompt_kernel<<<static_cast<unsigned>((warps + 3) / 4), 128, 0, st>>>(p);
  return launched();
}

}  // extern "C"
