// Helpers of the serving calls (serve.cu, prefix.cu).
#pragma once
#include <cstdint>

#include "../../include/smla_serve.h"
#include "internal.h"

namespace smla {

inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Argument checks of a cache whose latent rows (need_kv) and indexer keys (need_idx)
// the call uses: the rules of smla.h.
inline int check_serve_cache(const smla_paged_cache* c, bool need_kv, bool need_idx) {
  if (!c || c->page_size <= 0 || c->num_pages <= 0) return SMLA_ERR_INVALID_ARG;
  if (c->page_size != kPage || c->num_pages > (1 << 25)) return SMLA_ERR_UNSUPPORTED;  // pool rows are int32
  if (need_kv) {
    const bool known = c->kv_dtype == SMLA_BF16 || c->kv_dtype == SMLA_FP8_E4M3 || c->kv_dtype == SMLA_FP8_DS_MLA;
    if (!known || !c->kv || !aligned_to(c->kv, 16)) return SMLA_ERR_INVALID_ARG;
    if (c->kv_dtype == SMLA_FP8_E4M3 && (!c->kv_scale || !aligned_to(c->kv_scale, 4))) return SMLA_ERR_INVALID_ARG;
  }
  if (need_idx) {
    const bool bf16 = c->idx_dtype == SMLA_BF16;
    if ((!bf16 && c->idx_dtype != SMLA_FP8_E4M3) || !c->k_idx || !aligned_to(c->k_idx, 16) || !aligned_to(c->k_idx_scale, 4) ||
        c->d_idx <= 0)
      return SMLA_ERR_INVALID_ARG;
    if (c->d_idx * (bf16 ? 2 : 1) != kIdxRowBytes) return SMLA_ERR_UNSUPPORTED;
  }
  return SMLA_OK;
}

// packed fp32: two independent IEEE operations an instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

}  // namespace smla
