// Helpers of the kernels that move rows (serve.cu, rows.cu): bf16 pairs, how a
// launch reports rows that it skips, checks of the workspace.
#pragma once
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "serve.h"

namespace smla {

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf_pack(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
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

inline int check_ws(void* workspace, size_t bytes) {
  return !workspace || !aligned_to(workspace, 16) || bytes < kStatusBytes ? SMLA_ERR_WORKSPACE : SMLA_OK;
}

inline int launched() { return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA; }

}  // namespace smla
