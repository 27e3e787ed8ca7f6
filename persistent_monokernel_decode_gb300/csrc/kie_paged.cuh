// Shared by the paged-cache operators: element conversion between the cache and activation types, and the launch
// functions that the C entry points (kie_paged.cu) call.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kie.h"

namespace kie {

constexpr int PAGED_MAX_GROUP = 8;   // query heads per KV head
constexpr int PAGED_ROWS = 16;       // block_size is a multiple: a 16-position tile never crosses a page

__host__ __device__ __forceinline__ int paged_dtype_bytes(int dtype) {
  return dtype == KIE_F32 ? 4 : dtype == KIE_E4M3 ? 1 : 2;
}

// One element of an activation tensor (uniform dtype) as fp32, and back, rounded to nearest even.
__device__ __forceinline__ float paged_load(const void *p, int64_t i, int dtype) {
  if (dtype == KIE_F32) return static_cast<const float *>(p)[i];
  if (dtype == KIE_F16) return __half2float(static_cast<const __half *>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
__device__ __forceinline__ void paged_store(void *p, int64_t i, int dtype, float v) {
  if (dtype == KIE_F32)
    static_cast<float *>(p)[i] = v;
  else if (dtype == KIE_F16)
    static_cast<__half *>(p)[i] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ float paged_from_e4m3(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

}  // namespace kie

cudaError_t kie_launch_paged_attention(const kie_paged_attention_args &a, cudaStream_t stream);
size_t kie_paged_attention_workspace_bytes(int n_heads, int n_kv_heads, int head_dim, int sms);
