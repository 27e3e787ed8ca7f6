// Shared by the paged-cache operators: rounding to the cache and activation types, and the launch functions that the C entry
// points (kie_paged.cu) call.
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

// An fp32 value as an element of an activation tensor (uniform dtype), rounded to nearest even.
__device__ __forceinline__ void paged_store(void *p, int64_t i, int dtype, float v) {
  if (dtype == KIE_F32)
    static_cast<float *>(p)[i] = v;
  else if (dtype == KIE_F16)
    static_cast<__half *>(p)[i] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ uint32_t pack2(float a, float b, int dtype) {
  if (dtype == KIE_F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Eight consecutive elements at p + i; VEC: p + i is aligned for 16-byte accesses.
template <bool VEC>
__device__ __forceinline__ void store8(void *p, int64_t i, int dtype, const float (&v)[8]) {
  if (!VEC) {
#pragma unroll
    for (int e = 0; e < 8; ++e) paged_store(p, i + e, dtype, v[e]);
    return;
  }
  if (dtype == KIE_F32) {
    float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
  *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) =
      make_uint4(pack2(v[0], v[1], dtype), pack2(v[2], v[3], dtype), pack2(v[4], v[5], dtype), pack2(v[6], v[7], dtype));
}

// The paged-cache kernels are launched so that their blocks may take their places while the kernel before them on the
// stream (one of them, as a rule: each of a step's operators needs the one before) still ends. The first thing a block
// does is to wait, on the device, until everything before it is complete and visible. It saves 0.3 to 0.4 us of each
// (extend of 256 requests 3.8 -> 3.4 us, append of 32 rows 2.4 -> 2.0 us, attention of 64 sequences of 64 6.0 -> 5.7).
// The short kernels let the next one in at once; the attention at the end of each block, for the next one's blocks would
// crowd on the SMs that were free first (the same attention: 8.0 us).
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void begin_after_previous() {
  wait_for_previous();
  let_next_begin();
}

template <class K, class... A>
cudaError_t launch_after_previous(K kernel, unsigned grid, unsigned threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace kie

cudaError_t kie_launch_paged_attention(const kie_paged_attention_args &a, int dev, int sms, cudaStream_t stream);
size_t kie_paged_attention_workspace_bytes(int n_heads, int n_kv_heads, int head_dim, int sms);
