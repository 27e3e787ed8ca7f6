// Log probabilities of tokens, entropies and the largest logits (kie_paged.cu holds the C entry).
#include "kie_device.cuh"
#include "kie_paged.cuh"

namespace kie {
namespace {

constexpr int LP_THREADS = 256, LP_WARPS = LP_THREADS / 32;

__device__ __forceinline__ float logit(const kie_token_logprobs_args &a, int64_t at) {
  if (a.dtype == KIE_F32) return static_cast<const float *>(a.logits)[at];
  if (a.dtype == KIE_F16) return __half2float(static_cast<const __half *>(a.logits)[at]);
  return __bfloat162float(static_cast<const __nv_bfloat16 *>(a.logits)[at]);
}

// A logit as an unsigned integer of the same order, NaN above +inf and -0 as 0.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t order) {
  return order == 0xffffffffu ? __uint_as_float(0x7fc00000u) : __uint_as_float(order & 0x80000000u ? order ^ 0x80000000u : ~order);
}

template <class T, class F>
__device__ __forceinline__ T block_reduce(T v, const F &f) {
  __shared__ T s_part[LP_WARPS];
#pragma unroll
  for (int o = 16; o; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = s_part[0];
#pragma unroll
  for (int w = 1; w < LP_WARPS; ++w) v = f(v, s_part[w]);
  return v;
}

__global__ void __launch_bounds__(LP_THREADS) token_logprobs_kernel(const kie_token_logprobs_args a) {
  begin_after_previous();
  const int64_t row = blockIdx.x, base = row * a.row_stride;
  const int tid = threadIdx.x;
  uint32_t top = 0;
  for (int i = tid; i < a.vocab; i += LP_THREADS) top = max(top, order_of(logit(a, base + i)));
  top = block_reduce(top, [](uint32_t x, uint32_t y) { return max(x, y); });
  const float m = value_of(top);
  const bool none = m == -INFINITY;
  float s = 0.f, t = 0.f;
  for (int i = tid; i < a.vocab; i += LP_THREADS) {
    const float d = logit(a, base + i) - m, w = expf(d);
    s += w;
    if (w != 0.f) t += w * d;
  }
  s = block_reduce(s, [](float x, float y) { return x + y; });
  t = block_reduce(t, [](float x, float y) { return x + y; });
  const float ls = none ? 0.f : logf(s);
  if (tid == 0) {
    if (a.entropy) a.entropy[row] = none ? 0.f : ls - t / s;
    if (a.logprob) {
      const int token = a.tokens[row];
      a.logprob[row] = (unsigned)token >= (unsigned)a.vocab ? 0.f : none ? -INFINITY : logit(a, base + token) - m - ls;
    }
  }
  unsigned long long last = ~0ull;
  for (int k = 0; k < a.top; ++k) {
    unsigned long long best = 0;
    for (int i = tid; i < a.vocab; i += LP_THREADS) {
      const unsigned long long key = (unsigned long long)order_of(logit(a, base + i)) << 32 | (uint32_t)~i;
      if (key < last && key > best) best = key;
    }
    last = block_reduce(best, [](unsigned long long x, unsigned long long y) { return max(x, y); });
    if (tid == 0) {
      a.top_ids[row * a.top + k] = (int)~(uint32_t)last;
      a.top_logprobs[row * a.top + k] = none ? -INFINITY : value_of((uint32_t)(last >> 32)) - m - ls;
    }
  }
}

}  // namespace
}  // namespace kie

cudaError_t kie_launch_token_logprobs(const kie_token_logprobs_args &a, int, cudaStream_t stream) {
  return kie::launch_after_previous(kie::token_logprobs_kernel, a.n_rows, kie::LP_THREADS, 0, stream, a);
}
