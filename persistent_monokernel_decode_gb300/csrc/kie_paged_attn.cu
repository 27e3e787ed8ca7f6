// Attention of one new token per sequence over a paged K/V cache.
#include <float.h>

#include "kie_device.cuh"
#include "kie_paged.cuh"

namespace kie {
namespace {

constexpr int PA_WARPS = 4;

__device__ __forceinline__ float cache_load(const void *p, int64_t i, int dtype) {
  return dtype == KIE_E4M3 ? paged_from_e4m3(static_cast<const uint8_t *>(p)[i]) : paged_load(p, i, dtype);
}

// One block per (sequence, query head); each warp walks every fourth position with its own running maximum and sum,
// a lane holding head_dim / 32 dimensions, and the warps are joined through shared memory.
template <int DH>
__global__ void __launch_bounds__(PA_WARPS * 32) paged_attn_simple(const kie_paged_attention_args a) {
  constexpr int N = DH / 32;
  __shared__ float sm[PA_WARPS], sl[PA_WARPS], so[PA_WARPS][DH];
  const int b = blockIdx.x / a.n_heads, h = blockIdx.x % a.n_heads;
  const int kh = h / (a.n_heads / a.pages.n_kv_heads);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bs = a.pages.block_size;
  const int len = (int)min((int64_t)max(a.lens[b], 0), (int64_t)a.max_blocks * bs);
  const int j0 = a.window > 0 ? max(0, len - a.window) : 0;
  float q[N], o[N], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = paged_load(a.q, b * a.q_stride[0] + h * a.q_stride[1] + lane * N + i, a.q_dtype) * a.scale;
    o[i] = 0.f;
  }
  for (int j = j0 + warp; j < len; j += PA_WARPS) {
    const int64_t page = a.block_table[b * a.table_stride + j / bs];
    if (page < 0 || page >= a.pages.n_blocks) continue;
    const int r = j % bs;
    const int64_t kat = page * a.pages.k_stride[0] + kh * a.pages.k_stride[1] + r * a.pages.k_stride[2] + lane * N;
    const int64_t vat = page * a.pages.v_stride[0] + kh * a.pages.v_stride[1] + r * a.pages.v_stride[2] + lane * N;
    float s = 0.f, ks = 1.f, vs = 1.f;
    if (a.pages.dtype == KIE_E4M3) {
      ks = a.pages.k_scale[page * a.pages.k_scale_stride[0] + kh * a.pages.k_scale_stride[1] +
                           r * a.pages.k_scale_stride[2]];
      vs = a.pages.v_scale[page * a.pages.v_scale_stride[0] + kh * a.pages.v_scale_stride[1] +
                           r * a.pages.v_scale_stride[2]];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(q[i], cache_load(a.pages.k, kat + i, a.pages.dtype), s);
    s = warp_sum(s) * ks;
    const float mn = fmaxf(m, s), c = m == mn ? 1.f : expf(m - mn), p = s == -INFINITY ? 0.f : expf(s - mn);
    l = fmaf(l, c, p);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = fmaf(o[i], c, p * vs * cache_load(a.pages.v, vat + i, a.pages.dtype));
    m = mn;
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) so[warp][lane * N + i] = o[i];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < PA_WARPS; ++w) M = fmaxf(M, sm[w]);
  for (int w = 0; w < PA_WARPS; ++w) L += sm[w] == -INFINITY ? 0.f : sl[w] * expf(sm[w] - M);
  for (int i = threadIdx.x; i < DH; i += PA_WARPS * 32) {
    float v = 0.f;
    for (int w = 0; w < PA_WARPS; ++w) v += sm[w] == -INFINITY ? 0.f : so[w][i] * expf(sm[w] - M);
    paged_store(a.out, b * a.out_stride[0] + h * a.out_stride[1] + i, a.q_dtype, L == 0.f ? 0.f : v / L);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[(int64_t)b * a.n_heads + h] = L == 0.f ? -INFINITY : M + logf(L);
}

}  // namespace
}  // namespace kie

size_t kie_paged_attention_workspace_bytes(int, int, int, int) { return 256; }

cudaError_t kie_launch_paged_attention(const kie_paged_attention_args &a, cudaStream_t stream) {
  const unsigned grid = (unsigned)a.n_seqs * (unsigned)a.n_heads;
  if (a.pages.head_dim == 64)
    kie::paged_attn_simple<64><<<grid, kie::PA_WARPS * 32, 0, stream>>>(a);
  else
    kie::paged_attn_simple<128><<<grid, kie::PA_WARPS * 32, 0, stream>>>(a);
  return cudaGetLastError();
}
