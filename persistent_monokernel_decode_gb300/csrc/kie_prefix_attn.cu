// The shared part of kie_paged_prefix_attention: attention of the rows of each group over the positions of their prefix.
// The rows' own positions, and the sum of both, are kie_paged_attn.cu's.
#include "kie_device.cuh"
#include "kie_paged.cuh"

namespace kie {
namespace {

constexpr int PX_WARPS = 8;

__device__ __forceinline__ float element(const void *p, int64_t i, int dtype) {
  if (dtype == KIE_F32) return static_cast<const float *>(p)[i];
  if (dtype == KIE_F16) return __half2float(static_cast<const __half *>(p)[i]);
  if (dtype == KIE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<const uint8_t *>(p)[i], __NV_E4M3)));
}

// A block is a query row, a warp its heads in turn: one position at a time, the dimensions over the lanes.
template <int DH>
__global__ void __launch_bounds__(32 * PX_WARPS) prefix_kernel(const PrefixArgs a) {
  begin_after_previous();
  constexpr int E = DH / 32;
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int g = -1, head = 0, tail = a.n_seqs;
  for (int i = 0, start = 0; i <= a.n_groups; ++i) {
    start = max(start, min(max(a.group_start[i], 0), a.n_seqs));
    if (start <= b)
      g = i, head = start;
    else if (i == g + 1)
      tail = start;
  }
  const auto sequence = [&](int r) { return a.seqs ? a.seqs[r] : r; };
  const auto length = [&](int r) { return (unsigned)sequence(r) < (unsigned)a.n_table ? row_len(a, r) : 0; };
  const int prefix = g >= 0 && g < a.n_groups ? min(max(a.prefix_lens[g], 0), a.max_blocks * a.pages.block_size) : 0;
  int seq = 0, reach = 0;  // of the row whose pages are read
  for (int r = head; r < tail && reach < prefix; ++r) {
    const int l = min(length(r), prefix);
    if (l > reach) reach = l, seq = sequence(r);
  }
  const int n = min(prefix, length(b));
  if (threadIdx.x == 0) a.row_lo[b] = n;
  const int group = a.n_heads / a.pages.n_kv_heads;
  const kie_pages &pg = a.pages;
  for (int h = warp; h < a.n_heads; h += PX_WARPS) {
    float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
    for (int e = 0; e < E; ++e)
      q[e] = element(a.q, b * a.q_stride[0] + h * a.q_stride[1] + lane + 32 * e, a.q_dtype) * a.scale * 1.4426950408889634f;
    for (int pos = 0; pos < n; ++pos) {
      const int page = a.block_table[seq * a.table_stride + pos / pg.block_size], at = pos % pg.block_size;
      if ((unsigned)page >= (unsigned)pg.n_blocks) continue;
      const int64_t ka = page * pg.k_stride[0] + h / group * pg.k_stride[1] + at * pg.k_stride[2];
      const int64_t va = page * pg.v_stride[0] + h / group * pg.v_stride[1] + at * pg.v_stride[2];
      float s = 0.f, vs = 1.f;
      for (int e = 0; e < E; ++e) s += q[e] * element(pg.k, ka + lane + 32 * e, pg.dtype);
      for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      if (pg.dtype == KIE_E4M3) {
        s *= pg.k_scale[page * pg.k_scale_stride[0] + h / group * pg.k_scale_stride[1] + at * pg.k_scale_stride[2]];
        vs = pg.v_scale[page * pg.v_scale_stride[0] + h / group * pg.v_scale_stride[1] + at * pg.v_scale_stride[2]];
      }
      if (s == -INFINITY) continue;
      const float mn = fmaxf(m, s), f = exp2f(m - mn), p = exp2f(s - mn);
      m = mn;
      l = l * f + p;
      for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * vs * element(pg.v, va + lane + 32 * e, pg.dtype);
    }
    const int64_t to = (int64_t)b * a.n_heads + h;
    for (int e = 0; e < E; ++e) a.prefix[to * DH + lane + 32 * e] = o[e];
    if (lane == 0) {
      float *ml = a.prefix + (int64_t)a.n_seqs * a.n_heads * DH + 2 * to;
      ml[0] = m, ml[1] = l;
    }
  }
}

}  // namespace
}  // namespace kie

size_t kie_paged_prefix_workspace_bytes(int n_seqs, int n_heads, int n_kv_heads, int head_dim, int sms) {
  return (kie_paged_attention_workspace_bytes(n_heads, n_kv_heads, head_dim, sms) + 255) / 256 * 256 +
         ((size_t)n_seqs * 4 + 255) / 256 * 256 + (size_t)n_seqs * n_heads * (head_dim + 2) * 4;
}

cudaError_t kie_launch_paged_prefix(const kie_paged_prefix_attention_args &args, int dev, int sms, cudaStream_t stream) {
  kie::PrefixArgs a;
  static_cast<kie_paged_attention_args &>(a) = kie::rows_in_lens(args.a);
  a.group_start = args.group_start;
  a.prefix_lens = args.prefix_lens;
  a.n_groups = args.n_groups;
  uint8_t *at = static_cast<uint8_t *>(a.workspace) +
                (kie_paged_attention_workspace_bytes(a.n_heads, a.pages.n_kv_heads, a.pages.head_dim, sms) + 255) / 256 * 256;
  a.row_lo = reinterpret_cast<int32_t *>(at);
  a.prefix = reinterpret_cast<float *>(at + ((size_t)a.n_seqs * 4 + 255) / 256 * 256);
  auto *kernel = a.pages.head_dim == 64 ? kie::prefix_kernel<64> : kie::prefix_kernel<128>;
  const cudaError_t e = kie::launch_after_previous(kernel, (unsigned)a.n_seqs, 32 * kie::PX_WARPS, 0, stream, a);
  return e != cudaSuccess ? e : kie_launch_paged_suffix(a, dev, sms, stream);
}
