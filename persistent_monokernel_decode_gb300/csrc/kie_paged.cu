// Paged K/V cache for a batch of sequences: page allocation and release, the append of new rows, and the C entry
// points with their argument checks (kie_paged_attn.cu holds the attention).
#include <limits.h>
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>

#include "kie_device.cuh"
#include "kie_paged.cuh"

namespace kie {
namespace {

// ---- pages and slots ---------------------------------------------------------------------------------------

constexpr int PX_THREADS = 512;

__device__ __forceinline__ long long warp_scan(long long v) {  // inclusive, over the lanes
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v += u;
  }
  return v;
}

// Inclusive sum over the block's threads; *total gets the sum of all. Every thread must call it.
__device__ __forceinline__ long long block_scan(long long v, long long *total) {
  __shared__ long long part[PX_THREADS / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_scan(v);
  __syncthreads();  // the last call's readers are done
  if (lane == 31) part[warp] = v;
  __syncthreads();
  long long before = 0, all = 0;
  for (int w = 0; w < PX_THREADS / 32; ++w) {
    if (w < warp) before += part[w];
    all += part[w];
  }
  *total = all;
  return v + before;
}

__device__ __forceinline__ int clamp_int(long long v) { return (int)(v > INT_MAX ? INT_MAX : v); }

// Every block scans all requests (two running sums: rows, and pages needed) and then writes its share: the requests
// r = blockIdx.x (mod grid) and the rows [blockIdx.x * per, + per). No block waits for another.
__global__ void __launch_bounds__(PX_THREADS) paged_extend_kernel(const kie_paged_extend_args a, int per) {
  __shared__ long long s_end[PX_THREADS], s_first[PX_THREADS];
  __shared__ int s_start[PX_THREADS], s_len[PX_THREADS], s_have[PX_THREADS];  // s_have < 0: not admitted
  const int tid = threadIdx.x, bs = a.block_size;
  const int n_free = min(max(*a.n_free, 0), a.free_capacity);
  const long long cap = (long long)a.max_blocks * bs;
  const long long t0 = (long long)blockIdx.x * per, t1 = min(t0 + per, (long long)a.n_rows);
  long long rows = 0, pages = 0;  // of the chunks before
  long long taken = 0;            // pages really given
  for (int r0 = 0; r0 < a.n_seqs; r0 += PX_THREADS) {
    const int r = r0 + tid;
    const bool in = r < a.n_seqs;
    const int len = in ? a.lens[r] : 0, nw = in ? a.new_lens[r] : 0;
    const bool sane = in && len >= 0 && nw >= 0;
    long long all;
    const long long end = rows + block_scan(sane ? nw : 0, &all), start = end - (sane ? nw : 0);
    const long long rows_next = rows + all;
    const long long sum = (long long)len + nw;
    const bool fits = sane && sum <= cap && end <= a.n_rows;
    const int have = sane ? (int)((len + (long long)bs - 1) / bs) : 0;
    const int need = fits ? (int)((sum + bs - 1) / bs) - have : 0;
    const long long after = pages + block_scan(need, &all);
    const bool ok = fits && (need == 0 || after <= n_free);
    pages += all;
    const long long first = after - need;
    block_scan(ok ? need : 0, &all);
    taken += all;
    s_end[tid] = in ? end : LLONG_MAX;
    s_start[tid] = clamp_int(start);
    s_first[tid] = first;
    s_len[tid] = len;
    s_have[tid] = ok ? have : -1;
    if (in && r % gridDim.x == blockIdx.x) {
      a.lens_out[r] = ok ? (int)sum : len;
      a.admitted[r] = ok;
      a.row_start[r] = clamp_int(start);
      if (ok)
        for (int j = 0; j < need; ++j)
          a.block_table[r * a.table_stride + have + j] = a.free_blocks[n_free - 1 - (first + j)];
    }
    __syncthreads();
    // rows of this chunk's requests that are this block's
    const long long lo = max(t0, rows), hi = min(t1, rows_next);
    for (long long t = lo + tid; t < hi; t += PX_THREADS) {
      int x = 0, n = min(PX_THREADS, a.n_seqs - r0);  // the first request whose rows end past t
      while (n > 0) {
        const int half = n >> 1;
        if (s_end[x + half] <= t) {
          x += half + 1;
          n -= half + 1;
        } else {
          n = half;
        }
      }
      const bool ok = s_have[x] >= 0;
      const int pos = s_len[x] + (int)(t - s_start[x]);
      int slot = -1;
      if (ok) {
        const int j = pos / bs;
        const int page = j < s_have[x] ? a.block_table[(r0 + x) * a.table_stride + j]
                                       : a.free_blocks[n_free - 1 - (s_first[x] + j - s_have[x])];
        slot = page * bs + pos % bs;
      }
      a.slots[t] = slot;
      a.positions[t] = ok ? pos : -1;
      a.seqs[t] = ok ? r0 + x : -1;
    }
    __syncthreads();
    rows = rows_next;
  }
  for (long long t = max(t0, rows) + tid; t < t1; t += PX_THREADS) {  // rows behind the last
    a.slots[t] = -1;
    a.positions[t] = -1;
    a.seqs[t] = -1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.row_start[a.n_seqs] = clamp_int(rows);
    *a.n_free_out = (int)(n_free - taken);
  }
}

__global__ void __launch_bounds__(PX_THREADS) paged_release_kernel(const kie_paged_release_args a) {
  __shared__ long long s_first[PX_THREADS];
  __shared__ int s_pages[PX_THREADS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, bs = a.block_size;
  const int n_free = min(max(*a.n_free, 0), a.free_capacity);
  long long pages = 0;
  for (int r0 = 0; r0 < a.n_seqs; r0 += PX_THREADS) {
    const int r = r0 + tid;
    const bool in = r < a.n_seqs, done = in && a.done[r];
    const int len = in ? a.lens[r] : 0;
    const int mine = done && len > 0 ? (int)min((len + (long long)bs - 1) / bs, (long long)a.max_blocks) : 0;
    long long all;
    s_first[tid] = pages + block_scan(mine, &all) - mine;
    s_pages[tid] = mine;
    pages += all;
    if (in && r % gridDim.x == blockIdx.x) a.lens_out[r] = done ? 0 : len;
    __syncthreads();
    // a warp to each of this block's requests
    const int n = min(PX_THREADS, a.n_seqs - r0);
    const int skew = (int)((blockIdx.x + gridDim.x - r0 % gridDim.x) % gridDim.x);
    for (int x = skew + warp * gridDim.x; x < n; x += gridDim.x * (PX_THREADS / 32))
      for (int j = lane; j < s_pages[x]; j += 32) {
        const long long to = n_free + s_first[x] + j;
        if (to < a.free_capacity) a.free_blocks[to] = a.block_table[(r0 + x) * a.table_stride + j];
      }
    __syncthreads();
  }
  if (blockIdx.x == 0 && tid == 0) *a.n_free_out = (int)min(n_free + pages, (long long)a.free_capacity);
}

// ---- append -------------------------------------------------------------------------------------------------

// Maximum that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ uint2 codes8(const float (&v)[8], float scale) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    w[e >> 2] |= (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(v[e], scale), __NV_SATFINITE, __NV_E4M3) << (8 * (e & 3));
  return make_uint2(w[0], w[1]);
}

constexpr int PP_THREADS = 256;

// DH / 16 threads to each head of each row: thread t holds elements 8t .. 8t + 7 and their partners of the other
// half. The rotation's products and sums are rounded one by one (no fused multiply-add), so that a plain fp32
// evaluation gives the same bits, and with them the same E4M3 codes.
template <int DH, bool VEC>
__global__ void __launch_bounds__(PP_THREADS) paged_append_kernel(const kie_paged_append_args a) {
  constexpr int TPH = DH / 16, HALF = DH / 2;
  const kie_pages &pg = a.pages;
  const unsigned nq = a.q ? a.n_heads : 0u, heads = nq + 2u * pg.n_kv_heads;
  const unsigned u = (blockIdx.x * PP_THREADS + threadIdx.x) / TPH;
  const int i0 = (threadIdx.x % TPH) * 8;
  if (u >= (unsigned)a.n_rows * heads) return;  // whole groups of TPH threads leave together
  const int row = u / heads;
  unsigned h = u % heads;
  const int slot = a.slots[row];
  const int pos = a.rope ? a.positions[row] : 0;
  if (slot < 0 || slot >= pg.n_blocks * pg.block_size || (a.rope && (pos < 0 || pos >= a.n_pos))) return;
  const int what = h < nq ? 0 : h < nq + pg.n_kv_heads ? 1 : 2;  // q, k, v
  h -= what == 0 ? 0u : what == 1 ? nq : nq + pg.n_kv_heads;
  float lo[8], hi[8];
  const void *src = what == 0 ? a.q : what == 1 ? a.k : a.v;
  const int64_t *ss = what == 0 ? a.q_stride : what == 1 ? a.k_stride : a.v_stride;
  const int64_t at = row * ss[0] + h * ss[1];
  if (what == 1 && a.k_pairs) {
    float x[8], y[8];
    load8<VEC>(src, at + 2 * i0, a.x_dtype, x);
    load8<VEC>(src, at + 2 * i0 + 8, a.x_dtype, y);
#pragma unroll
    for (int e = 0; e < 4; ++e) lo[e] = x[2 * e], hi[e] = x[2 * e + 1], lo[4 + e] = y[2 * e], hi[4 + e] = y[2 * e + 1];
  } else {
    load8<VEC>(src, at + i0, a.x_dtype, lo);
    load8<VEC>(src, at + i0 + HALF, a.x_dtype, hi);
  }
  if (what < 2 && a.rope) {
    const float4 *cs = reinterpret_cast<const float4 *>(a.rope + ((int64_t)pos * HALF + i0) * 2);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 w = cs[e];  // cos, sin of two pairs
      const float c[2] = {w.x, w.z}, s[2] = {w.y, w.w};
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const float x = lo[2 * e + f], y = hi[2 * e + f];
        lo[2 * e + f] = __fsub_rn(__fmul_rn(x, c[f]), __fmul_rn(y, s[f]));
        hi[2 * e + f] = __fadd_rn(__fmul_rn(y, c[f]), __fmul_rn(x, s[f]));
      }
    }
  }
  if (what == 0) {
    const int64_t to = row * a.q_out_stride[0] + h * a.q_out_stride[1] + i0;
    store8<VEC>(a.q_out, to, a.x_dtype, lo);
    store8<VEC>(a.q_out, to + HALF, a.x_dtype, hi);
    return;
  }
  const int64_t page = slot / pg.block_size, off = slot % pg.block_size;
  const int64_t *cst = what == 1 ? pg.k_stride : pg.v_stride;
  const int64_t to = page * cst[0] + h * cst[1] + off * cst[2] + i0;
  void *dst = what == 1 ? pg.k : pg.v;
  if (pg.dtype != KIE_E4M3) {
    store8<true>(dst, to, pg.dtype, lo);
    store8<true>(dst, to + HALF, pg.dtype, hi);
    return;
  }
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max_nan(top, max_nan(fabsf(lo[e]), fabsf(hi[e])));
  const unsigned group = ((1u << TPH) - 1u) << ((threadIdx.x & 31) / TPH * TPH);
#pragma unroll
  for (int o = 1; o < TPH; o <<= 1) top = max_nan(top, __shfl_xor_sync(group, top, o));
  const float scale = top == 0.f ? 0x1p-126f : __fdiv_rn(top, 448.f);
  uint8_t *q8 = static_cast<uint8_t *>(dst);
  *reinterpret_cast<uint2 *>(q8 + to) = codes8(lo, scale);
  *reinterpret_cast<uint2 *>(q8 + to + HALF) = codes8(hi, scale);
  if (i0 == 0) {
    const int64_t *sst = what == 1 ? pg.k_scale_stride : pg.v_scale_stride;
    (what == 1 ? pg.k_scale : pg.v_scale)[page * sst[0] + h * sst[1] + off * sst[2]] = scale;
  }
}

// ---- checks of arguments ------------------------------------------------------------------------------------

thread_local char g_paged_error[256] = "";

int refuse(const char *msg) {
  snprintf(g_paged_error, sizeof(g_paged_error), "%s", msg);
  return KIE_ERR_INVALID;
}

int finish(cudaError_t e, const char *what) {
  if (e == cudaSuccess) return KIE_OK;
  snprintf(g_paged_error, sizeof(g_paged_error), "%s: %s", what, cudaGetErrorString(e));
  return KIE_ERR_CUDA;
}

bool aligned(const void *p, size_t n) { return (uintptr_t)p % n == 0; }

const char *check_pages(const kie_pages &p) {
  if (p.n_blocks < 1 || p.n_kv_heads < 1) return "the pages need n_blocks >= 1 and n_kv_heads >= 1";
  if (p.head_dim != 64 && p.head_dim != 128) return "head_dim must be 64 or 128";
  if (p.block_size < PAGED_ROWS || p.block_size % PAGED_ROWS) return "block_size must be a positive multiple of 16";
  if ((int64_t)p.n_blocks * p.block_size > INT_MAX) return "n_blocks * block_size must be below 2^31";
  if (p.dtype != KIE_F16 && p.dtype != KIE_BF16 && p.dtype != KIE_E4M3) return "pages are KIE_F16, KIE_BF16 or KIE_E4M3";
  if (!p.k || !p.v) return "k or v of the pages is NULL";
  if (!aligned(p.k, 16) || !aligned(p.v, 16)) return "the pages must be 16-byte aligned";
  const int unit = 16 / paged_dtype_bytes(p.dtype);
  for (int i = 0; i < 3; ++i)
    if (p.k_stride[i] % unit || p.v_stride[i] % unit) return "the pages' strides must be multiples of 16 bytes";
  if (llabs(p.k_stride[2]) >= 1 << 26 || llabs(p.v_stride[2]) >= 1 << 26) return "the strides of positions must be below 2^26";
  if (p.dtype == KIE_E4M3 && (!p.k_scale || !p.v_scale)) return "E4M3 pages need k_scale and v_scale";
  if (p.dtype == KIE_E4M3 && (!aligned(p.k_scale, 4) || !aligned(p.v_scale, 4))) return "scales must be 4-byte aligned";
  return nullptr;
}

bool activation(int dtype) { return dtype == KIE_F16 || dtype == KIE_BF16 || dtype == KIE_F32; }

bool aligned_rows(const void *p, const int64_t (&stride)[2], int dtype) {
  const int unit = 16 / paged_dtype_bytes(dtype);
  return aligned(p, 16) && stride[0] % unit == 0 && stride[1] % unit == 0;
}

bool sm_count(int *dev, int *sms) {
  return cudaGetDevice(dev) == cudaSuccess &&
         cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev) == cudaSuccess;
}

}  // namespace
}  // namespace kie

using namespace kie;

const char *kie_paged_last_error(void) { return g_paged_error; }

int kie_paged_extend(const kie_paged_extend_args *p, void *stream) {
  if (!p) return refuse("the arguments are NULL");
  const kie_paged_extend_args &a = *p;
  if (a.n_seqs < 0 || a.n_rows < 0 || a.max_blocks < 1 || a.free_capacity < 0)
    return refuse("n_seqs, n_rows and free_capacity must be >= 0 and max_blocks >= 1");
  if (a.block_size < PAGED_ROWS || a.block_size % PAGED_ROWS) return refuse("block_size must be a positive multiple of 16");
  if ((int64_t)a.max_blocks * a.block_size > INT_MAX) return refuse("max_blocks * block_size must be below 2^31");
  if (!a.n_free || !a.n_free_out || !a.row_start) return refuse("n_free, n_free_out or row_start is NULL");
  if (a.n_seqs > 0 && (!a.lens || !a.new_lens || !a.block_table || !a.lens_out || !a.admitted))
    return refuse("an array of the requests is NULL");
  if (a.n_rows > 0 && (!a.slots || !a.positions || !a.seqs)) return refuse("an array of the rows is NULL");
  if (a.free_capacity > 0 && !a.free_blocks) return refuse("free_blocks is NULL");
  if (a.n_seqs > 1 && a.table_stride < a.max_blocks) return refuse("table_stride is below max_blocks");
  if (a.n_free_out == a.n_free || (a.n_seqs > 0 && (a.lens_out == a.lens || a.lens_out == a.new_lens)))
    return refuse("lens_out and n_free_out must not be the inputs");
  int dev, sms;
  if (!sm_count(&dev, &sms)) return finish(cudaErrorInvalidDevice, "device query");
  const int grid = (int)std::min<int64_t>(sms, std::max<int64_t>(1, ((int64_t)a.n_rows + PX_THREADS - 1) / PX_THREADS));
  const int per = (int)(((int64_t)a.n_rows + grid - 1) / grid);
  paged_extend_kernel<<<grid, PX_THREADS, 0, (cudaStream_t)stream>>>(a, per);
  return finish(cudaGetLastError(), "paged_extend");
}

int kie_paged_release(const kie_paged_release_args *p, void *stream) {
  if (!p) return refuse("the arguments are NULL");
  const kie_paged_release_args &a = *p;
  if (a.n_seqs < 0 || a.max_blocks < 1 || a.free_capacity < 0)
    return refuse("n_seqs and free_capacity must be >= 0 and max_blocks >= 1");
  if (a.block_size < PAGED_ROWS || a.block_size % PAGED_ROWS) return refuse("block_size must be a positive multiple of 16");
  if ((int64_t)a.max_blocks * a.block_size > INT_MAX) return refuse("max_blocks * block_size must be below 2^31");
  if (!a.n_free || !a.n_free_out) return refuse("n_free or n_free_out is NULL");
  if (a.n_seqs > 0 && (!a.lens || !a.done || !a.block_table || !a.lens_out)) return refuse("an array of the requests is NULL");
  if (a.free_capacity > 0 && !a.free_blocks) return refuse("free_blocks is NULL");
  if (a.n_seqs > 1 && a.table_stride < a.max_blocks) return refuse("table_stride is below max_blocks");
  if (a.n_free_out == a.n_free || (a.n_seqs > 0 && a.lens_out == a.lens))
    return refuse("lens_out and n_free_out must not be the inputs");
  int dev, sms;
  if (!sm_count(&dev, &sms)) return finish(cudaErrorInvalidDevice, "device query");
  const int grid = std::min(sms, std::max(1, (a.n_seqs + PX_THREADS / 32 - 1) / (PX_THREADS / 32)));
  paged_release_kernel<<<grid, PX_THREADS, 0, (cudaStream_t)stream>>>(a);
  return finish(cudaGetLastError(), "paged_release");
}

int kie_paged_append(const kie_paged_append_args *p, void *stream) {
  if (!p) return refuse("the arguments are NULL");
  const kie_paged_append_args &a = *p;
  if (const char *e = check_pages(a.pages)) return refuse(e);
  if (a.n_rows < 0) return refuse("n_rows must be >= 0");
  if (!activation(a.x_dtype)) return refuse("k, v and q are KIE_F16, KIE_BF16 or KIE_F32");
  if (a.q && (!a.q_out || a.n_heads < 1)) return refuse("q needs q_out and n_heads >= 1");
  if (a.n_rows == 0) return KIE_OK;
  if (!a.k || !a.v || !a.slots) return refuse("k, v or slots is NULL");
  if (a.rope && (!a.positions || a.n_pos < 1)) return refuse("a rope table needs positions and n_pos >= 1");
  if (a.rope && !aligned(a.rope, 16)) return refuse("the rope table must be 16-byte aligned");
  if (a.q && a.q_out == a.q && (a.q_stride[0] != a.q_out_stride[0] || a.q_stride[1] != a.q_out_stride[1]))
    return refuse("q_out in place of q needs q's strides");
  const int64_t units = (int64_t)a.n_rows * ((a.q ? a.n_heads : 0) + 2ll * a.pages.n_kv_heads);
  if (units > INT_MAX / 8) return refuse("too many rows x heads (2^28 at most)");
  const int tph = a.pages.head_dim / 16;
  const unsigned grid = (unsigned)((units * tph + PP_THREADS - 1) / PP_THREADS);
  const bool vec = aligned_rows(a.k, a.k_stride, a.x_dtype) && aligned_rows(a.v, a.v_stride, a.x_dtype) &&
                   (!a.q || (aligned_rows(a.q, a.q_stride, a.x_dtype) && aligned_rows(a.q_out, a.q_out_stride, a.x_dtype)));
  cudaStream_t s = (cudaStream_t)stream;
  if (a.pages.head_dim == 64) {
    if (vec)
      paged_append_kernel<64, true><<<grid, PP_THREADS, 0, s>>>(a);
    else
      paged_append_kernel<64, false><<<grid, PP_THREADS, 0, s>>>(a);
  } else {
    if (vec)
      paged_append_kernel<128, true><<<grid, PP_THREADS, 0, s>>>(a);
    else
      paged_append_kernel<128, false><<<grid, PP_THREADS, 0, s>>>(a);
  }
  return finish(cudaGetLastError(), "paged_append");
}

size_t kie_paged_attention_workspace(int n_heads, int n_kv_heads, int head_dim) {
  int dev, sms;
  if (n_kv_heads < 1 || n_heads < 1 || n_heads % n_kv_heads || n_heads / n_kv_heads > PAGED_MAX_GROUP ||
      (head_dim != 64 && head_dim != 128) || !sm_count(&dev, &sms))
    return 0;
  return kie_paged_attention_workspace_bytes(n_heads, n_kv_heads, head_dim, sms);
}

int kie_paged_attention(const kie_paged_attention_args *p, void *stream) {
  if (!p) return refuse("the arguments are NULL");
  const kie_paged_attention_args &a = *p;
  if (const char *e = check_pages(a.pages)) return refuse(e);
  if (a.n_seqs < 0 || a.max_blocks < 1 || a.window < 0) return refuse("n_seqs and window must be >= 0 and max_blocks >= 1");
  if ((int64_t)a.max_blocks * a.pages.block_size > 1 << 30) return refuse("max_blocks * block_size must not pass 2^30");
  if (a.n_heads < 1 || a.n_heads % a.pages.n_kv_heads) return refuse("n_heads must be a multiple of n_kv_heads");
  if (a.n_heads / a.pages.n_kv_heads > PAGED_MAX_GROUP) return refuse("more than 8 query heads per KV head");
  if ((int64_t)a.n_seqs * a.n_heads > INT_MAX) return refuse("n_seqs * n_heads must be below 2^31");
  if (!activation(a.q_dtype)) return refuse("q is KIE_F16, KIE_BF16 or KIE_F32");
  if (a.pages.dtype == KIE_BF16 && a.q_dtype != KIE_BF16) return refuse("BF16 pages take BF16 queries");
  if (a.pages.dtype == KIE_F16 && a.q_dtype == KIE_BF16) return refuse("F16 pages take F16 or F32 queries");
  if (!(a.scale == a.scale) || a.scale - a.scale != 0.f) return refuse("scale must be finite");
  if (a.n_seqs == 0) return KIE_OK;
  if (!a.q || !a.out || !a.block_table || !a.lens) return refuse("q, out, block_table or lens is NULL");
  if (a.n_seqs > 1 && a.table_stride < a.max_blocks) return refuse("table_stride is below max_blocks");
  int dev, sms;
  if (!sm_count(&dev, &sms)) return finish(cudaErrorInvalidDevice, "device query");
  const size_t need = kie_paged_attention_workspace_bytes(a.n_heads, a.pages.n_kv_heads, a.pages.head_dim, sms);
  if (!a.workspace || a.workspace_bytes < need || !aligned(a.workspace, 256))
    return refuse("the workspace is NULL, unaligned (256 bytes) or smaller than kie_paged_attention_workspace");
  return finish(kie_launch_paged_attention(a, dev, sms, (cudaStream_t)stream), "paged_attention");
}
