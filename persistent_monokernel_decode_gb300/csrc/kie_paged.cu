// Paged K/V cache for a batch of sequences: page allocation and release, the append of new rows, and the C entry
// points with their argument checks (kie_paged_attn.cu holds the attention).
#include <limits.h>
#include <stdio.h>

#include <algorithm>
#include <initializer_list>

#include "kie_device.cuh"
#include "kie_paged.cuh"

namespace kie {
namespace {

// ---- pages and slots ---------------------------------------------------------------------------------------

constexpr int PX_THREADS = 512;

// Inclusive sums of v and w over the block's threads; all[0], all[1] get the sums of all. Every thread must call it.
__device__ __forceinline__ void block_scan(long long &v, long long &w, long long (&all)[2]) {
  constexpr int WARPS = PX_THREADS / 32;
  __shared__ long long part[2][WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, v, o), b = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) v += a, w += b;
  }
  __syncthreads();  // the last call's readers are done
  if (lane == 31) part[0][warp] = v, part[1][warp] = w;
  __syncthreads();
  long long a = lane < WARPS ? part[0][lane] : 0, b = lane < WARPS ? part[1][lane] : 0;  // every warp scans the warps' sums
#pragma unroll
  for (int o = 1; o < WARPS; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) a += x, b += y;
  }
  all[0] = __shfl_sync(0xffffffffu, a, WARPS - 1);
  all[1] = __shfl_sync(0xffffffffu, b, WARPS - 1);
  const long long before_v = __shfl_sync(0xffffffffu, a, (warp + 31) & 31);
  const long long before_w = __shfl_sync(0xffffffffu, b, (warp + 31) & 31);
  if (warp > 0) v += before_v, w += before_w;
}

__device__ __forceinline__ int clamp_int(long long v) { return (int)(v > INT_MAX ? INT_MAX : v); }

// Every block scans all requests (two running sums in one pass: rows, and pages needed) and then writes its share: the
// requests r = blockIdx.x (mod grid) and the rows [blockIdx.x * per, + per). No block waits for another. One scan does
// for both sums although a request whose rows do not fit needs no pages: such requests are all behind those that fit.
// Bound by latency (a load, the scan, a search and a load): 1,025 requests with 84,285 rows, 1.05 MB, take 6.3 us, 256
// requests with a token each 3.4 us, of which an empty launch is about 2. Long prompts add to that: one thread takes all
// pages of a request, one after the other (a load and a store that may alias), 35 ns each. A prompt of 8,192 tokens at
// page size 16 takes 21 us, one of 131,072 288 us.
// PER requests to a thread: 1 up to 512 requests (each request's pages are then taken by a thread of its own), else 4.
template <int PER>
__global__ void __launch_bounds__(PX_THREADS) paged_extend_kernel(const kie_paged_extend_args a, int per) {
  begin_after_previous();
  constexpr int CHUNK = PX_THREADS * PER;  // requests of a pass over the block
  __shared__ int s_end[CHUNK], s_first[CHUNK], s_start[CHUNK], s_len[CHUNK], s_have[CHUNK];  // s_have < 0: not admitted
  __shared__ int s_taken;  // pages given
  const int tid = threadIdx.x, bs = a.block_size;
  const int n_free = min(max(*a.n_free, 0), a.free_capacity);
  const long long cap = (long long)a.max_blocks * bs;
  const long long t0 = (long long)blockIdx.x * per, t1 = min(t0 + per, (long long)a.n_rows);
  long long rows = 0, pages = 0;  // of the chunks before
  if (tid == 0) s_taken = 0;
  for (int r0 = 0; r0 < a.n_seqs; r0 += CHUNK) {
    int len[PER], nw[PER], have[PER], need[PER];
    long long v = 0, w = 0, all[2];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int r = r0 + tid * PER + i;
      len[i] = r < a.n_seqs ? a.lens[r] : -1;
      nw[i] = r < a.n_seqs ? a.new_lens[r] : -1;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool sane = len[i] >= 0 && nw[i] >= 0;
      const long long sum = (long long)len[i] + nw[i];
      have[i] = sane && sum <= cap ? (int)(((unsigned)len[i] + bs - 1) / (unsigned)bs) : -1;  // -1: no room in the table
      need[i] = have[i] >= 0 ? (int)((unsigned)(sum + bs - 1) / (unsigned)bs) - have[i] : 0;
      v += sane ? nw[i] : 0;
      w += need[i];
    }
    const long long mine_v = v, mine_w = w;
    block_scan(v, w, all);
    long long end = rows + v - mine_v, after = pages + w - mine_w;
    int taken = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int x = tid * PER + i, r = r0 + x;
      const long long start = end, first = after;
      if (len[i] >= 0 && nw[i] >= 0) end += nw[i];
      after += need[i];
      const bool ok = have[i] >= 0 && end <= a.n_rows && (need[i] == 0 || after <= n_free);
      if (ok && need[i]) taken = (int)after;
      s_end[x] = r < a.n_seqs ? clamp_int(end) : INT_MAX;
      s_start[x] = clamp_int(start);
      s_first[x] = clamp_int(first);
      s_len[x] = len[i];
      s_have[x] = ok ? have[i] : -1;
      if (r < a.n_seqs && r % gridDim.x == blockIdx.x) {
        a.lens_out[r] = ok ? len[i] + nw[i] : len[i];
        a.admitted[r] = ok;
        a.row_start[r] = clamp_int(start);
        if (ok)
          for (int j = 0; j < need[i]; ++j)
            a.block_table[r * a.table_stride + have[i] + j] = a.free_blocks[n_free - 1 - (first + j)];
      }
    }
    if (taken) atomicMax(&s_taken, taken);  // the pages up to the last request admitted
    const long long rows_next = rows + all[0];
    pages += all[1];
    __syncthreads();
    // rows of this chunk's requests that are this block's
    const long long lo = max(t0, rows), hi = min(t1, rows_next);
    for (long long t = lo + tid; t < hi; t += PX_THREADS) {
      int x = 0, n = min(CHUNK, a.n_seqs - r0);  // the first request whose rows end past t
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
      const int pos = ok ? s_len[x] + (int)(t - s_start[x]) : -1;
      long long slot = -1;
      if (ok) {
        const int j = (int)((unsigned)pos / (unsigned)bs);
        const int page = j < s_have[x] ? a.block_table[(r0 + x) * a.table_stride + j]
                                       : a.free_blocks[n_free - 1 - ((long long)s_first[x] + j - s_have[x])];
        slot = (long long)page * bs + pos - j * bs;
        if (slot > INT_MAX) slot = -1;  // no page of a cache: the append would have to find its slot out of range
      }
      a.slots[t] = (int)max(slot, -1ll);
      a.positions[t] = pos;
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
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0) {
    a.row_start[a.n_seqs] = clamp_int(rows);
    *a.n_free_out = n_free - s_taken;
  }
}

// Every block scans the page counts of all finished requests and copies the pages of its share, the requests
// r = blockIdx.x (mod grid), a team of threads to each: 128 up to 512 requests (few, whose pages may be many), else a
// warp. Bound by latency like the above (256 requests 2.4 us, 2,047 requests 3.4 us).
__host__ __device__ constexpr int px_team(int per) { return per == 1 ? 128 : 32; }
template <int PER>
__global__ void __launch_bounds__(PX_THREADS) paged_release_kernel(const kie_paged_release_args a) {
  begin_after_previous();
  constexpr int CHUNK = PX_THREADS * PER, PX_TEAM = px_team(PER);  // requests of a pass over the block
  __shared__ long long s_first[CHUNK];
  __shared__ int s_pages[CHUNK];
  const int tid = threadIdx.x, bs = a.block_size;
  const int n_free = min(max(*a.n_free, 0), a.free_capacity);
  long long pages = 0;
  for (int r0 = 0; r0 < a.n_seqs; r0 += CHUNK) {
    int len[PER], mine[PER];
    bool done[PER];
    long long v = 0, unused = 0, all[2];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int r = r0 + tid * PER + i;
      done[i] = r < a.n_seqs && a.done[r];
      len[i] = r < a.n_seqs ? a.lens[r] : 0;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      mine[i] = done[i] && len[i] > 0 ? min((int)(((unsigned)len[i] + bs - 1) / (unsigned)bs), a.max_blocks) : 0;
      v += mine[i];
    }
    const long long sum = v;
    block_scan(v, unused, all);
    v += pages - sum;
    pages += all[0];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int x = tid * PER + i, r = r0 + x;
      s_first[x] = v;
      s_pages[x] = mine[i];
      v += mine[i];
      if (r < a.n_seqs && r % gridDim.x == blockIdx.x) a.lens_out[r] = done[i] ? 0 : len[i];
    }
    __syncthreads();
    const int n = min(CHUNK, a.n_seqs - r0);
    const int skew = (int)((blockIdx.x + gridDim.x - r0 % gridDim.x) % gridDim.x);
    for (int x = skew + (tid / PX_TEAM) * gridDim.x; x < n; x += gridDim.x * (PX_THREADS / PX_TEAM)) {
      const int *from = a.block_table + (r0 + x) * a.table_stride;
      const long long to = n_free + s_first[x];
      const int count = (int)min((long long)s_pages[x], a.free_capacity - to);
      for (int j0 = tid % PX_TEAM; j0 < count; j0 += 4 * PX_TEAM) {  // four loads in flight
        int id[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) id[i] = j0 + i * PX_TEAM < count ? from[j0 + i * PX_TEAM] : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j0 + i * PX_TEAM < count) a.free_blocks[to + j0 + i * PX_TEAM] = id[i];
      }
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

constexpr int PP_THREADS = 128;
constexpr int PP_HEADS = 2;  // heads of a row that a thread takes: their loads are in flight together, and share the angles

__device__ __forceinline__ bool codes_fast(float scale) { return scale >= 0x1p-90f && scale <= 0x1p90f; }

// E4M3 codes of v / scale, the quotient correctly rounded. With r = RN(1 / scale), q = RN(v r) and the exact remainder
// v - q scale, RN(q + r remainder) is the correctly rounded quotient (Markstein, IBM J. Res. Dev. 34, 1990); the row's
// elements are at most 448 scale, so nothing overflows, and a remainder that underflows belongs to a quotient below
// 2^-50, whose code is 0 either way. Scales near the ends of the range take the division.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float scale, float r, bool fast) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = v[4 * h + e];
      if (fast) {
        const float q0 = __fmul_rn(x, r);
        q[e] = __fmaf_rn(__fmaf_rn(-q0, scale, x), r, q0);
      } else {
        q[e] = __fdiv_rn(x, scale);
      }
    }
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[2], q[3]), __NV_SATFINITE, __NV_E4M3);
    w[h] = lo | hi << 16;
  }
  return make_uint2(w[0], w[1]);
}

// Eight consecutive elements of type X, as loaded.
template <int X>
struct Eight {
  static constexpr int WORDS = X == KIE_F32 ? 8 : 4;
  uint32_t w[WORDS];
  template <bool VEC>
  __device__ __forceinline__ void load(const void *p, int64_t i) {
    if (VEC) {
      const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p) + i * (WORDS / 2));
#pragma unroll
      for (int k = 0; k < WORDS / 4; ++k) {
        const uint4 x = s[k];
        w[4 * k] = x.x, w[4 * k + 1] = x.y, w[4 * k + 2] = x.z, w[4 * k + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < WORDS; ++k)
        w[k] = X == KIE_F32 ? static_cast<const uint32_t *>(p)[i + k]
                            : static_cast<const uint16_t *>(p)[i + 2 * k] |
                                  (uint32_t) static_cast<const uint16_t *>(p)[i + 2 * k + 1] << 16;
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < WORDS; ++k) {
      if (X == KIE_F32) {
        v[k] = __uint_as_float(w[k]);
      } else if (X == KIE_F16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
        v[(2 * k) & 7] = f.x, v[(2 * k + 1) & 7] = f.y;
      } else {
        v[(2 * k) & 7] = __uint_as_float(w[k] << 16), v[(2 * k + 1) & 7] = __uint_as_float(w[k] & 0xffff0000u);
      }
    }
  }
};

// DH / 16 threads to PP_HEADS heads of a row, a warp's teams on the same heads of neighbouring rows (so that a warp does
// not diverge between queries, keys and values): thread t holds elements 8t .. 8t + 7 of each and their partners of the
// other half. The rotation's products and sums are rounded one by one (no fused multiply-add), so that a plain fp32
// evaluation gives the same bits, and with them the same E4M3 codes. Bound by HBM where there are many rows (each
// element is read and written once): 8,192 fp32 rows of 16 + 8 heads, 189 MB, take 31 us, 6.1 TB/s; 16-bit rows take as
// many instructions for half the bytes and reach 5.0 TB/s (bf16 pages), 4.0-4.5 (E4M3, whose maxima and quotients add a
// third); their kernels spill 8 to 12 bytes at the 64 registers that eight blocks leave. Resident blocks that loop with the
// next row's loads in flight were no faster into E4M3 (14.5 us instead of 14.4 for 4,097 rows) and 4 % faster into bf16
// pages (8,192 rows 19.8 us instead of 20.7); one form is kept for both. Two heads to a thread: one reached 3.8 TB/s on the
// bf16 rows, four 5.1 but 74 % of two's rate on fp32 ones. Few rows are a chain of two loads (32 rows 2.0 us, an empty launch included).
template <int DH, int X, bool VEC>
__global__ void __launch_bounds__(PP_THREADS, X == KIE_F32 ? 6 : 8) paged_append_kernel(const kie_paged_append_args a) {
  begin_after_previous();
  constexpr int TPH = DH / 16, HALF = DH / 2;
  const kie_pages &pg = a.pages;
  const unsigned nq = a.q ? a.n_heads : 0u, heads = nq + 2u * pg.n_kv_heads, groups = (heads + PP_HEADS - 1) / PP_HEADS;
  const unsigned warp = (blockIdx.x * PP_THREADS + threadIdx.x) / 32, lane = threadIdx.x & 31;
  const int i0 = (lane % TPH) * 8;
  const int row = warp / groups * (32 / TPH) + lane / TPH;
  const unsigned head0 = warp % groups * PP_HEADS;
  if (row >= a.n_rows) return;  // whole teams of TPH threads leave together
  const int slot = a.slots[row];
  const int pos = a.rope ? a.positions[row] : 0;
  Eight<X> raw[PP_HEADS][2];  // as they are: converted when it is their turn
#pragma unroll
  for (int j = 0; j < PP_HEADS; ++j) {
    const unsigned head = head0 + j;
    if (head >= heads) break;
    const bool is_q = head < nq, is_k = !is_q && head < nq + pg.n_kv_heads;
    const unsigned h = head - (is_q ? 0u : is_k ? nq : nq + pg.n_kv_heads);
    const void *src = is_q ? a.q : is_k ? a.k : a.v;
    const int64_t *ss = is_q ? a.q_stride : is_k ? a.k_stride : a.v_stride;
    const int64_t at = row * ss[0] + h * ss[1];
    // k_pairs: element pairs (i, i + HALF) are adjacent; they are told apart below
    const bool pairs = is_k && a.k_pairs;
    raw[j][0].template load<VEC>(src, at + (pairs ? 2 * i0 : i0));
    raw[j][1].template load<VEC>(src, at + (pairs ? 2 * i0 + 8 : i0 + HALF));
  }
  if (slot < 0 || slot >= pg.n_blocks * pg.block_size || (a.rope && (pos < 0 || pos >= a.n_pos))) return;
  float c[8], s[8];
  if (a.rope && head0 < nq + pg.n_kv_heads) {
    const float4 *cs = reinterpret_cast<const float4 *>(a.rope + ((int64_t)pos * HALF + i0) * 2);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 w = cs[e];  // cos, sin of two pairs
      c[2 * e] = w.x, s[2 * e] = w.y, c[2 * e + 1] = w.z, s[2 * e + 1] = w.w;
    }
  }
  const int64_t page = (unsigned)slot / (unsigned)pg.block_size, off = (unsigned)slot % (unsigned)pg.block_size;
#pragma unroll
  for (int j = 0; j < PP_HEADS; ++j) {
    const unsigned head = head0 + j;
    if (head >= heads) break;
    const bool is_q = head < nq, is_k = !is_q && head < nq + pg.n_kv_heads;
    const unsigned h = head - (is_q ? 0u : is_k ? nq : nq + pg.n_kv_heads);
    float lo[8], hi[8];
    raw[j][0].get(lo);
    raw[j][1].get(hi);
    if (is_k && a.k_pairs) {
      float x[8], y[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = lo[2 * e], y[e] = lo[2 * e + 1];
        x[4 + e] = hi[2 * e], y[4 + e] = hi[2 * e + 1];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) lo[e] = x[e], hi[e] = y[e];
    }
    if (a.rope && (is_q || is_k)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = lo[e], y = hi[e];
        lo[e] = __fsub_rn(__fmul_rn(x, c[e]), __fmul_rn(y, s[e]));
        hi[e] = __fadd_rn(__fmul_rn(y, c[e]), __fmul_rn(x, s[e]));
      }
    }
    if (is_q) {
      const int64_t to = row * a.q_out_stride[0] + h * a.q_out_stride[1] + i0;
      store8<VEC>(a.q_out, to, X, lo);
      store8<VEC>(a.q_out, to + HALF, X, hi);
      continue;
    }
    const int64_t *cst = is_k ? pg.k_stride : pg.v_stride;
    const int64_t to = page * cst[0] + h * cst[1] + off * cst[2] + i0;
    void *dst = is_k ? pg.k : pg.v;
    if (pg.dtype != KIE_E4M3) {
      store8<true>(dst, to, pg.dtype, lo);
      store8<true>(dst, to + HALF, pg.dtype, hi);
      continue;
    }
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max_nan(top, max_nan(fabsf(lo[e]), fabsf(hi[e])));
    const unsigned lanes = ((1u << TPH) - 1u) << ((threadIdx.x & 31) / TPH * TPH);
#pragma unroll
    for (int o = 1; o < TPH; o <<= 1) top = max_nan(top, __shfl_xor_sync(lanes, top, o));
    float scale = __fdiv_rn(top, 448.f);
    if (scale == 0.f) scale = 0x1p-126f;  // a row of zeros, or (fp32) of elements up to 448 * 2^-150: all codes are 0
    const float r = __frcp_rn(scale);
    const bool fast = codes_fast(scale);
    uint8_t *q8 = static_cast<uint8_t *>(dst);
    *reinterpret_cast<uint2 *>(q8 + to) = codes8(lo, scale, r, fast);
    *reinterpret_cast<uint2 *>(q8 + to + HALF) = codes8(hi, scale, r, fast);
    if (i0 == 0) {
      const int64_t *sst = is_k ? pg.k_scale_stride : pg.v_scale_stride;
      (is_k ? pg.k_scale : pg.v_scale)[page * sst[0] + h * sst[1] + off * sst[2]] = scale;
    }
  }
}

template <int DH, int X>
cudaError_t launch_append(const kie_paged_append_args &a, unsigned grid, bool vec, cudaStream_t s) {
  auto *kernel = vec ? paged_append_kernel<DH, X, true> : paged_append_kernel<DH, X, false>;
  return launch_after_previous(kernel, grid, PP_THREADS, 0, s, a);
}

// ---- checks of arguments ------------------------------------------------------------------------------------

thread_local char g_paged_error[256] = "";

int refuse(const char *msg) {
  snprintf(g_paged_error, sizeof(g_paged_error), "%s", msg);
  return KIE_ERR_INVALID;
}

int finish(cudaError_t e, const char *what) {
  if (e == cudaSuccess) return KIE_OK;
  cudaGetLastError();  // reported here: the next caller's check shall not find it again
  snprintf(g_paged_error, sizeof(g_paged_error), "%s: %s", what, cudaGetErrorString(e));
  return KIE_ERR_CUDA;
}

bool aligned(const void *p, size_t n) { return (uintptr_t)p % n == 0; }

bool strides_fit(const int64_t (&st)[3], int64_t most_of_positions) {
  return st[0] >= 0 && st[0] < 1ll << 31 && st[1] >= 0 && st[1] < 1ll << 31 && st[2] >= 0 && st[2] < most_of_positions;
}

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
  for (const auto *st : {&p.k_stride, &p.v_stride})
    if (!strides_fit(*st, 1ll << 26)) return "strides must be from 0 to below 2^31, those of positions below 2^26";
  if (p.dtype == KIE_E4M3 && (!p.k_scale || !p.v_scale)) return "E4M3 pages need k_scale and v_scale";
  if (p.dtype == KIE_E4M3 && (!strides_fit(p.k_scale_stride, 1ll << 31) || !strides_fit(p.v_scale_stride, 1ll << 31)))
    return "the scales' strides must be from 0 to below 2^31";
  if (p.dtype == KIE_E4M3 && (!aligned(p.k_scale, 4) || !aligned(p.v_scale, 4))) return "scales must be 4-byte aligned";
  return nullptr;
}

bool ints_aligned(std::initializer_list<const void *> arrays) {
  for (const void *p : arrays)
    if (!aligned(p, 4)) return false;
  return true;
}

bool activation(int dtype) { return dtype == KIE_F16 || dtype == KIE_BF16 || dtype == KIE_F32; }

bool aligned_rows(const void *p, const int64_t (&stride)[2], int dtype) {
  const int unit = 16 / paged_dtype_bytes(dtype);
  return aligned(p, 16) && stride[0] % unit == 0 && stride[1] % unit == 0;
}

// A dimension that is written but has no stride: its elements are one, and which block's value stays is open.
template <int N>
bool repeats(const int64_t (&stride)[N], const int (&size)[N]) {
  for (int i = 0; i < N; ++i)
    if (stride[i] == 0 && size[i] > 1) return true;
  return false;
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
  if (!ints_aligned({a.lens, a.new_lens, a.free_blocks, a.n_free, a.block_table, a.lens_out, a.n_free_out, a.row_start, a.slots,
                     a.positions, a.seqs}))
    return refuse("an int32 array is not 4-byte aligned");
  if (a.n_free_out == a.n_free || (a.n_seqs > 0 && (a.lens_out == a.lens || a.lens_out == a.new_lens)))
    return refuse("lens_out and n_free_out must not be the inputs");
  int dev, sms;
  if (!sm_count(&dev, &sms)) return finish(cudaErrorInvalidDevice, "device query");
  const int grid = (int)std::min<int64_t>(sms, std::max<int64_t>(1, ((int64_t)a.n_rows + PX_THREADS - 1) / PX_THREADS));
  const int per = (int)(((int64_t)a.n_rows + grid - 1) / grid);
  auto *kernel = a.n_seqs <= PX_THREADS ? paged_extend_kernel<1> : paged_extend_kernel<4>;
  return finish(launch_after_previous(kernel, grid, PX_THREADS, 0, (cudaStream_t)stream, a, per), "paged_extend");
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
  if (!ints_aligned({a.lens, a.n_free, a.block_table, a.free_blocks, a.lens_out, a.n_free_out}))
    return refuse("an int32 array is not 4-byte aligned");
  if (a.n_free_out == a.n_free || (a.n_seqs > 0 && a.lens_out == a.lens))
    return refuse("lens_out and n_free_out must not be the inputs");
  int dev, sms;
  if (!sm_count(&dev, &sms)) return finish(cudaErrorInvalidDevice, "device query");
  const int teams = PX_THREADS / px_team(a.n_seqs <= PX_THREADS ? 1 : 4);
  const int grid = std::min(sms, std::max(1, (a.n_seqs + teams - 1) / teams));
  auto *kernel = a.n_seqs <= PX_THREADS ? paged_release_kernel<1> : paged_release_kernel<4>;
  return finish(launch_after_previous(kernel, grid, PX_THREADS, 0, (cudaStream_t)stream, a), "paged_release");
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
  if (!ints_aligned({a.slots, a.positions})) return refuse("an int32 array is not 4-byte aligned");
  for (const void *x : {a.k, a.v, a.q, (const void *)a.q_out})
    if (!aligned(x, paged_dtype_bytes(a.x_dtype))) return refuse("k, v, q or q_out is not aligned to its elements");
  if (a.q && a.q_out == a.q && (a.q_stride[0] != a.q_out_stride[0] || a.q_stride[1] != a.q_out_stride[1]))
    return refuse("q_out in place of q needs q's strides");
  const int64_t heads = (a.q ? a.n_heads : 0) + 2ll * a.pages.n_kv_heads, groups = (heads + PP_HEADS - 1) / PP_HEADS;
  if (a.n_rows * groups * PP_HEADS > 1ll << 28) return refuse("too many rows x heads (2^28 at most)");
  if (a.q && repeats(a.q_out_stride, {a.n_rows, a.n_heads})) return refuse("q_out has a stride of 0 (an expanded tensor)");
  const kie_pages &pg = a.pages;
  for (const auto *st : {&pg.k_stride, &pg.v_stride, &pg.k_scale_stride, &pg.v_scale_stride})
    if ((pg.dtype == KIE_E4M3 || st == &pg.k_stride || st == &pg.v_stride) &&
        repeats(*st, {pg.n_blocks, pg.n_kv_heads, pg.block_size}))
      return refuse("pages or scales that are written have a stride of 0 (an expanded tensor)");
  const int tph = a.pages.head_dim / 16;
  const int64_t warps = (a.n_rows + 32 / tph - 1) / (32 / tph) * groups;
  const unsigned grid = (unsigned)((warps * 32 + PP_THREADS - 1) / PP_THREADS);
  const bool vec = aligned_rows(a.k, a.k_stride, a.x_dtype) && aligned_rows(a.v, a.v_stride, a.x_dtype) &&
                   (!a.q || (aligned_rows(a.q, a.q_stride, a.x_dtype) && aligned_rows(a.q_out, a.q_out_stride, a.x_dtype)));
  cudaStream_t s = (cudaStream_t)stream;
  const bool wide = a.pages.head_dim == 128;
  cudaError_t e;
  if (a.x_dtype == KIE_F16)
    e = wide ? launch_append<128, KIE_F16>(a, grid, vec, s) : launch_append<64, KIE_F16>(a, grid, vec, s);
  else if (a.x_dtype == KIE_BF16)
    e = wide ? launch_append<128, KIE_BF16>(a, grid, vec, s) : launch_append<64, KIE_BF16>(a, grid, vec, s);
  else
    e = wide ? launch_append<128, KIE_F32>(a, grid, vec, s) : launch_append<64, KIE_F32>(a, grid, vec, s);
  return finish(e, "paged_append");
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
  if (!a.q || !a.out || !a.block_table) return refuse("q, out or block_table is NULL");
  if (!a.seqs != !a.positions) return refuse("seqs and positions go together");
  if (!a.seqs == !a.lens) return refuse("either lens or seqs and positions must be given, the other NULL");
  if (a.seqs && a.n_table < 0) return refuse("n_table must be >= 0");
  if ((a.seqs ? a.n_table : a.n_seqs) > 1 && a.table_stride < a.max_blocks) return refuse("table_stride is below max_blocks");
  if (!ints_aligned({a.block_table, a.lens, a.seqs, a.positions, a.lse}))
    return refuse("block_table, lens, seqs, positions or lse is not 4-byte aligned");
  if (!aligned(a.q, paged_dtype_bytes(a.q_dtype)) || !aligned(a.out, paged_dtype_bytes(a.q_dtype)))
    return refuse("q or out is not aligned to its elements");
  if ((double)a.n_seqs * a.max_blocks * a.pages.block_size * a.pages.n_kv_heads > 0x1p45)
    return refuse("n_seqs * max_blocks * block_size * n_kv_heads must not pass 2^45");
  if (a.out == a.q && ((a.n_seqs > 1 && a.out_stride[0] != a.q_stride[0]) || (a.n_heads > 1 && a.out_stride[1] != a.q_stride[1])))
    return refuse("out in place of q needs q's strides");
  if (repeats(a.out_stride, {a.n_seqs, a.n_heads})) return refuse("out has a stride of 0 (an expanded tensor)");
  int dev, sms;
  if (!sm_count(&dev, &sms)) return finish(cudaErrorInvalidDevice, "device query");
  const size_t need = kie_paged_attention_workspace_bytes(a.n_heads, a.pages.n_kv_heads, a.pages.head_dim, sms);
  if (!a.workspace || a.workspace_bytes < need || !aligned(a.workspace, 256))
    return refuse("the workspace is NULL, unaligned (256 bytes) or smaller than kie_paged_attention_workspace");
  return finish(kie_launch_paged_attention(a, dev, sms, (cudaStream_t)stream), "paged_attention");
}
