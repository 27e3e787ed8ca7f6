// Attention of one new token per sequence over a paged K/V cache, split over the cache's length and joined.
//
// The work is a list of items (sequence, KV head), each a row of units of 64 positions. Every block of the grid takes
// an equal run of consecutive units, whatever items they belong to, so a ragged batch and a single long sequence load
// the GPU alike; a block keeps the whole items of its run to itself and publishes the pieces of the (at most two)
// items that it shares with its neighbours, which a second kernel joins.
//
// Inside a block each of four warps takes 16 positions of a unit. Both products run as mma.sync m16n8k16 with the
// KV head's query heads (at most 8) as rows 0-7 of A and, where 16 bits do not hold a value exactly, its remainder
// in rows 8-15: S = Q K^T, then O += P V with the weights P as two 16-bit parts, the accumulators' two row halves being
// summed in the same lane. The running maximum, sum and output of a warp's positions stay in registers; a tile's
// scores never leave the lanes that hold them (the accumulator of S is the A operand of P V).
#include <float.h>

#include "kie_device.cuh"
#include "kie_paged.cuh"

namespace kie {
namespace {

constexpr int PA_WARPS = 4;
constexpr int PA_THREADS = PA_WARPS * 32;
constexpr int PA_TILE = 16;                 // positions of a warp's tile: the k of one P V step; pages are multiples
constexpr int PA_UNIT = PA_WARPS * PA_TILE;
constexpr int PA_BLOCKS_PER_SM = 2;
constexpr int PA_ROWS = PAGED_MAX_GROUP;
constexpr int PA_RING_BYTES = 24 * 1024;    // a warp's ring: 4 warps x 2 blocks x 24 KB = 192 KB of an SM
constexpr int PA_MAX_SLOTS = 12;
constexpr float LOG2E = 1.4426950408889634f;
// fp16 weights are kept as 2^14 p: an fp16 pair then holds them to 2^-39 of the largest instead of 2^-25.
constexpr float P_BIAS = 14.f;

enum { PG_F16 = 0, PG_BF16 = 1, PG_E4M3 = 2 };

__host__ __device__ constexpr int pa_half_bytes(int kind, int dh) { return PA_TILE * dh * (kind == PG_E4M3 ? 1 : 2); }
__host__ __device__ constexpr int pa_slots(int kind, int dh) {
  return PA_RING_BYTES / pa_half_bytes(kind, dh) < PA_MAX_SLOTS ? PA_RING_BYTES / pa_half_bytes(kind, dh) : PA_MAX_SLOTS;
}

// A block's shared memory: the warps' rings, the E4M3 scales of each ring entry, the joining of the four warps.
template <int KIND, int DH>
struct PaSmem {
  static constexpr int NS = pa_slots(KIND, DH), HALF = pa_half_bytes(KIND, DH);
  uint8_t ring[PA_WARPS][NS][HALF];
  float scale[PA_WARPS][KIND == PG_E4M3 ? NS : 1][PA_TILE];
  float o[PA_WARPS][PA_ROWS][DH];
  float m[PA_WARPS][PA_ROWS], l[PA_WARPS][PA_ROWS];
  uint32_t live[PA_WARPS][NS / 2];
};

__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async4(void *dst, const void *src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// x = mant * 2^e with 1 <= |mant| < 2 (below 2^-126: e = -126 and |mant| < 1; an infinity or NaN is its own mant).
__device__ __forceinline__ void split_exponent(float x, float *mant, float *e) {
  const uint32_t bits = __float_as_uint(x), field = (bits >> 23) & 255u;
  *mant = field == 0u ? x * 0x1p126f : field == 255u ? x : __uint_as_float((bits & 0x807fffffu) | 0x3f800000u);
  *e = (float)(field == 0u ? -126 : (int)field - 127);
}

template <int KIND>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (KIND == PG_BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int KIND>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  return pack2(a, b, KIND == PG_BF16 ? KIE_BF16 : KIE_F16);
}
// What pack16 left of a and b, packed.
template <int KIND>
__device__ __forceinline__ uint32_t rest16(float a, float b, uint32_t packed) {
  float2 h;
  if (KIND == PG_BF16)
    h = make_float2(__uint_as_float(packed << 16), __uint_as_float(packed & 0xffff0000u));
  else
    h = __half22float2(*reinterpret_cast<const __half2 *>(&packed));
  return pack16<KIND>(a - h.x, b - h.y);
}

// Two E4M3 codes as two fp16 values (exact).
__device__ __forceinline__ uint32_t e4m3x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}

// ---- the list of units --------------------------------------------------------------------------------------

// One sequence's span: positions [lo, len), its tiles from tile0 on, in n units (at least one, so that a sequence of
// no positions still writes its zeros).
struct Span {
  int lo, len, tile0, n;
};
__device__ __forceinline__ Span span_of(const kie_paged_attention_args &a, int b) {
  Span s;
  s.len = (int)min((int64_t)max(a.lens[b], 0), (int64_t)a.max_blocks * a.pages.block_size);
  s.lo = a.window > 0 ? max(0, s.len - a.window) : 0;
  s.tile0 = s.lo / PA_TILE;
  s.n = max(1, (s.len - s.tile0 * PA_TILE + PA_UNIT - 1) / PA_UNIT);
  return s;
}

// A place in the list: unit `unit` of item (b, h).
struct Cursor {
  Span s;
  int b, h, unit;
  __device__ __forceinline__ void next(const kie_paged_attention_args &a) {
    if (++unit < s.n) return;
    unit = 0;
    if (++h < a.pages.n_kv_heads) return;
    h = 0;
    if (++b < a.n_seqs) s = span_of(a, b);
  }
};

// This block's run of units: the cursor at its first unit, and how many there are; total units of the list and units
// per block. Every thread gets the same; two block barriers.
__device__ __forceinline__ int locate(const kie_paged_attention_args &a, Cursor *c, long long *total, long long *per_block) {
  __shared__ long long s_warp[PA_WARPS];
  __shared__ int s_b;
  __shared__ long long s_off;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (a.n_seqs + PA_THREADS - 1) / PA_THREADS;
  const int b0 = min(tid * per, a.n_seqs), b1 = min(b0 + per, a.n_seqs);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += span_of(a, b).n;
  long long up = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += v;
  }
  if (lane == 31) s_warp[warp] = up;
  __syncthreads();
  long long all = 0, before = up - mine;
#pragma unroll
  for (int w = 0; w < PA_WARPS; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  const int heads = a.pages.n_kv_heads;
  all *= heads;
  before *= heads;
  *total = all;
  *per_block = (all + gridDim.x - 1) / gridDim.x;
  const long long u0 = blockIdx.x * *per_block;
  if (u0 >= before && u0 < before + mine * heads) {
    long long at = before;
    int b = b0;
    for (;; ++b) {
      const long long n = (long long)span_of(a, b).n * heads;
      if (u0 < at + n) break;
      at += n;
    }
    s_b = b;
    s_off = u0 - at;
  }
  __syncthreads();
  if (u0 >= all) return 0;
  c->b = s_b;
  c->s = span_of(a, s_b);
  c->h = (int)(s_off / c->s.n);
  c->unit = (int)(s_off % c->s.n);
  return (int)min(*per_block, all - u0);
}

// ---- workspace ----------------------------------------------------------------------------------------------

// Per block: a header {first KV item it starts but does not end (or -1), the block that ends it}, and two pieces, [0]
// of the item that an earlier block started and [1] of the one in the header: o [group][dh], then m and l [group].
// (rounded to 16 bytes)
__host__ __device__ __forceinline__ size_t pa_piece_floats(int group, int dh) { return ((size_t)group * (dh + 2) + 3) / 4 * 4; }
__host__ __device__ __forceinline__ size_t pa_header_bytes(int blocks) { return ((size_t)blocks * 8 + 255) / 256 * 256; }
__device__ __forceinline__ float *pa_piece(const kie_paged_attention_args &a, int blocks, int block, int which) {
  const int group = a.n_heads / a.pages.n_kv_heads;
  return reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + pa_header_bytes(blocks)) +
         ((size_t)block * 2 + which) * pa_piece_floats(group, a.pages.head_dim);
}

// ---- the kernel ---------------------------------------------------------------------------------------------

template <int KIND, int DH, bool SPLIT>
__global__ void __launch_bounds__(PA_THREADS, PA_BLOCKS_PER_SM) paged_attn_kernel(const kie_paged_attention_args a) {
  using Sm = PaSmem<KIND, DH>;
  constexpr int NS = Sm::NS, ES = KIND == PG_E4M3 ? 1 : 2;
  constexpr int CH = DH * ES / 16;        // 16-byte chunks of a row
  constexpr int LOADS = PA_TILE * CH / 32;  // chunks each lane copies of a half
  constexpr int KSTEPS = DH / 16, NT = DH / 8, EC = 16 / ES;  // EC: elements of a chunk
  extern __shared__ __align__(128) uint8_t pa_raw[];
  Sm &sm = *reinterpret_cast<Sm *>(pa_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int group = a.n_heads / a.pages.n_kv_heads;
  const int tiles_per_page = a.pages.block_size / PA_TILE;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Cursor c;
  long long total, per_block;
  const int n_units = locate(a, &c, &total, &per_block);
  if (threadIdx.x == 0) reinterpret_cast<int2 *>(a.workspace)[blockIdx.x] = make_int2(-1, -1);
  if (n_units == 0) return;

  // chunk swizzles: K rows g and g + 1 of a tile are read together (chunks t + 4i), V rows 2t of one chunk pair
  const auto k_chunk = [](int row, int ch) { return CH >= 8 ? ch ^ ((row & 1) << 2) : ch; };
  const auto v_chunk = [](int row, int ch) { return CH >= 8 ? ch ^ (((row >> 1) & 3) << 1) : ch ^ (((row >> 1) & 1) << 1); };

  // ---- producer side: the warp's tile of unit `p`, K half first, then V
  Cursor p = c;
  int p_index = 0;  // unit of the run that p stands at
  int64_t p_page = -1;
  auto fetch_page = [&]() {  // the page id of p's tile, requested one unit before it is used
    const int tile = p.s.tile0 + p.unit * PA_WARPS + warp;
    p_page = -1;
    if (p_index < n_units && tile * PA_TILE < p.s.len) p_page = a.block_table[p.b * a.table_stride + tile / tiles_per_page];
  };
  uint32_t p_live = 0;
  auto issue = [&](int slot, bool is_v) {
    if (!is_v) {
      p_live = 0;
      if (p_page >= 0 && p_page < a.pages.n_blocks) {
        const int pos = (p.s.tile0 + p.unit * PA_WARPS + warp) * PA_TILE;
        const int hi = min(PA_TILE, p.s.len - pos), lo = max(0, p.s.lo - pos);
        p_live = ((1u << hi) - 1u) & ~((1u << lo) - 1u);
      }
      if (lane == 0) sm.live[warp][p_index % (NS / 2)] = p_live;
    }
    if (p_live) {
      const int r0 = (p.s.tile0 + p.unit * PA_WARPS + warp) % tiles_per_page * PA_TILE;
      const int64_t *st = is_v ? a.pages.v_stride : a.pages.k_stride;
      const uint8_t *src = static_cast<const uint8_t *>(is_v ? a.pages.v : a.pages.k) +
                           (p_page * st[0] + p.h * st[1] + r0 * st[2]) * ES;
      uint8_t *dst = sm.ring[warp][slot];
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int row = (lane + 32 * i) / CH, ch = (lane + 32 * i) % CH;
        const int to = is_v ? v_chunk(row, ch) : k_chunk(row, ch);
        cp_async16(dst + (row * CH + to) * 16, src + (int64_t)row * st[2] * ES + ch * 16, (p_live >> row) & 1u);
      }
      if (KIND == PG_E4M3 && lane < PA_TILE) {
        const int64_t *ss = is_v ? a.pages.v_scale_stride : a.pages.k_scale_stride;
        cp_async4(&sm.scale[warp][slot][lane],
                  (is_v ? a.pages.v_scale : a.pages.k_scale) + p_page * ss[0] + p.h * ss[1] + (r0 + lane) * ss[2],
                  (p_live >> lane) & 1u);
      }
    }
    if (is_v) {
      if (++p_index < n_units) p.next(a);
      fetch_page();
    }
  };

  fetch_page();
  for (int x = 0; x < NS - 1; ++x) {
    issue(x, x & 1);
    cp_commit();
  }

  uint32_t qa[KSTEPS][SPLIT ? 4 : 2];
  float row_scale = 0.f;
  float o[NT][4], m = -INFINITY, l = 0.f, mw = -INFINITY;  // mw: the weights' reference (E4M3: of p * v_scale)
  bool first = true;
  int ring = 0;  // slot of the next half
  bool starts = c.unit == 0;  // this block holds the item's first unit

  for (int u = 0; u < n_units; ++u) {
    if (first) {  // a new item: its query heads as A fragments, row g of the group
      first = false;
      const bool vec = ((uintptr_t)a.q | (uintptr_t)(a.q_stride[0] * paged_dtype_bytes(a.q_dtype)) |
                        (uintptr_t)(a.q_stride[1] * paged_dtype_bytes(a.q_dtype))) % 16 == 0;
      const int64_t at = c.b * a.q_stride[0] + (int64_t)(c.h * group + g) * a.q_stride[1];
      float f[DH / 4];
#pragma unroll
      for (int i = 0; i < DH / 32; ++i) {
        // 8 consecutive dimensions a time, in the order of the K chunks that meet them
        const int d = EC == 8 ? 8 * (t + 4 * i) : 16 * (t + 4 * (i >> 1)) + 8 * (i & 1);
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (g < group) {
          if (vec)
            load8<true>(a.q, at + d, a.q_dtype, v);
          else
            load8<false>(a.q, at + d, a.q_dtype, v);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[8 * i + e] = v[e];
      }
      row_scale = a.scale * LOG2E;
      if (SPLIT) {  // bring the row's largest element to [2^13, 2^14) by a power of two
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < DH / 4; ++i) top = fmaxf(top, fabsf(f[i]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int e = 0;
        if (top > 0.f && top <= FLT_MAX) e = max(-120, min(120, 13 - ilogbf(top)));
        const float up = __int_as_float((127 + e) << 23);
        row_scale *= __int_as_float((127 - e) << 23);
#pragma unroll
        for (int i = 0; i < DH / 4; ++i) f[i] *= up;
      }
#pragma unroll
      for (int s = 0; s < KSTEPS; ++s) {
        qa[s][0] = pack16<KIND>(f[4 * s], f[4 * s + 1]);
        qa[s][1] = pack16<KIND>(f[4 * s + 2], f[4 * s + 3]);
        if (SPLIT) {
          qa[s][SPLIT ? 2 : 0] = rest16<KIND>(f[4 * s], f[4 * s + 1], qa[s][0]);
          qa[s][SPLIT ? 3 : 0] = rest16<KIND>(f[4 * s + 2], f[4 * s + 3], qa[s][1]);
        }
      }
      m = mw = -INFINITY;
      l = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    }

    // ---- K half: scores of the tile's 16 positions
    cp_wait<NS - 2>();
    __syncwarp();
    issue((ring + NS - 1) % NS, true);
    cp_commit();
    const uint32_t live = sm.live[warp][u % (NS / 2)];
    uint32_t pa[4];
    if (live) {
      float s[2][4] = {};
      const uint8_t *kt = sm.ring[warp][ring];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = 8 * j + g;
#pragma unroll
        for (int i = 0; i < CH / 4; ++i) {
          const uint4 w = *reinterpret_cast<const uint4 *>(kt + (row * CH + k_chunk(row, t + 4 * i)) * 16);
          const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < EC / 4; ++e) {  // four dimensions of this lane to a step
            const int st = i * (EC / 4) + e;
            const uint32_t b0 = KIND == PG_E4M3 ? e4m3x2(r[e & 3] & 0xffffu) : r[(2 * e) & 3];
            const uint32_t b1 = KIND == PG_E4M3 ? e4m3x2(r[e & 3] >> 16) : r[(2 * e + 1) & 3];
            const uint32_t A[4] = {qa[st][0], SPLIT ? qa[st][SPLIT ? 2 : 0] : 0u, qa[st][1], SPLIT ? qa[st][SPLIT ? 3 : 0] : 0u};
            mma16<KIND>(s[j], A, b0, b1);
          }
        }
      }
      // scores in log2 units, row g, positions 8j + 2t, 8j + 2t + 1
      float v[4], w[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float2 ks = make_float2(1.f, 1.f);
        if (KIND == PG_E4M3) ks = *reinterpret_cast<const float2 *>(&sm.scale[warp][KIND == PG_E4M3 ? ring : 0][8 * j + 2 * t]);
        v[2 * j] = (SPLIT ? s[j][0] + s[j][2] : s[j][0]) * row_scale * ks.x;
        v[2 * j + 1] = (SPLIT ? s[j][1] + s[j][3] : s[j][1]) * row_scale * ks.y;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (!((live >> (8 * j + 2 * t + e)) & 1u)) v[2 * j + e] = -INFINITY;
      }
      float top = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.f : mn;
      float sum = 0.f;
      if (KIND != PG_E4M3) {
        const float bias = KIND == PG_F16 ? P_BIAS : 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] = ex2(v[e] - ref + bias);
          sum += w[e];
        }
        const float corr = m == mn ? 1.f : ex2(m - ref);
        l = fmaf(l, corr, sum);
        if (__any_sync(0xffffffffu, corr != 1.f)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] *= corr;
        }
        m = mn;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += ex2(v[e] - ref);
        l = fmaf(l, m == mn ? 1.f : ex2(m - ref), sum);
        m = mn;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = v[e];
      }
      if (KIND != PG_E4M3) {
        pa[0] = pack16<KIND>(w[0], w[1]);
        pa[2] = pack16<KIND>(w[2], w[3]);
        pa[1] = rest16<KIND>(w[0], w[1], pa[0]);
        pa[3] = rest16<KIND>(w[2], w[3], pa[2]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) pa[e] = __float_as_uint(w[e]);
      }
    }
    ring = ring + 1 == NS ? 0 : ring + 1;

    // ---- V half: the outputs
    cp_wait<NS - 2>();
    __syncwarp();
    issue((ring + NS - 1) % NS, false);
    cp_commit();
    if (live) {
      if (KIND == PG_E4M3) {
        // The weight of a row's codes is p times its scale mant * 2^e: a second running maximum, of log2 p + e, keeps it
        // in fp16's range whatever the size of the scales.
        float v[4], w[4], mant[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 vs = *reinterpret_cast<const float2 *>(&sm.scale[warp][KIND == PG_E4M3 ? ring : 0][8 * j + 2 * t]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float ex;
            split_exponent(e ? vs.y : vs.x, &mant[2 * j + e], &ex);
            v[2 * j + e] = __uint_as_float(pa[2 * j + e]) + ex;  // -inf where masked
          }
        }
        float top = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float mn = fmaxf(mw, top), ref = mn == -INFINITY ? 0.f : mn;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = ex2(v[e] - ref + P_BIAS) * mant[e];
        const float corr = mw == mn ? 1.f : ex2(mw - ref);
        if (__any_sync(0xffffffffu, corr != 1.f)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] *= corr;
        }
        mw = mn;
        pa[0] = pack16<KIND>(w[0], w[1]);
        pa[2] = pack16<KIND>(w[2], w[3]);
        pa[1] = rest16<KIND>(w[0], w[1], pa[0]);
        pa[3] = rest16<KIND>(w[2], w[3], pa[2]);
      }
      const uint8_t *vt = sm.ring[warp][ring];
#pragma unroll
      for (int i = 0; i < DH / 64; ++i) {
        uint32_t b[2][8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // positions 2t + 8k and the next
          const int row = 2 * t + 8 * k;
          if (KIND == PG_E4M3) {
            const int e = g + 8 * i;  // 8 dimensions: half a chunk
            const uint2 x = *reinterpret_cast<const uint2 *>(vt + (row * CH + v_chunk(row, e >> 1)) * 16 + (e & 1) * 8);
            const uint2 y = *reinterpret_cast<const uint2 *>(vt + ((row + 1) * CH + v_chunk(row + 1, e >> 1)) * 16 + (e & 1) * 8);
            const uint32_t X[2] = {x.x, x.y}, Y[2] = {y.x, y.y};
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint32_t lo = __byte_perm(X[q], Y[q], 0x5140), hi = __byte_perm(X[q], Y[q], 0x7362);
              b[k][4 * q] = e4m3x2(lo & 0xffffu), b[k][4 * q + 1] = e4m3x2(lo >> 16);
              b[k][4 * q + 2] = e4m3x2(hi & 0xffffu), b[k][4 * q + 3] = e4m3x2(hi >> 16);
            }
          } else {
            const uint4 x = *reinterpret_cast<const uint4 *>(vt + (row * CH + v_chunk(row, g + 8 * i)) * 16);
            const uint4 y = *reinterpret_cast<const uint4 *>(vt + ((row + 1) * CH + v_chunk(row + 1, g + 8 * i)) * 16);
            const uint32_t X[4] = {x.x, x.y, x.z, x.w}, Y[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              b[k][2 * q] = __byte_perm(X[q], Y[q], 0x5410);
              b[k][2 * q + 1] = __byte_perm(X[q], Y[q], 0x7632);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) mma16<KIND>(o[8 * i + j], pa, b[0][j], b[1][j]);
      }
    }
    ring = ring + 1 == NS ? 0 : ring + 1;

    // ---- the item's end, or the run's: join the four warps
    const bool ends = c.unit + 1 == c.s.n;
    if (ends || u + 1 == n_units) {
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      float back = 1.f;  // brings o to the reference of l
      if (KIND == PG_E4M3) back = mw == -INFINITY ? 0.f : ex2(mw - P_BIAS - (m == -INFINITY ? 0.f : m));
      if (g < group) {
        if (t == 0) {
          sm.m[warp][g] = KIND == PG_F16 ? m - P_BIAS : m;
          sm.l[warp][g] = l;
        }
        // a lane holds 16 consecutive dimensions of row g to every 64
#pragma unroll
        for (int i = 0; i < DH / 64; ++i)
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              float4 x;
              float *xs = &x.x;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int n = 8 * i + 4 * q + e;
                xs[e] = (o[n][half] + o[n][half + 2]) * back;
              }
              *reinterpret_cast<float4 *>(&sm.o[warp][g][16 * (t + 4 * i) + 8 * half + 4 * q]) = x;
            }
      }
      __syncthreads();
      const bool whole = ends && starts;
      float *piece = pa_piece(a, gridDim.x, blockIdx.x, starts ? 1 : 0);
      for (int x = threadIdx.x; x < group * (DH / 4); x += PA_THREADS) {
        const int r = x / (DH / 4), d = x % (DH / 4) * 4;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < PA_WARPS; ++w) M = fmaxf(M, sm.m[w][r]);
        const float ref = M == -INFINITY ? 0.f : M;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < PA_WARPS; ++w) {
          const float f = ex2(sm.m[w][r] - ref);
          const float4 y = *reinterpret_cast<const float4 *>(&sm.o[w][r][d]);
          L = fmaf(sm.l[w][r], f, L);
          acc.x = fmaf(y.x, f, acc.x), acc.y = fmaf(y.y, f, acc.y), acc.z = fmaf(y.z, f, acc.z), acc.w = fmaf(y.w, f, acc.w);
        }
        if (whole) {
          const int64_t head = (int64_t)c.h * group + r;
          paged_finish4(a, c.b, head, d, acc, M, L);
        } else {
          *reinterpret_cast<float4 *>(piece + r * DH + d) = acc;
          if (d == 0) {
            piece[group * DH + r] = M;
            piece[group * (DH + 1) + r] = L;
          }
        }
      }
      if (starts && !ends && threadIdx.x == 0) {
        const long long last = blockIdx.x * per_block + u + (c.s.n - 1 - c.unit);  // the item's last unit
        reinterpret_cast<int2 *>(a.workspace)[blockIdx.x] =
            make_int2(c.b * a.pages.n_kv_heads + c.h, (int)(last / per_block));
      }
      __syncthreads();
      first = true;
      starts = true;
    }
    if (u + 1 < n_units) c.next(a);
  }
  cp_wait<0>();
}

// Joins the pieces of the item that block blockIdx.x of the attention started and did not end, for one query head:
// out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i over pieces in block order.
constexpr int PJ_THREADS = 128;
template <int DH>
__global__ void __launch_bounds__(PJ_THREADS) paged_join_kernel(const kie_paged_attention_args a) {
  constexpr int LANES = DH / 4, SETS = PJ_THREADS / LANES;  // a thread holds four dimensions of every SETS-th piece
  __shared__ float4 s_acc[SETS][LANES];
  __shared__ float s_m[SETS], s_l[SETS];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int blocks = gridDim.x, r = blockIdx.y, group = a.n_heads / a.pages.n_kv_heads;
  const int2 head = reinterpret_cast<const int2 *>(a.workspace)[blockIdx.x];
  if (head.x < 0) return;
  const int set = threadIdx.x / LANES, d = threadIdx.x % LANES * 4;
  const int n = head.y - (int)blockIdx.x + 1;
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = set; i < n; i += SETS) {
    const float *p = pa_piece(a, blocks, blockIdx.x + i, i == 0 ? 1 : 0);
    const float4 y = *reinterpret_cast<const float4 *>(p + r * DH + d);
    const float m = p[group * DH + r], l = p[group * (DH + 1) + r];
    const float mn = fmaxf(M, m), ref = mn == -INFINITY ? 0.f : mn;
    const float f = ex2(m - ref), k = ex2(M - ref);
    L = fmaf(L, k, l * f);
    acc.x = fmaf(acc.x, k, y.x * f), acc.y = fmaf(acc.y, k, y.y * f);
    acc.z = fmaf(acc.z, k, y.z * f), acc.w = fmaf(acc.w, k, y.w * f);
    M = mn;
  }
  s_acc[set][d / 4] = acc;
  if (d == 0) {
    s_m[set] = M;
    s_l[set] = L;
  }
  __syncthreads();
  if (set != 0) return;
  for (int s = 1; s < SETS; ++s) {
    const float m = s_m[s], mn = fmaxf(M, m), ref = mn == -INFINITY ? 0.f : mn;
    const float f = ex2(m - ref), k = ex2(M - ref);
    const float4 y = s_acc[s][d / 4];
    L = fmaf(L, k, s_l[s] * f);
    acc.x = fmaf(acc.x, k, y.x * f), acc.y = fmaf(acc.y, k, y.y * f);
    acc.z = fmaf(acc.z, k, y.z * f), acc.w = fmaf(acc.w, k, y.w * f);
    M = mn;
  }
  paged_finish4(a, head.x / a.pages.n_kv_heads, (int64_t)(head.x % a.pages.n_kv_heads) * group + r, d, acc, M, L);
}

template <int KIND, int DH, bool SPLIT>
cudaError_t launch(const kie_paged_attention_args &a, int blocks, cudaStream_t stream) {
  const int smem = sizeof(PaSmem<KIND, DH>);
  cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<KIND, DH, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  paged_attn_kernel<KIND, DH, SPLIT><<<blocks, PA_THREADS, smem, stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the joining kernel is launched while the attention runs and waits for its end on the device
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, a.n_heads / a.pages.n_kv_heads);
  cfg.blockDim = dim3(PJ_THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<DH>, a);
}

template <int DH>
cudaError_t launch_dh(const kie_paged_attention_args &a, int blocks, cudaStream_t stream) {
  if (a.pages.dtype == KIE_BF16) return launch<PG_BF16, DH, false>(a, blocks, stream);
  if (a.pages.dtype == KIE_E4M3) return launch<PG_E4M3, DH, true>(a, blocks, stream);
  return a.q_dtype == KIE_F32 ? launch<PG_F16, DH, true>(a, blocks, stream) : launch<PG_F16, DH, false>(a, blocks, stream);
}

}  // namespace
}  // namespace kie

size_t kie_paged_attention_workspace_bytes(int n_heads, int n_kv_heads, int head_dim, int sms) {
  const int blocks = sms * kie::PA_BLOCKS_PER_SM;
  return kie::pa_header_bytes(blocks) + (size_t)blocks * 2 * kie::pa_piece_floats(n_heads / n_kv_heads, head_dim) * 4;
}

cudaError_t kie_launch_paged_attention(const kie_paged_attention_args &a, int sms, cudaStream_t stream) {
  const int blocks = sms * kie::PA_BLOCKS_PER_SM;
  return a.pages.head_dim == 64 ? kie::launch_dh<64>(a, blocks, stream) : kie::launch_dh<128>(a, blocks, stream);
}
