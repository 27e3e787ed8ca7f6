// Attention of one new token per sequence over a paged K/V cache, split over the cache's length and joined.
//
// The work is a list of items (sequence, KV head), each a row of units of 64 positions. Every block of the grid takes
// an equal run of consecutive units, whatever items they belong to, so a ragged batch and a single long sequence load
// the GPU alike; a block keeps the whole items of its run to itself and publishes the pieces of the (at most two)
// items that it shares with its neighbours, which a second kernel joins.
//
// Inside a block each of four warps takes a quarter of a unit, one tile. Both products run as mma.sync m16n8k16 in the
// transposed form, so that no row of an instruction is wasted on the at most 8 query heads of a KV head: S^T = K Q^T
// (16 positions x 8 heads) and O^T += V^T P^T (16 dimensions x 8 heads). K is the A operand as it lies in shared memory
// (ldmatrix), V through ldmatrix.trans; the weights P pass from accumulator to B operand with movmatrix. Where 16 bits
// do not hold a B value exactly (fp32 queries; the weights), its remainder goes through a second mma. The running sum
// and output of a warp's positions stay in registers.
//
// The reference of the softmax is not the running maximum but a value that stays within 2^8 of it: weights up to 2^15
// fit in fp16, so it is only moved (with the shuffles and the rescaling that this costs) when a weight passes that.
#include <float.h>

#include "kie_device.cuh"
#include "kie_paged.cuh"

namespace kie {
namespace {

constexpr int PA_WARPS = 4;
constexpr int PA_THREADS = PA_WARPS * 32;
constexpr int PA_BLOCKS_PER_SM = 3;
constexpr int PA_ROWS = PAGED_MAX_GROUP;
constexpr int PA_RING_BYTES = 16 * 1024;    // a warp's ring: 4 warps x 3 blocks x 16 KB = 192 KB of an SM
constexpr float LOG2E = 1.4426950408889634f;
// Weights are kept as 2^7 2^(v - ref): an fp16 pair holds them to 2^-25, which is 2^-32 of the largest.
constexpr float P_BIAS = 7.f, P_LIMIT = 32768.f;
// Scales of E4M3 value rows count into the reference down to this (log2), so that the plain weights stay finite.
constexpr float MIN_LOG2_SCALE = -60.f;

enum { PG_F16 = 0, PG_BF16 = 1, PG_E4M3 = 2 };

// A warp's tile: 16 positions (32 of E4M3), as one half of K rows and one of V rows of 32 * DH bytes each.
template <int KIND, int DH>
struct PaTile {
  static constexpr int ES = KIND == PG_E4M3 ? 1 : 2, SUBS = KIND == PG_E4M3 ? 2 : 1;  // 16-position parts
  static constexpr int POS = 16 * SUBS, UNIT = POS * PA_WARPS;
  static constexpr int ROW = DH * ES, CH = ROW / 16, HALF = POS * ROW;  // bytes; 16-byte chunks of a row
  static constexpr int NS = PA_RING_BYTES / HALF;                       // ring slots, a half each
  static constexpr int LOADS = HALF / 512;                              // chunks each lane copies
};

// A block's shared memory: the warps' rings (the slot last used also joins the four warps), the E4M3 scales of each
// slot, which positions of it are live, and the warps' references and sums.
template <int KIND, int DH>
struct PaSmem {
  using T = PaTile<KIND, DH>;
  uint8_t ring[PA_WARPS][T::NS][T::HALF];
  float scale[PA_WARPS][KIND == PG_E4M3 ? T::NS : 1][32];
  float m[PA_WARPS][PA_ROWS], l[PA_WARPS][PA_ROWS];
  uint32_t live[PA_WARPS][T::NS];
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The same where live, else 16 zero bytes (nothing is read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(void *dst, const void *src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
// The transpose of an 8 x 8 matrix of 16-bit elements held as two neighbours per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
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

// One sequence's span: positions [lo, len), in n units of UNIT positions from `from` on, a multiple of 16 (at least one
// unit, so that a sequence of no positions still writes its zeros).
struct Span {
  int lo, len, from, n;
};
template <int UNIT>
__device__ __forceinline__ Span span_of(const kie_paged_attention_args &a, int b) {
  Span s;
  s.len = min(max(a.lens[b], 0), a.max_blocks * a.pages.block_size);
  s.lo = a.window > 0 ? max(0, s.len - a.window) : 0;
  s.from = s.lo & ~15;
  s.n = max(1, (int)((unsigned)(s.len - s.from + UNIT - 1) / UNIT));
  return s;
}

// A place in the list: unit `unit` of item (b, h).
template <int UNIT>
struct Cursor {
  Span s;
  int b, h, unit;
  __device__ __forceinline__ void next(const kie_paged_attention_args &a) {
    if (++unit < s.n) return;
    unit = 0;
    if (++h < a.pages.n_kv_heads) return;
    h = 0;
    if (++b < a.n_seqs) s = span_of<UNIT>(a, b);
  }
};

// This block's run of units: the cursor at its first unit, and how many there are; total units of the list and units
// per block. Every thread gets the same; two block barriers.
template <int UNIT>
__device__ __forceinline__ int locate(const kie_paged_attention_args &a, Cursor<UNIT> *c, long long *total, long long *per_block) {
  __shared__ long long s_warp[PA_WARPS];
  __shared__ int s_b;
  __shared__ long long s_off;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (a.n_seqs + PA_THREADS - 1) / PA_THREADS;
  const int b0 = min(tid * per, a.n_seqs), b1 = min(b0 + per, a.n_seqs);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += span_of<UNIT>(a, b).n;
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
      const long long n = (long long)span_of<UNIT>(a, b).n * heads;
      if (u0 < at + n) break;
      at += n;
    }
    s_b = b;
    s_off = u0 - at;
  }
  __syncthreads();
  if (u0 >= all) return 0;
  c->b = s_b;
  c->s = span_of<UNIT>(a, s_b);
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

// Two consecutive elements at p + i as fp32; pair: p + i is aligned for one access.
__device__ __forceinline__ float2 load_pair(const void *p, int64_t i, int dtype, bool pair) {
  if (!pair) return make_float2(paged_load(p, i, dtype), paged_load(p, i + 1, dtype));
  if (dtype == KIE_F32) return *reinterpret_cast<const float2 *>(static_cast<const float *>(p) + i);
  const uint32_t w = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p) + i);
  if (dtype == KIE_F16) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Where column d of a warp's output row r lies in the joining area: the accumulators' four column pairs of a lane
// quad go to different banks.
template <int KIND>
__device__ __forceinline__ int join_col(int r, int d) {
  return d ^ (((r >> 1) & 3) << (KIND == PG_E4M3 ? 4 : 3));
}

template <int KIND, int DH, bool SPLIT>
__global__ void __launch_bounds__(PA_THREADS, PA_BLOCKS_PER_SM) paged_attn_kernel(const kie_paged_attention_args a) {
  using T = PaTile<KIND, DH>;
  using Sm = PaSmem<KIND, DH>;
  constexpr int NS = T::NS, CH = T::CH, ROW = T::ROW, ES = T::ES, SUBS = T::SUBS, LOADS = T::LOADS;
  constexpr int KSTEPS = DH / 16, MT = DH / 16;
  constexpr uint32_t FULL = SUBS == 2 ? 0xffffffffu : 0xffffu;
  static_assert(T::HALF >= PA_ROWS * DH * 4, "the joining area is one slot");
  extern __shared__ __align__(1024) uint8_t pa_raw[];
  Sm &sm = *reinterpret_cast<Sm *>(pa_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int group = a.n_heads / a.pages.n_kv_heads;
  const unsigned bs = a.pages.block_size;
  const int bs_shift = (bs & (bs - 1)) ? -1 : __ffs(bs) - 1;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Cursor<T::UNIT> c;
  long long total, per_block;
  const int n_units = locate(a, &c, &total, &per_block);
  if (threadIdx.x == 0) reinterpret_cast<int2 *>(a.workspace)[blockIdx.x] = make_int2(-1, -1);
  if (n_units == 0) return;

  // Chunk ch of row r of a half lies at chunk ch ^ swz(r): the eight rows of an 8 x 8 matrix fall in different banks.
  const auto swz = [](int row) { return CH >= 8 ? row & 7 : (row >> 1) & 3; };

  // ---- producer side: the warp's tile of unit `p`, K half first, then V. A lane copies chunks lane + 32 i.
  Cursor<T::UNIT> p = c;
  int p_index = 0;  // unit of the run that p stands at
  uint32_t p_live = 0;
  int p_page[SUBS];
  const int row0 = lane / CH;  // row of the lane's first chunk; the next are 32 / CH rows on
  const uint32_t dst_lane = (lane * 16) ^ (swz(row0) << 4);
  const int64_t k_lane = (row0 * a.pages.k_stride[2]) * ES + (lane % CH) * 16, k_step = a.pages.k_stride[2] * ES * (32 / CH);
  const int64_t v_lane = (row0 * a.pages.v_stride[2]) * ES + (lane % CH) * 16, v_step = a.pages.v_stride[2] * ES * (32 / CH);
  const uint32_t ring0 = smem_u32(sm.ring[warp]);
  auto first_pos = [&](const Cursor<T::UNIT> &x) { return x.s.from + (x.unit * PA_WARPS + warp) * T::POS; };
  auto fetch_page = [&]() {  // the page ids of p's tile, requested one unit before they are used
    const int pos = first_pos(p);
#pragma unroll
    for (int i = 0; i < SUBS; ++i) {
      p_page[i] = -1;
      if (p_index < n_units && pos + 16 * i < p.s.len) {
        const unsigned at = pos + 16 * i;
        p_page[i] = a.block_table[p.b * a.table_stride + (bs_shift >= 0 ? at >> bs_shift : at / bs)];
      }
    }
  };
  auto issue = [&](int slot, bool is_v) {
    const int pos = first_pos(p);
    if (!is_v) {
      const int hi = p.s.len - pos, lo = p.s.lo - pos;
      p_live = hi >= T::POS ? FULL : hi > 0 ? (1u << hi) - 1u : 0u;
      if (lo > 0) p_live &= lo >= 32 ? 0u : ~((1u << lo) - 1u);
#pragma unroll
      for (int i = 0; i < SUBS; ++i)
        if ((unsigned)p_page[i] >= (unsigned)a.pages.n_blocks) p_live &= ~(0xffffu << (16 * i));
      if (lane == 0) sm.live[warp][slot] = p_live;
    }
    if (p_live) {
      const int64_t *st = is_v ? a.pages.v_stride : a.pages.k_stride;
      const int64_t step = is_v ? v_step : k_step;
      const uint32_t dst = ring0 + slot * T::HALF + dst_lane;
#pragma unroll
      for (int s = 0; s < SUBS; ++s) {
        const unsigned at = pos + 16 * s, off = bs_shift >= 0 ? at & (bs - 1) : at % bs;
        const uint32_t live = (p_live >> (16 * s)) & 0xffffu;
        const int64_t page = live ? p_page[s] : 0;  // an address inside the pages even where nothing is read
        const uint8_t *src = static_cast<const uint8_t *>(is_v ? a.pages.v : a.pages.k) +
                             (page * st[0] + p.h * st[1] + off * st[2]) * ES + (is_v ? v_lane : k_lane);
        constexpr int N = LOADS / SUBS;
        if (live == 0xffffu) {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            cp_async16((dst ^ (swz((i + s * N) * (32 / CH)) << 4)) + (i + s * N) * 512, src);
            src += step;
          }
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            cp_async16((dst ^ (swz((i + s * N) * (32 / CH)) << 4)) + (i + s * N) * 512, src,
                       (p_live >> (row0 + (i + s * N) * (32 / CH))) & 1u);
            src += step;
          }
        }
      }
      if (KIND == PG_E4M3) {  // a row's scale to each lane
        const int64_t *ss = is_v ? a.pages.v_scale_stride : a.pages.k_scale_stride;
        const unsigned at = pos + lane, off = bs_shift >= 0 ? at & (bs - 1) : at % bs;
        const bool live = (p_live >> lane) & 1u;
        const int64_t page = live ? (lane < 16 ? p_page[0] : p_page[SUBS - 1]) : 0;
        cp_async4(&sm.scale[warp][KIND == PG_E4M3 ? slot : 0][lane],
                  (is_v ? a.pages.v_scale : a.pages.k_scale) + page * ss[0] + p.h * ss[1] + off * ss[2],
                  live);
      }
    }
    if (is_v) {
      if (++p_index < n_units) {
        p.next(a);
        if (p.unit == 0 && warp == 0) {  // a new item: its queries towards L2, a line to a lane
          const int bytes = DH * paged_dtype_bytes(a.q_dtype), at = lane * 128;
          const int r = at / bytes;
          if (r < group)
            prefetch_l2(static_cast<const uint8_t *>(a.q) +
                        (p.b * a.q_stride[0] + (int64_t)(p.h * group + r) * a.q_stride[1]) * paged_dtype_bytes(a.q_dtype) +
                        at % bytes);
        }
      }
      fetch_page();
    }
  };

  fetch_page();
#pragma unroll
  for (int x = 0; x < NS - 1; ++x) {
    issue(x, x & 1);
    cp_commit();
  }

  // ---- consumer side. Lane (g, t) holds, of the accumulators, heads 2t and 2t + 1; of the B operands, head g.
  const uint32_t k_at = ((lane & 15) * ROW) + (((lane >> 4) ^ swz(lane & 7)) << 4);  // ldmatrix row of the lane
  const uint32_t v_at = ((((lane >> 4) << 3) + (lane & 7)) * ROW) + ((((lane >> 3) & 1) ^ swz(lane & 7)) << 4);
  uint32_t qb[KSTEPS][SPLIT ? 4 : 2];
  float rs[2], m[2], bias[2], l[2], o[MT][4];  // rs: score scale in log2 units; bias: P_BIAS - m
  bool first = true;
  bool starts = c.unit == 0;  // this block holds the item's first unit
  int ring = 0;               // slot of the next half

  for (int u = 0; u < n_units; ++u) {
    if (first) {  // a new item: its query heads as B fragments
      first = false;
      const int qs = paged_dtype_bytes(a.q_dtype);
      const bool pair = ((uintptr_t)a.q | (uintptr_t)(a.q_stride[0] * qs) | (uintptr_t)(a.q_stride[1] * qs)) % (2 * qs) == 0;
      const int64_t at = c.b * a.q_stride[0] + (int64_t)(c.h * group + g) * a.q_stride[1];
      float2 f[KSTEPS][2];
#pragma unroll
      for (int st = 0; st < KSTEPS; ++st)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // E4M3 rows come as four codes to a lane, so that the k order of a step is 4t .. 4t + 3
          const int d = 16 * st + (KIND == PG_E4M3 ? 4 * t + 2 * e : 2 * t + 8 * e);
          f[st][e] = g < group ? load_pair(a.q, at + d, a.q_dtype, pair) : make_float2(0.f, 0.f);
        }
      float down = 1.f;
      if (SPLIT) {  // bring the head's largest element to [2^13, 2^14) by a power of two
        float top = 0.f;
#pragma unroll
        for (int st = 0; st < KSTEPS; ++st)
#pragma unroll
          for (int e = 0; e < 2; ++e) top = fmaxf(top, fmaxf(fabsf(f[st][e].x), fabsf(f[st][e].y)));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int e2 = 0;
        if (top > 0.f && top <= FLT_MAX) e2 = max(-120, min(120, 140 - (int)(__float_as_uint(top) >> 23)));
        const float up = __int_as_float((127 + e2) << 23);
        down = __int_as_float((127 - e2) << 23);
#pragma unroll
        for (int st = 0; st < KSTEPS; ++st)
#pragma unroll
          for (int e = 0; e < 2; ++e) f[st][e].x *= up, f[st][e].y *= up;
      }
#pragma unroll
      for (int st = 0; st < KSTEPS; ++st)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          qb[st][e] = pack16<KIND>(f[st][e].x, f[st][e].y);
          if (SPLIT) qb[st][SPLIT ? 2 + e : e] = rest16<KIND>(f[st][e].x, f[st][e].y, qb[st][e]);
        }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        rs[h] = a.scale * LOG2E;
        if (SPLIT) rs[h] *= __shfl_sync(0xffffffffu, down, 8 * t + 4 * h);  // of head 2t + h
        m[h] = -INFINITY;
        bias[h] = P_BIAS;
        l[h] = 0.f;
      }
#pragma unroll
      for (int n = 0; n < MT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    }

    // ---- K half: scores of the tile, s[.][2p + h] of position g + 8p and head 2t + h
    cp_wait<NS - 2>();
    __syncwarp();
    issue(ring == 0 ? NS - 1 : ring - 1, (NS - 1) & 1);
    cp_commit();
    const uint32_t live = sm.live[warp][ring];
    float s[SUBS][4];
    if (live) {
      const uint32_t kt = ring0 + ring * T::HALF + k_at;
#pragma unroll
      for (int i = 0; i < SUBS; ++i) {
        float x[2][4] = {};
        if (KIND != PG_E4M3) {
#pragma unroll
          for (int st = 0; st < KSTEPS; ++st) {
            uint32_t A[4];
            ldsm4(A, kt ^ (st << 5));
            mma16<KIND>(x[SPLIT ? 0 : st & 1], A, qb[st][0], qb[st][1]);
            if (SPLIT) mma16<KIND>(x[1], A, qb[st][SPLIT ? 2 : 0], qb[st][SPLIT ? 3 : 0]);
          }
        } else {
#pragma unroll
          for (int st = 0; st < KSTEPS; st += 2) {
            uint32_t r[4];
            ldsm4(r, (kt ^ (st << 4)) + i * 16 * ROW);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t A[4] = {e4m3x2(r[2 * k] & 0xffffu), e4m3x2(r[2 * k + 1] & 0xffffu), e4m3x2(r[2 * k] >> 16),
                                     e4m3x2(r[2 * k + 1] >> 16)};
              mma16<KIND>(x[0], A, qb[st + k][0], qb[st + k][1]);
              mma16<KIND>(x[1], A, qb[st + k][SPLIT ? 2 : 0], qb[st + k][SPLIT ? 3 : 0]);
            }
          }
        }
        float ks[2] = {1.f, 1.f};
        if (KIND == PG_E4M3) {
          ks[0] = sm.scale[warp][KIND == PG_E4M3 ? ring : 0][16 * i + g];
          ks[1] = sm.scale[warp][KIND == PG_E4M3 ? ring : 0][16 * i + g + 8];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] = (x[0][e] + x[1][e]) * ks[e >> 1];
      }
    }
    ring = ring + 1 == NS ? 0 : ring + 1;

    // ---- V half: weights and outputs
    cp_wait<NS - 2>();
    __syncwarp();
    issue(ring == 0 ? NS - 1 : ring - 1, NS & 1);
    cp_commit();
    if (live) {
      float vs[SUBS][2], w[SUBS][4], part[2] = {0.f, 0.f};
      bool far = m[0] == -INFINITY || m[1] == -INFINITY;
      auto weights = [&]() {
        part[0] = part[1] = 0.f;
#pragma unroll
        for (int i = 0; i < SUBS; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = fmaf(s[i][e], rs[e & 1], bias[e & 1]);
            if (live != FULL && !((live >> (16 * i + g + 8 * (e >> 1))) & 1u)) x = -INFINITY;
            const float y = ex2(x);
            part[e & 1] += y;
            w[i][e] = KIND == PG_E4M3 ? y * vs[i][e >> 1] : y;
          }
      };
#pragma unroll
      for (int i = 0; i < SUBS; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          vs[i][k] = KIND == PG_E4M3 ? sm.scale[warp][KIND == PG_E4M3 ? ring : 0][16 * i + g + 8 * k] : 1.f;
      weights();
#pragma unroll
      for (int i = 0; i < SUBS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) far = far || fabsf(w[i][e]) > P_LIMIT;
      if (__any_sync(0xffffffffu, far)) {  // move the references to the maxima so far
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < SUBS; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if ((live >> (16 * i + g + 8 * (e >> 1))) & 1u)
              top[e & 1] = fmaxf(top[e & 1], fmaf(s[i][e], rs[e & 1],
                                                  KIND == PG_E4M3 ? fmaxf(lg2(fabsf(vs[i][e >> 1])), MIN_LOG2_SCALE) : 0.f));
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], x));
          const float mn = fmaxf(m[h], top[h]);
          f[h] = m[h] == mn ? 1.f : ex2(m[h] - mn);
          m[h] = mn;
          bias[h] = P_BIAS - (mn == -INFINITY ? 0.f : mn);
          l[h] *= f[h];
        }
#pragma unroll
        for (int n = 0; n < MT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][e] *= f[e & 1];
        weights();
      }
      l[0] += part[0];
      l[1] += part[1];
      const uint32_t vt = ring0 + ring * T::HALF + v_at;
#pragma unroll
      for (int i = 0; i < SUBS; ++i) {
        const uint32_t h0 = pack16<KIND>(w[i][0], w[i][1]), h1 = pack16<KIND>(w[i][2], w[i][3]);
        const uint32_t r0 = rest16<KIND>(w[i][0], w[i][1], h0), r1 = rest16<KIND>(w[i][2], w[i][3], h1);
        const uint32_t B[4] = {transpose8(h0), transpose8(h1), transpose8(r0), transpose8(r1)};
        if (KIND != PG_E4M3) {
#pragma unroll
          for (int n = 0; n < MT; ++n) {
            uint32_t A[4];
            ldsm4_trans(A, vt ^ (n << 5));
            mma16<KIND>(o[n], A, B[0], B[1]);
            mma16<KIND>(o[n], A, B[2], B[3]);
          }
        } else {
          // a transposed pair of codes: positions 2t, 2t + 1 of dimensions 2g and 2g + 1, rows g and g + 8 of the tile
#pragma unroll
          for (int n = 0; n < MT; n += 2) {
            uint32_t r[4];
            ldsm4_trans(r, (vt ^ (n << 4)) + i * 16 * ROW);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t x = __byte_perm(r[k], 0u, 0x3120), y = __byte_perm(r[2 + k], 0u, 0x3120);
              const uint32_t A[4] = {e4m3x2(x & 0xffffu), e4m3x2(x >> 16), e4m3x2(y & 0xffffu), e4m3x2(y >> 16)};
              mma16<KIND>(o[n + k], A, B[0], B[1]);
              mma16<KIND>(o[n + k], A, B[2], B[3]);
            }
          }
        }
      }
    }

    // ---- the item's end, or the run's: join the four warps through the slot just used
    const bool ends = c.unit + 1 == c.s.n;
    if (ends || u + 1 == n_units) {
      __syncwarp();  // every lane is done with the slot
      float *join = reinterpret_cast<float *>(sm.ring[warp][ring]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], x);
        const int r = 2 * t + h;
        if (g == 0) {
          sm.m[warp][r] = m[h] - P_BIAS;
          sm.l[warp][r] = l[h];
        }
#pragma unroll
        for (int n = 0; n < MT; ++n) {
          if (KIND == PG_E4M3) {
            *reinterpret_cast<float2 *>(&join[r * DH + join_col<KIND>(r, 16 * n + 2 * g)]) = make_float2(o[n][h], o[n][2 + h]);
          } else {
            join[r * DH + join_col<KIND>(r, 16 * n + g)] = o[n][h];
            join[r * DH + join_col<KIND>(r, 16 * n + g + 8)] = o[n][2 + h];
          }
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
          const float4 y = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(sm.ring[w][ring]) + r * DH +
                                                             join_col<KIND>(r, d));
          L = fmaf(sm.l[w][r], f, L);
          acc.x = fmaf(y.x, f, acc.x), acc.y = fmaf(y.y, f, acc.y), acc.z = fmaf(y.z, f, acc.z), acc.w = fmaf(y.w, f, acc.w);
        }
        if (whole) {
          paged_finish4(a, c.b, (int64_t)c.h * group + r, d, acc, M, L);
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
      __syncthreads();  // the next half may land in the slot, and the next item's sums in theirs
      first = true;
      starts = true;
    }
    ring = ring + 1 == NS ? 0 : ring + 1;
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
