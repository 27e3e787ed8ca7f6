// kie_paged_prefix_attention: a plan, attention of the rows of each group over the positions of their prefix, the rows' own
// positions beside it (kie_paged_attn.cu), and the join of the pieces of both.
//
// For one KV head, the query heads of a group's rows are the rows of a matrix: with 5 query heads a KV head, 25 sequences
// fill the 128 rows of a tensor-core tile, so that what kie_paged_attn.cu has to do as matrix-vector products becomes
// S = Q K^T and O += P V on tcgen05. A tile is two such halves, which share what is loaded of K and V. Work is a list of items
// (group, tile of its rows, KV head), each a row of units of 64 positions; every block, one to an SM, takes an equal run of the
// list and writes a piece (O, reference, sum of weights) for each item that it has part in.
//
// In a block a warp brings K and another V into a ring by TMA (one for both took 1,300 cycles for each 64 positions in pages
// of 16), a warp issues the MMAs of each half (one for both, which waits for one half while the other could go on: 3,800
// instead of 2,200 cycles a unit, 256 rows 70 instead of 64 us), four turn E4M3 codes into fp16 on the way where there are
// codes, and four for each half hold the softmax: thread = row = TMEM lane, so its maxima and sums need no shuffles. S is
// double-buffered in TMEM, so that the scores of the next unit are formed while this one's weights are; the weights go back
// over the scores, as the TMEM operand of the second product. As in kie_paged_attn.cu, the softmax's reference stays within
// 2^8 of the running maximum and O is only rescaled when a weight would pass 2^15, weights and fp32 queries are two 16-bit
// parts, and the sum of weights is of the weights before they are rounded. (Two bf16 parts hold a weight to 2^-17: of the
// outputs of 256 rows below 0.27 % are a bf16 step from those of an fp32 evaluation, at the same distance from 64 bits. With
// one part, 2^-9 of a weight, 256 rows take 62.1 instead of 64.7 us and 64 samples 34.3 instead of 34.9.)
//
// Measured: 64 rows of 20 / 4 heads over 8,192 positions and up to 512 of their own, fp16, 37 us (plan 4, prefix 23, own
// positions 3 more behind it, join 6); 256 rows of 16 / 4 heads in 8 groups over 4,096 and up to 1,024 of their own,
// bf16, 64 us (5, 33, 21, 6); 4 rows over 1,024, fp32 queries, 16 us (4, 9, 2, 3); 61 rows, 5 prefixes of 513 to 8,191,
// on E4M3, 38. The prefix kernel is bound by the chain QK, softmax, PV of a half (2,200 cycles a unit; its MMAs alone are
// 900, the tensor pipe is busy for 24 to 35 %), and takes 5 us until its first MMA; beside it one block of the other
// kernel fits an SM, so that large own parts run on behind it.
#include <cuda.h>
#include <float.h>
#include <limits.h>

#include <algorithm>
#include <atomic>

#include "kie_device.cuh"
#include "kie_paged.cuh"
#include "kie_tc.cuh"

namespace kie {
namespace {

constexpr int PX_M = 128, PX_N = 64;       // rows of a half of a tile (an MMA's), positions of a unit
// Warps: four of the softmax for each half of a tile, the loaders of K and of V, one that issues the MMAs of each half, and
// where the cache holds codes those that convert them.
constexpr int PX_SOFT = 4, PX_LOADER = 8, PX_ISSUER = 10, PX_CONVERT = 12, PX_CONVERTERS = 4;
// Registers of a thread: with 12 warps they leave room on the SM for a block of the rows' own attention on 16-bit pages.
constexpr int PX_REGISTERS = 112;
// Depth of what is kept per unit besides K and V. The loaders are at most NS + RAW <= 6 halves ahead of the oldest one in use,
// so at most four units ahead of the one whose weights are formed.
constexpr int PX_TILES = 8;
constexpr uint32_t PX_TMEM = 512;          // columns: for each half, S twice and O
constexpr float LOG2E = 1.4426950408889634f;
constexpr float P_BIAS = 7.f, P_STEP = 8.f;  // weights are 2^7 2^(v - reference), below 2^15
constexpr float MIN_LOG2_SCALE = -60.f, MAX_LOG2_SCALE = 127.f;  // of E4M3 values, as in kie_paged_attn.cu

enum { PG_F16 = 0, PG_BF16 = 1, PG_E4M3 = 2 };

template <int KIND, int DH, bool SPLIT>
struct PxShape {
  static constexpr int Q_HALF = PX_M * DH * 2 * (SPLIT ? 2 : 1), SLOT = PX_N * DH * 2, CODES = PX_N * DH;
  static constexpr int NS = KIND == PG_E4M3 ? 3 : 5;     // ring slots
  static constexpr int RAW = KIND == PG_E4M3 ? 3 : 1;  // of codes as they come
  static constexpr int THREADS = 32 * (PX_CONVERT + (KIND == PG_E4M3 ? PX_CONVERTERS : 0));
};

// Of the block's waits: how long each may take, and whether one took longer. Then the barriers' phases no longer tell what
// has happened, so that nothing that waits on them goes on: the block gives up (see prefix_kernel).
struct Waits {
  unsigned long long limit_ns;
  int failed;
};

template <int KIND, int DH, bool SPLIT>
struct PxSmem {
  using T = PxShape<KIND, DH, SPLIT>;
  static constexpr bool E4M3 = KIND == PG_E4M3;
  uint8_t q[2][T::Q_HALF];       // of each half: [part][64-dim block][row][128 B], 16-byte chunks swizzled by the row
  uint8_t ring[T::NS][T::SLOT];  // [64-dim block][position][128 B], the same
  uint8_t raw[E4M3 ? T::RAW : 1][E4M3 ? T::CODES : 16];  // [position][DH]
  float scale[E4M3 ? PX_TILES : 1][3][E4M3 ? PX_N : 1];  // of K, of V, log2 of V's
  uint32_t live[PX_TILES];       // bit i: positions 16 i .. 16 i + 15 lie on a page
  float rs[2][PX_M];             // score scale of a row, in log2 units
  uint64_t full[T::NS], empty[T::NS], unit[PX_TILES], s_full[2][2], p_full[2][2], pv_done[2][2], fix, raw_full[T::RAW], raw_empty[T::RAW];
  int reach;                     // positions of the prefix that the longest row of the group has
  int sent[2];                   // units of K and of V that the loaders have brought for the item
  uint32_t tmem;
  Waits waits;
};

// 32 consecutive columns of the warp's 32 TMEM lanes, a lane's to each thread. Nothing waits for them here.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// True in one lane of the (converged) warp. The compiler knows that no more than one thread is at what is behind it.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// tcgen05.mma with A in TMEM.
__device__ __forceinline__ void tc_mma_ts(uint32_t dtmem, uint32_t atmem, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(dtmem),
      "r"(atmem), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}

// Matrix descriptors of 128-byte rows whose 16-byte chunks are swizzled by the row (mod 8): groups of 8 rows are 1,024 bytes
// apart. `lead` is the step between 64-element blocks of a row, which only an operand that is contiguous along M or N uses.
__device__ __forceinline__ uint64_t px_desc(uint32_t saddr, uint32_t lead) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f16, fp32 accumulator, M = 128; B contiguous along N where b_mn is set.
__host__ __device__ constexpr uint32_t px_idesc(int n, bool bf16, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(PX_M >> 4) << 24);
}

// Eight floats, a whole sector, to a 32-byte aligned address.
__device__ __forceinline__ void store8(float *p, const float *v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
               "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float log2_scale(float x) { return fminf(fmaxf(lg2(fabsf(x)), MIN_LOG2_SCALE), MAX_LOG2_SCALE); }

template <int KIND>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  return pack2(a, b, KIND == PG_BF16 ? KIE_BF16 : KIE_F16);
}
template <int KIND>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
  if (KIND == PG_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ uint32_t e4m3x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}

// A box of the tensor behind a map, at these coordinates, into shared memory; what lies outside the tensor becomes zeros.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Waits for a phase of a barrier of this block, for a limited time; false if that ran out, here or in another wait.
__device__ __forceinline__ bool px_wait(uint64_t *bar, uint32_t parity, Waits *waits) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (int spins = 1;; ++spins) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((spins & 63) == 0) {
      if (*static_cast<volatile int *>(&waits->failed)) return false;
      if (globaltimer() - t0 > waits->limit_ns) {
        *static_cast<volatile int *>(&waits->failed) = 1;
        return false;
      }
    }
  }
}

// The same for a whole warp at once.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, Waits *waits) {
  return __all_sync(0xffffffffu, px_wait(bar, parity, waits)) != 0;
}

// After a failure: for a copy or products that are under way, for the same time at most, whatever else has run out.
__device__ __noinline__ void settle(uint64_t *bar, uint32_t parity, const Waits *waits) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer() - t0 > waits->limit_ns) return;
}

// K and V of the cache as tensors of four dimensions: dims, and three that order tells, two bits each (0 position, 1 head, 2
// page); boxes of `rows` positions.
struct PrefixMaps {
  CUtensorMap k, v;
  int order[2], rows;
};

// ---- the list ------------------------------------------------------------------------------------------------

__device__ __forceinline__ int clamp_start(const PrefixArgs &a, int g) { return min(max(a.group_start[g], 0), a.n_seqs); }

// Group g: rows [start, end), its prefix, tiles of `members` rows, and units of an item.
struct Group {
  int start, end, prefix, units;
  __device__ __forceinline__ int tiles(int members) const { return (end - start + members - 1) / members; }
};
__device__ __forceinline__ Group group_of(const PrefixArgs &a, int g, int start, int end) {
  Group x;
  x.start = start;
  x.end = end;
  x.prefix = min(max(a.prefix_lens[g], 0), a.max_blocks * a.pages.block_size);
  x.units = end > start ? (x.prefix + PX_N - 1) / PX_N : 0;
  return x;
}
// Places in the list of a group's items.
__device__ __forceinline__ long long places_of(const PrefixArgs &a, const Group &x, int members) {
  return x.units ? (long long)x.tiles(members) * a.pages.n_kv_heads * (x.units + PX_ITEM_COST) : 0;
}

// Length of a query row whose sequence has a table row, else 0.
__device__ __forceinline__ int sequence_of(const PrefixArgs &a, int b) { return a.seqs ? a.seqs[b] : b; }
__device__ __forceinline__ int length_of(const PrefixArgs &a, int b) {
  return (unsigned)sequence_of(a, b) < (unsigned)a.n_table ? row_len(a, b) : 0;
}

__device__ __forceinline__ long long divide_up(long long a, unsigned b) {  // a 64-bit division takes a few hundred cycles
  a += b - 1;
  return (a >> 32) == 0 ? (long long)((unsigned)a / b) : a / b;
}

constexpr int PL_THREADS = 1024;
// Sums over the block in thread order: v becomes the sum of the threads' before this one, *all of all.
__device__ __forceinline__ long long sum_before(long long v, long long *all) {
  __shared__ long long s_warp[PL_THREADS / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long up = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += x;
  }
  if (lane == 31) s_warp[warp] = up;
  __syncthreads();
  long long w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += x;
  }
  *all = __shfl_sync(0xffffffffu, w, 31);
  const long long before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return up - v + (warp > 0 ? before : 0);
}

// The list: what each row and each block of the prefixes' kernel has to know. Every block of the plan goes over all groups and
// then sees to its share of the rows and blocks.
__global__ void __launch_bounds__(PL_THREADS) plan_kernel(const PrefixArgs a, int prefix_blocks) {
  begin_after_previous();
  extern __shared__ long long base[];  // places before each group, and before the end
  int *const starts = reinterpret_cast<int *>(base + a.n_groups + 1);
  const int tid = threadIdx.x, G = a.n_groups, heads = a.pages.n_kv_heads, group = a.n_heads / heads, members = 2 * (PX_M / group);
  const int each = (G + PL_THREADS - 1) / PL_THREADS, g0 = min(tid * each, G), g1 = min(g0 + each, G);
  bool falls = false;
  long long mine = 0, total;
  for (int g = g0; g < g1; ++g) {
    const int start = clamp_start(a, g), end = clamp_start(a, g + 1);
    falls |= end < start;
    mine += places_of(a, group_of(a, g, start, end), members);
    starts[g] = start;
  }
  if (tid == 0) starts[G] = clamp_start(a, G);
  if (__syncthreads_or(falls)) {  // a start below an earlier one counts as that one
    if (tid == 0)
      for (int g = 0; g < G; ++g) starts[g + 1] = max(starts[g + 1], starts[g]);
    __syncthreads();
    mine = 0;
    for (int g = g0; g < g1; ++g) mine += places_of(a, group_of(a, g, starts[g], starts[g + 1]), members);
  }
  long long at = sum_before(mine, &total);
  for (int g = g0; g < g1; ++g) {
    base[g] = at;
    at += places_of(a, group_of(a, g, starts[g], starts[g + 1]), members);
  }
  if (tid == 0) base[G] = total;
  __syncthreads();
  const long long per = max(divide_up(total, prefix_blocks), (long long)PX_MIN_RUN);
  if (blockIdx.x == 0 && tid == 0) *a.per_block = per;
  for (int k = blockIdx.x * PL_THREADS + tid; k < prefix_blocks; k += gridDim.x * PL_THREADS) {
    const long long v0 = k * per;
    PrefixBlock b = {-1, 0, 0, 0, 0};
    if (v0 < total) {
      int lo = 0, hi = G;  // the last group that begins at v0 or before it and is not empty
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (base[mid] <= v0)
          lo = mid;
        else
          hi = mid;
      }
      const Group x = group_of(a, lo, starts[lo], starts[lo + 1]);
      const unsigned span = x.units + PX_ITEM_COST;
      b.g = lo, b.start = x.start, b.end = x.end;
      b.item = (int)(divide_up(v0 - base[lo] + 1, span) - 1);
      b.place = base[lo] + (long long)b.item * span;
    }
    a.blocks[k] = b;
  }
  for (int b = blockIdx.x * PL_THREADS + tid; b < a.n_seqs; b += gridDim.x * PL_THREADS) {
    int lo = 0, hi = G + 1;  // the number of starts that are not behind the row
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (starts[mid] <= b)
        lo = mid + 1;
      else
        hi = mid;
    }
    const int g = lo - 1;
    PrefixRow row = {};
    if (g >= 0 && g < G) {
      const Group x = group_of(a, g, starts[g], starts[g + 1]);
      const int t = (b - x.start) / members, first = x.start + t * members;
      row.lo = min(x.prefix, length_of(a, b));
      row.units = x.units;
      row.place = base[g] + (long long)t * heads * (x.units + PX_ITEM_COST);
      row.slot = first * a.n_heads;
      row.rows = min(members, x.end - first) * group;
      row.local = (b - first) * group;
    }
    a.row_lo[b] = row.lo;
    a.rows[b] = row;
  }
}

// The E neighbouring elements of a query that start at `at`, as they are: fp32 (WIDE) or two to a word; zeros if not live.
template <bool WIDE, int E>
__device__ __forceinline__ void load_query(const PrefixArgs &a, bool vec, bool live, int64_t at, uint32_t (&w)[WIDE ? E : E / 2]) {
  constexpr int N = WIDE ? E : E / 2;
#pragma unroll
  for (int e = 0; e < N; ++e) w[e] = 0u;
  if (!live) return;
  if (vec) {
    const void *p = static_cast<const uint8_t *>(a.q) + at * (WIDE ? 4 : 2);
    if (N == 4) {
      const uint4 x = *static_cast<const uint4 *>(p);
      w[0] = x.x, w[N > 1 ? 1 : 0] = x.y, w[N > 2 ? 2 : 0] = x.z, w[N - 1] = x.w;
    } else if (N == 2) {
      const uint2 x = *static_cast<const uint2 *>(p);
      w[0] = x.x, w[N - 1] = x.y;
    } else {
      w[0] = *static_cast<const uint32_t *>(p);
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      w[e] = WIDE ? static_cast<const uint32_t *>(a.q)[at + e]
                  : static_cast<const uint16_t *>(a.q)[at + 2 * e] | (uint32_t) static_cast<const uint16_t *>(a.q)[at + 2 * e + 1] << 16;
  }
}

// ---- the three roles of a block, for units u0 .. u0 + n - 1 of an item -------------------------------------------
// `tiles` and `halves` count the units, and the halves of them in the ring, of the items before. The halves' order is that
// of their use: K0, K1, V0, K2, V1, .., V(n - 1).

// A wait by parity tells a phase of a barrier from the one before it only: whoever waits here knows that the one before is
// over, and the next one cannot end before it has gone on. (Hence two barriers for S, for P and for what follows P, each
// taking every second unit.)

// Slot of a half, and the parity of its round through the ring.
template <int NS>
struct Half {
  uint32_t slot, round;
  __device__ __forceinline__ explicit Half(uint32_t i) : slot(i % NS), round(i / NS & 1u) {}
};

// The halves of n units come as K0 K1 V0 K2 V1 ...: where K or V of unit u comes,
__device__ __forceinline__ int half_of(int u, int n, bool is_v) {
  return is_v ? min(2 * u + 2, 2 * n - 1) : max(2 * u - 1, 0);
}
// and of half i its unit, and whether it is V.
__device__ __forceinline__ int unit_of(int i, int n, bool *is_v) {
  if (i == 0) return *is_v = false, 0;
  if (i == 2 * n - 1) return *is_v = true, n - 1;
  *is_v = !(i & 1);
  return (i & 1) ? (i + 1) / 2 : i / 2 - 1;
}

// The warp that loads K, or V. Finds the group's longest row (the first of them), through whose table row the prefix is read, and loads, without
// waiting for the queries. Returns the number of units, all of them with positions. *mending: the last copy is one of V's end, and
// did not come in time.
template <int KIND, int DH, bool SPLIT>
__device__ __forceinline__ int load_item(const PrefixArgs &a, const PrefixMaps &maps, PxSmem<KIND, DH, SPLIT> &sm, const Group &x,
                                         bool is_v, int h, int u0, int u1, uint32_t tiles, uint32_t halves, uint32_t &fixes,
                                         bool *mending) {
  using T = PxShape<KIND, DH, SPLIT>;
  constexpr bool CODES = KIND == PG_E4M3;
  constexpr int NS = CODES ? T::RAW : T::NS, KB = CODES ? 1 : DH / 64;
  constexpr uint32_t BYTES = CODES ? T::CODES : T::SLOT;
  const int lane = threadIdx.x & 31;
  int reach = 0, source = x.start;
#pragma unroll 2
  for (int b = x.start + lane; b < x.end; b += 32) {
    const int len = min(x.prefix, length_of(a, b));
    if (len > reach) reach = len, source = b;
  }
  const int mine = reach;
  reach = __reduce_max_sync(0xffffffffu, reach);
  source = __reduce_min_sync(0xffffffffu, mine == reach ? source : INT_MAX);
  if (lane == 0 && !is_v) sm.reach = reach;
  asm volatile("bar.arrive 1, %0;" ::"n"(T::THREADS) : "memory");  // the others, once the queries are there
  const int n = max(0, min(u1, (reach + PX_N - 1) / PX_N) - u0);
  const int *pages = a.block_table + (n > 0 ? sequence_of(a, source) : 0) * a.table_stride;
  const unsigned bs = a.pages.block_size;

  // lane: page and place in it of 16 positions, of eight units from `batch` on and of the eight behind them
  int batch = u0, page_a, at_a, page_b, at_b;
  const auto fetch = [&](int unit, int *page, int *at) {
    const int pos = unit * PX_N + 16 * lane;
    const unsigned j = (unsigned)pos / bs;
    *at = pos - (int)(j * bs);
    *page = unit < u0 + n && pos < reach ? pages[j] : -1;
    if ((unsigned)*page >= (unsigned)a.pages.n_blocks) *page = -1;
  };
  fetch(u0, &page_a, &at_a);
  fetch(u0 + 8, &page_b, &at_b);
  const int runs = PX_N / maps.rows;  // boxes of maps.rows positions by 128 bytes
  uint64_t *const full = CODES ? sm.raw_full : sm.full, *const empty = CODES ? sm.raw_empty : sm.empty;
  const uint32_t ring = smem_u32(CODES ? &sm.raw[0][0] : &sm.ring[0][0]);
  float ks[2], vs[2];         // E4M3: the next unit's scales, positions lane and lane + 32
  const auto request_scales = [&](int unit) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int row = lane + 32 * k, from = (unit - batch) * 4 + (row >> 4);
      const int page = __shfl_sync(0xffffffffu, page_a, from & 31), off = __shfl_sync(0xffffffffu, at_a, from & 31) + (row & 15);
      ks[k] = vs[k] = 0.f;
      if (page >= 0 && unit * PX_N + row < reach) {
        ks[k] = a.pages.k_scale[page * a.pages.k_scale_stride[0] + h * a.pages.k_scale_stride[1] + off * a.pages.k_scale_stride[2]];
        vs[k] = a.pages.v_scale[page * a.pages.v_scale_stride[0] + h * a.pages.v_scale_stride[1] + off * a.pages.v_scale_stride[2]];
      }
    }
  };
  const auto turn_to = [&](int unit) {
    if (unit < batch + 8) return;
    batch += 8;
    page_a = page_b, at_a = at_b;
    fetch(batch + 8, &page_b, &at_b);
  };
  if (CODES && !is_v && n > 0) request_scales(u0);
  const CUtensorMap *const map = is_v ? &maps.v : &maps.k;
  const int order = maps.order[is_v];
  const auto load = [&](int u) {
    const int unit = u0 + u;
    const uint32_t half = halves + half_of(u, n, is_v), slot = half % NS;
    turn_to(unit);
    const uint32_t live = __ballot_sync(0xffffffffu, page_a >= 0) >> ((unit - batch) * 4) & 15u;
    if (blockIdx.x == a.stop_block && half >= a.stop_half) return false;
    if (!warp_wait(&empty[slot], (half / NS & 1u) ^ 1u, &sm.waits)) return false;
    // rows of V behind the end would meet weights of 0 as whatever they hold: they become zeros before the MMA may begin
    const int tail = reach - unit * PX_N;
    const bool mend = !CODES && is_v && tail < PX_N;
    uint64_t *const bar = mend ? &sm.fix : &full[slot];
    const bool one = elect_one();
    if (one) mbar_arrive_expect_tx(bar, BYTES);
    uint32_t to = ring + slot * BYTES;
#pragma unroll 1
    for (int run = 0; run < runs; ++run, to += maps.rows * (CODES ? DH : 128)) {
      const int from = (unit - batch) * 4 + run * (maps.rows >> 4);
      const int p = __shfl_sync(0xffffffffu, page_a, from), y = __shfl_sync(0xffffffffu, at_a, from);
      const int z = p >= 0 ? p : a.pages.n_blocks;
      const auto coordinate = [&](int what) { return (what & 3) == 0 ? y : (what & 3) == 1 ? h : z; };
      if (one) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
          tma_box(to + kb * (PX_N * 128), map, kb * 64, coordinate(order), coordinate(order >> 2), coordinate(order >> 4), bar);
      }
    }
    __syncwarp();
    if (mend) {
      if (!warp_wait(&sm.fix, fixes++ & 1u, &sm.waits)) return *mending = true, false;
      for (int k = tail * 8 + lane; k < PX_N * 8; k += 32)
#pragma unroll
        for (int b = 0; b < KB; ++b)
          *reinterpret_cast<uint4 *>(&sm.ring[CODES ? 0 : slot][b * (PX_N * 128) + k * 16]) = make_uint4(0u, 0u, 0u, 0u);
      fence_async_proxy();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[slot]);
    }
    if (!is_v) {
      const uint32_t k = (tiles + u) % PX_TILES;
      if (CODES) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sm.scale[CODES ? k : 0][0][CODES ? lane + 32 * e : 0] = ks[e];
          sm.scale[CODES ? k : 0][1][CODES ? lane + 32 * e : 0] = vs[e];
          sm.scale[CODES ? k : 0][2][CODES ? lane + 32 * e : 0] = log2_scale(vs[e]);
        }
        __syncwarp();
      }
      if (lane == 0) {
        sm.live[k] = live;
        mbar_arrive(&sm.unit[k]);
      }
    }
    if (CODES && !is_v && u + 1 < n) {
      turn_to(unit + 1);
      request_scales(unit + 1);
    }
    return true;
  };
  int sent = 0;
#pragma unroll 1
  while (sent < n && load(sent)) ++sent;
  if (lane == 0) sm.sent[is_v] = sent;
  return n;
}

// A loader, when the block has given up and every warp has stopped: waits for its copies that are under way. Slots that were
// asked for again since have been read, so that it is the ring's last round at most.
template <int KIND, int DH, bool SPLIT>
__device__ __forceinline__ void settle_loads(PxSmem<KIND, DH, SPLIT> &sm, bool is_v, int n, uint32_t halves, uint32_t fixes,
                                             bool mending) {
  using T = PxShape<KIND, DH, SPLIT>;
  constexpr bool CODES = KIND == PG_E4M3;
  constexpr int NS = CODES ? T::RAW : T::NS;
  const int k = sm.sent[0], v = sm.sent[1], own = is_v ? v : k;
  const int last = max(k > 0 ? half_of(k - 1, n, false) : -1, v > 0 ? half_of(v - 1, n, true) : -1);
  for (int u = max(0, own - NS); u < own; ++u) {
    const int i = half_of(u, n, is_v);
    const uint32_t half = halves + i;
    if (i + NS > last) settle(CODES ? &sm.raw_full[half % NS] : &sm.full[half % NS], half / NS & 1u, &sm.waits);
  }
  if (mending) settle(&sm.fix, (fixes - 1) & 1u, &sm.waits);
}

// PX_CONVERTERS warps: codes of the raw ring into fp16 in the other one, positions from the prefix's end on as zeros.
template <int KIND, int DH, bool SPLIT>
__device__ __forceinline__ void convert_item(PxSmem<KIND, DH, SPLIT> &sm, int ct, int reach, int u0, int n, uint32_t halves) {
  using T = PxShape<KIND, DH, SPLIT>;
  constexpr int CH = DH / 16, THREADS = 32 * PX_CONVERTERS, STEP = THREADS / CH, NS = T::NS, RAW = T::RAW;
  const int row0 = ct / CH, chunk = ct % CH, c = 2 * (chunk & 3), lane = ct & 31;
  for (int i = 0; i < 2 * n; ++i) {
    bool is_v;
    const int tail = reach - (u0 + unit_of(i, n, &is_v)) * PX_N;
    const uint32_t half = halves + i;
    if (!warp_wait(&sm.raw_full[half % RAW], half / RAW & 1u, &sm.waits)) return;
    if (!warp_wait(&sm.empty[half % NS], (half / NS & 1u) ^ 1u, &sm.waits)) return;
    const uint8_t *from = sm.raw[half % RAW] + chunk * 16;
    uint8_t *slot = sm.ring[half % NS] + (chunk >> 2) * (PX_N * 128);
#pragma unroll
    for (int k = 0; k < PX_N / STEP; ++k) {
      const int row = row0 + k * STEP;
      uint4 w = *reinterpret_cast<const uint4 *>(from + row * DH);
      if (row >= tail) w = make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4 *>(slot + row * 128 + ((c ^ (row & 7)) << 4)) =
          make_uint4(e4m3x2(w.x & 0xffffu), e4m3x2(w.x >> 16), e4m3x2(w.y & 0xffffu), e4m3x2(w.y >> 16));
      *reinterpret_cast<uint4 *>(slot + row * 128 + (((c + 1) ^ (row & 7)) << 4)) =
          make_uint4(e4m3x2(w.z & 0xffffu), e4m3x2(w.z >> 16), e4m3x2(w.w & 0xffffu), e4m3x2(w.w >> 16));
    }
    fence_async_proxy();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&sm.full[half % NS]);
      mbar_arrive(&sm.raw_empty[half % RAW]);
    }
  }
}

// The warp that issues for half w of a tile, an elected lane of which does. parts: halves of the tile that have rows. Returns the
// number of products that were issued: QK0, QK1, PV0, QK2, PV1, ..
template <int KIND, int DH, bool SPLIT>
__device__ __forceinline__ int multiply_item(PxSmem<KIND, DH, SPLIT> &sm, uint32_t tmem, int w, int parts, int n,
                                              uint32_t units, uint32_t halves) {
  using T = PxShape<KIND, DH, SPLIT>;
  constexpr int NS = T::NS, KB = DH / 64;
  constexpr uint32_t S_DESC = px_idesc(PX_N, KIND == PG_BF16, false), O_DESC = px_idesc(DH, KIND == PG_BF16, true);
  // descriptors of the first step; those of the others are 16-byte units further (addresses stay below 2^18)
  const uint64_t q0 = px_desc(smem_u32(sm.q[w]), 16), k0 = px_desc(smem_u32(sm.ring), 16), v0 = px_desc(smem_u32(sm.ring), PX_N * 128);
  constexpr uint32_t SLOT = T::SLOT / 16;
  uint32_t half = halves;
#pragma unroll 1
  for (int j = 0; j <= n; ++j) {
    if (j < n) {  // S = Q K^T
      const Half<NS> x(half);
      const uint32_t tile = units + j, buf = tile & 1u;
      if (!warp_wait(&sm.full[x.slot], x.round, &sm.waits)) return half - halves;
      if (j >= 2 && !warp_wait(&sm.pv_done[w][buf], (tile - 2) >> 1 & 1u, &sm.waits)) return half - halves;  // unit j - 2 is done with it
      tc_fence_after();
      if (elect_one()) {
        const uint64_t k = k0 + x.slot * SLOT;
        const uint32_t to = tmem + buf * PX_N;
#pragma unroll
        for (int p = SPLIT ? 1 : 0; p >= 0; --p)  // the second parts first: a large sum is cut off fewer times
#pragma unroll
          for (int s = 0; s < DH / 16; ++s)
            tc_mma(to, q0 + (p * KB + s / 4) * (PX_M * 8) + s % 4 * 2, k + s / 4 * (PX_N * 8) + s % 4 * 2, S_DESC,
                   p < (SPLIT ? 1 : 0) || s ? 1u : 0u);
        tc_commit(&sm.s_full[w][buf]);
        tc_commit(&sm.empty[x.slot]);
        if (parts == 1) tc_commit(&sm.empty[x.slot]);
      }
      __syncwarp();
      ++half;
    }
    if (j > 0) {  // O += P V
      const Half<NS> x(half);
      const uint32_t tile = units + j - 1, buf = tile & 1u;
      if (!warp_wait(&sm.full[x.slot], x.round, &sm.waits)) return half - halves;
      if (!warp_wait(&sm.p_full[w][buf], tile >> 1 & 1u, &sm.waits)) return half - halves;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t v = v0 + x.slot * SLOT;
        const uint32_t to = tmem + 2 * PX_N, p = tmem + buf * PX_N;
#pragma unroll
        for (int part = 1; part >= 0; --part)  // as above
#pragma unroll
          for (int s = 0; s < PX_N / 16; ++s)
            tc_mma_ts(to, p + s * 16 + part * 8, v + s * 128, O_DESC, j > 1 || s || !part ? 1u : 0u);
        tc_commit(&sm.pv_done[w][buf]);
        tc_commit(&sm.empty[x.slot]);
        if (parts == 1) tc_commit(&sm.empty[x.slot]);
      }
      __syncwarp();
      ++half;
    }
  }
  return half - halves;
}

// An issuer, when the block has given up and every warp has stopped: waits for the products that are under way, the last of
// which are of two units at most.
template <int KIND, int DH, bool SPLIT>
__device__ __forceinline__ void settle_products(PxSmem<KIND, DH, SPLIT> &sm, int w, int n, uint32_t units, int issued) {
  for (int i = max(0, issued - 4); i < issued; ++i) {
    bool is_pv;
    const uint32_t tile = units + unit_of(i, n, &is_pv);
    settle(is_pv ? &sm.pv_done[w][tile & 1u] : &sm.s_full[w][tile & 1u], tile >> 1 & 1u, &sm.waits);
  }
}

// Two fp32 operations at a time.
using Two = unsigned long long;
__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 both(Two r) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(r));
  return f;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// A thread is the row `row` of half `w`, which attends to positions below lim; `rows`: whether the warp has any row at all. m,
// l: the reference (log2 units) and the sum of weights. units: of the half, in the items before. O is complete on return; false if a wait ran out.
template <int KIND, int DH, bool SPLIT>
__device__ __forceinline__ bool soften_item(PxSmem<KIND, DH, SPLIT> &sm, uint32_t tmem, int w, int row, bool rows, int lim, int u0,
                                            int n, uint32_t tiles, uint32_t units, float *m_out, float *l_out) {
  constexpr bool E4M3 = KIND == PG_E4M3;
  const float rs = lim > 0 ? sm.rs[w][row] : 1.f;
  const uint32_t t_o = tmem + 2 * PX_N;
  const int lane = row & 31;
  float m = -INFINITY, l = 0.f;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const uint32_t place = (tiles + j) % PX_TILES, tile = units + j, t_s = tmem + (tile & 1u) * PX_N;
    const int left = lim - (u0 + j) * PX_N;  // positions of the unit that the row attends to
    if (!warp_wait(&sm.unit[place], (tiles + j) / PX_TILES & 1u, &sm.waits)) return false;
    if (!warp_wait(&sm.s_full[w][tile & 1u], tile >> 1 & 1u, &sm.waits)) return false;
    tc_fence_after();
    if (rows) {
      const uint32_t live = sm.live[place];
      const float *scale = &sm.scale[E4M3 ? place : 0][0][0];  // E4M3: of K, V, log2 of V's
      float s[2][32];
      tmem_ld32(t_s, s[0]);
      tmem_ld32(t_s + 32, s[1]);
      tmem_wait_ld();
      if (E4M3) {
#pragma unroll
        for (int e = 0; e < PX_N; e += 2) {
          const float2 k = *reinterpret_cast<const float2 *>(scale + (E4M3 ? e : 0));
          const float2 f = both(mul2(two(s[e / 32][e % 32], s[e / 32][e % 32 + 1]), two(k.x, k.y)));
          s[e / 32][e % 32] = f.x, s[e / 32][e % 32 + 1] = f.y;
        }
      }
      if (!__all_sync(0xffffffffu, left >= PX_N && live == 15u)) {
#pragma unroll
        for (int e = 0; e < PX_N; ++e)
          if (e >= left || !(live >> (e / 16) & 1u)) s[e / 32][e % 32] = -INFINITY;
      }
      const Two rs2 = two(rs, rs);
      float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < PX_N; e += 2) {
        float2 f = make_float2(s[e / 32][e % 32], s[e / 32][e % 32 + 1]);
        if (E4M3) {
          const float2 ls = *reinterpret_cast<const float2 *>(scale + (E4M3 ? 2 * PX_N + e : 0));
          f = both(fma2(two(f.x, f.y), rs2, two(ls.x, ls.y)));
        }
        tops[e / 2 & 3] = fmaxf(tops[e / 2 & 3], fmaxf(f.x, f.y));
      }
      float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
      if (!E4M3) top *= rs;
      const bool far = top > m + P_STEP;
      if (__any_sync(0xffffffffu, far)) {
        const float mn = far ? top : m, f = far && m != -INFINITY ? ex2(m - mn) : 1.f;
        m = mn;
        l *= f;
        if (j > 0) {
          if (!warp_wait(&sm.pv_done[w][(tile - 1) & 1u], (tile - 1) >> 1 & 1u, &sm.waits)) return false;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < DH; c += 16) {
            float o[16];
            tmem_ld16(t_o + c, o);
            uint32_t y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(o[e] * f);
            tmem_st16(t_o + c, y);
          }
        }
      }
      const float bias = P_BIAS - (m == -INFINITY ? 0.f : m);
      const Two bias2 = two(bias, bias), minus2 = two(-1.f, -1.f);
      Two part[2] = {0, 0};
#pragma unroll
      for (int c = 0; c < PX_N; c += 16) {  // the weights of 16 positions: eight columns of first parts, eight of second ones
        uint32_t y[16];
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const int at = c + e;
          const float2 x = both(fma2(two(s[at / 32][at % 32], s[at / 32][at % 32 + 1]), rs2, bias2));
          Two p = two(ex2(x.x), ex2(x.y));
          part[e / 2 & 1] = add2(part[e / 2 & 1], p);
          if (E4M3) {
            const float2 vs = *reinterpret_cast<const float2 *>(scale + (E4M3 ? PX_N + at : 0));
            p = mul2(p, two(vs.x, vs.y));
          }
          const float2 f = both(p);
          const uint32_t hi = pack16<KIND>(f.x, f.y);
          const float2 b = unpack16<KIND>(hi);
          const float2 lo = both(fma2(two(b.x, b.y), minus2, p));
          y[e / 2] = hi;
          y[8 + e / 2] = pack16<KIND>(lo.x, lo.y);
        }
        tmem_st16(t_s + c, y);
      }
      const float2 f = both(add2(part[0], part[1]));
      l += f.x + f.y;
      tmem_wait_st();
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.p_full[w][tile & 1u]);
  }
  if (n > 0 && !warp_wait(&sm.pv_done[w][(units + n - 1) & 1u], (units + n - 1) >> 1 & 1u, &sm.waits)) return false;
  *m_out = m;
  *l_out = l;
  return true;
}

// ---- the kernel ----------------------------------------------------------------------------------------------

// The rows of queries of an item, in the layout of an MMA operand, by every warp but the loaders.
template <int KIND, int DH, bool SPLIT>
__device__ __forceinline__ void stage_queries(const PrefixArgs &a, PxSmem<KIND, DH, SPLIT> &sm, int first, int h, int group, int rows0,
                                              int rows) {
  constexpr int KB = DH / 64, E = DH / 32, AHEAD = 4, WARPS = PxShape<KIND, DH, SPLIT>::THREADS / 32 - 2, CH = DH / 8;
  const int w = threadIdx.x >> 5, warp = w < PX_LOADER ? w : w - 2, lane = threadIdx.x & 31;
  const bool bf16_q = a.q_dtype == KIE_BF16;
  const int size = paged_dtype_bytes(a.q_dtype);
  const uintptr_t odd = (uintptr_t)a.q | (uintptr_t)(a.q_stride[0] * size) | (uintptr_t)(a.q_stride[1] * size);
  if (!SPLIT && !(KIND == PG_E4M3 && bf16_q) && a.scale > 0.f && odd % 16 == 0) {  // as they are, 16 bytes at a time
    if (lane == 0)
      for (int r = warp; r < rows; r += WARPS) sm.rs[r >= rows0][r >= rows0 ? r - rows0 : r] = fmaxf(a.scale, FLT_MIN) * LOG2E;
    const uint16_t *q = static_cast<const uint16_t *>(a.q) + (int64_t)first * a.q_stride[0] + (int64_t)h * group * a.q_stride[1];
#pragma unroll 4
    for (int i = warp * 32 + lane; i < rows * CH; i += 32 * WARPS) {
      const int r = i / CH, c = i % CH, w = r >= rows0, at = w ? r - rows0 : r;  // rows from rows0 on are the second half's
      const uint4 x = *reinterpret_cast<const uint4 *>(q + r / group * a.q_stride[0] + r % group * a.q_stride[1] + c * 8);
      *reinterpret_cast<uint4 *>(sm.q[w] + (c >> 3) * (PX_M * 128) + at * 128 + (((c & 7) ^ (at & 7)) << 4)) = x;
    }
    return;
  }
  // a warp takes a row at a time, a lane E neighbouring elements of it; the loads of four rows are on their way together
  const bool vec = odd % (E * size) == 0;
#pragma unroll 1
  for (int r0 = warp; r0 < rows; r0 += AHEAD * WARPS) {
    uint32_t raw[AHEAD][SPLIT ? E : E / 2];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int r = r0 + k * WARPS;
      const int64_t at = (int64_t)(first + r / group) * a.q_stride[0] + (int64_t)(h * group + r % group) * a.q_stride[1] + lane * E;
      load_query<SPLIT, E>(a, vec, r < rows, at, raw[k]);
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int r = r0 + k * WARPS;
      if (r >= rows) break;
      float q[E];
#pragma unroll
      for (int e = 0; e < E; ++e) q[e] = SPLIT ? __uint_as_float(raw[k][SPLIT ? e : 0]) : 0.f;
      if (!SPLIT) {
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          const float2 f = bf16_q ? unpack16<PG_BF16>(raw[k][e]) : unpack16<PG_F16>(raw[k][e]);
          q[2 * e] = f.x, q[2 * e + 1] = f.y;
        }
      }
      // Where 16 bits do not hold every query, the row's largest element is brought to [2^13, 2^14) by a power of two. The
      // sign of the scale goes into the queries, so that the largest score is the largest product.
      float up = a.scale < 0.f ? -1.f : 1.f, rs = fmaxf(fabsf(a.scale), FLT_MIN) * LOG2E;
      if (SPLIT || (KIND == PG_E4M3 && bf16_q)) {
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) top = fmaxf(top, fabsf(q[e]));
        top = warp_max(top);
        int e2 = 0;
        if (top > 0.f && top <= FLT_MAX) e2 = max(-120, min(120, 140 - (int)(__float_as_uint(top) >> 23)));
        up *= __int_as_float((127 + e2) << 23);
        rs = fmaxf(rs * __int_as_float((127 - e2) << 23), FLT_MIN);  // not 0: the scores of masked positions stay -inf
      }
      const int half = r >= rows0, place = half ? r - rows0 : r;
      if (lane == 0) sm.rs[half][place] = rs;
      uint32_t hi[E / 2], lo[E / 2];
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        const float u = q[2 * e] * up, v = q[2 * e + 1] * up;
        if (!SPLIT) {
          hi[e] = pack16<KIND>(u, v);
          lo[e] = 0u;
        } else {
          // The first part is cut off, not rounded, and a remainder of 0 becomes the least there is: both parts then have
          // the sign of the query, and an infinity in K gives the score that it should instead of NaN.
          const float f[2] = {u, v};
          uint16_t parts[2][2];
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const __half b = __float2half_rz(f[s]);
            uint16_t low = __half_as_ushort(__float2half_rn(f[s] - __half2float(b)));
            if ((low & 0x7fffu) == 0) low = (uint16_t)((__float_as_uint(f[s]) >> 16 & 0x8000u) | 1u);
            if ((__half_as_ushort(b) & 0x7fffu) == 0) low = 0;
            parts[0][s] = __half_as_ushort(b);
            parts[1][s] = low;
          }
          hi[e] = parts[0][0] | (uint32_t)parts[0][1] << 16;
          lo[e] = parts[1][0] | (uint32_t)parts[1][1] << 16;
        }
      }
      const int byte = lane * E * 2;  // of the row; 128 bytes to a block
      uint8_t *to = sm.q[half] + (byte >> 7) * (PX_M * 128) + place * 128 + ((((byte >> 4) & 7) ^ (place & 7)) << 4) + (byte & 15);
#pragma unroll
      for (int p = 0; p < (SPLIT ? 2 : 1); ++p) {
        const uint32_t(&y)[E / 2] = p ? lo : hi;
        if (E == 4)
          *reinterpret_cast<uint2 *>(to + p * KB * PX_M * 128) = make_uint2(y[0], y[E / 2 - 1]);
        else
          *reinterpret_cast<uint32_t *>(to + p * KB * PX_M * 128) = y[0];
      }
    }
  }
}

template <int KIND, int DH, bool SPLIT>
__global__ void __maxnreg__(PX_REGISTERS)
prefix_kernel(const PrefixArgs a, const __grid_constant__ PrefixMaps maps) {
  using T = PxShape<KIND, DH, SPLIT>;
  using Sm = PxSmem<KIND, DH, SPLIT>;
  constexpr int NS = T::NS;
  extern __shared__ __align__(1024) uint8_t px_raw[];
  Sm &sm = *reinterpret_cast<Sm *>(px_raw);
  const int tid = threadIdx.x, warp = tid >> 5;
  const int heads = a.pages.n_kv_heads, group = a.n_heads / heads, members = 2 * (PX_M / group);
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&sm.full[i], KIND == PG_E4M3 ? PX_CONVERTERS : 1), mbar_init(&sm.empty[i], 2);
    for (int i = 0; i < T::RAW; ++i) mbar_init(&sm.raw_full[i], 1), mbar_init(&sm.raw_empty[i], PX_CONVERTERS);
    for (int i = 0; i < PX_TILES; ++i) mbar_init(&sm.unit[i], 1);
    for (int i = 0; i < 4; ++i)
      mbar_init(&sm.s_full[i / 2][i % 2], 1), mbar_init(&sm.p_full[i / 2][i % 2], PX_SOFT), mbar_init(&sm.pv_done[i / 2][i % 2], 1);
    mbar_init(&sm.fix, 1);
    fence_barrier_init();
    sm.waits = {a.wait_ns, 0};
    asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.k) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.v) : "memory");
  }
  wait_for_previous();
  let_next_begin();  // the rows' own positions need nothing of this kernel
  const PrefixBlock begin = a.blocks[blockIdx.x];
  const long long per = *a.per_block;
  if (begin.place < 0) return;
  const long long v0 = blockIdx.x * per, v1 = v0 + per;  // places behind the list's end are behind its last item
  if (warp == PX_ISSUER) {
    tmem_alloc(&sm.tmem, PX_TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const int part = warp / PX_SOFT, in_part = tid % PX_M;  // of the softmax's threads: the half of the tile, and the row there
  const uint32_t my_tmem = tmem + ((uint32_t)((warp & 3) * 32) << 16) + part * (PX_TMEM / 2), t_o = my_tmem + 2 * PX_N;

  // units of all items so far; of those that had rows in each half of the tile; halves (K or V) in the ring; mended halves
  uint32_t tiles = 0, units[2] = {0, 0}, halves = 0, fixes = 0;
  int g = begin.g, item = begin.item;  // the item is the group's item-th: tile * heads + head
  Group x = group_of(a, g, begin.start, begin.end);
  long long place = begin.place;
  bool lost = false;  // a wait has run out: this item's results, and those of whatever the block still has to do, are NaN
  for (;;) {
    // ---- an item, or this block's part of it: units [u0, u1)
    const int t = item / heads, h = item % heads, first = x.start + t * members;
    const int rows = min(members, x.end - first) * group, rows0 = min(rows, members / 2 * group);
    const int u0 = (int)max(0ll, v0 - place - PX_ITEM_COST), u1 = (int)min((long long)x.units, v1 - place - PX_ITEM_COST);
    const int mine = part < 2 && in_part < (part ? rows - rows0 : rows0) ? in_part + part * rows0 : -1;  // the row, of the tile
    const int64_t slot = (int64_t)first * a.n_heads + h * rows + (int64_t)PX_TILE * blockIdx.x;
    if (u1 > u0 && !lost) {
      int n, issued = 0;
      bool mending = false;
      if (warp == PX_LOADER || warp == PX_LOADER + 1) {
        n = load_item<KIND, DH, SPLIT>(a, maps, sm, x, warp != PX_LOADER, h, u0, u1, tiles, halves, fixes, &mending);
      } else {
        const int lim = mine >= 0 ? min(x.prefix, length_of(a, first + mine / group)) : 0;
        stage_queries<KIND, DH, SPLIT>(a, sm, first, h, group, rows0, rows);
        fence_async_proxy();
        asm volatile("bar.sync 1, %0;" ::"n"(T::THREADS) : "memory");
        const int reach = sm.reach;
        n = max(0, min(u1, (reach + PX_N - 1) / PX_N) - u0);
        if (warp == PX_ISSUER || warp == PX_ISSUER + 1) {
          const int w = warp - PX_ISSUER;
          if (w == 0 || rows > rows0)
            issued = multiply_item<KIND, DH, SPLIT>(sm, tmem + w * (PX_TMEM / 2), w, rows > rows0 ? 2 : 1, n, w ? units[1] : units[0], halves);
        } else if (part >= 2) {
          if constexpr (KIND == PG_E4M3) convert_item<KIND, DH, SPLIT>(sm, tid - 32 * PX_CONVERT, reach, u0, n, halves);
        } else if (part == 0 || rows > rows0) {
          float m = -INFINITY, l = 0.f;
          const bool some = __any_sync(0xffffffffu, mine >= 0);
          const bool ok = soften_item<KIND, DH, SPLIT>(sm, my_tmem, part, in_part, some, lim, u0, n, tiles, part ? units[1] : units[0], &m, &l);
          // the piece: eight dimensions of a row at a time, rows side by side
          float *to = a.prefix + slot * DH + 8 * mine;
          tc_fence_after();
          if (some) {
#pragma unroll 1
            for (int c = 0; c < DH; c += 32) {
              float o[32];
              if (ok && n > 0) {
                tmem_ld32(t_o + c, o);
                tmem_wait_ld();
              } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0.f;
              }
              if (mine >= 0) {
#pragma unroll
                for (int e = 0; e < 32; e += 8) store8(to + (int64_t)(c + e) * rows, &o[e]);
              }
            }
          }
          if (mine >= 0) a.prefix_ml[slot + mine] = make_float2(m - P_BIAS, l);
          tc_fence_before();
        }
      }
      lost = __syncthreads_or(*static_cast<volatile int *>(&sm.waits.failed)) != 0;  // whoever gave up sees its own mark
      tc_fence_after();
      if (lost) {  // no copy may land, and no product be formed, when the block has ended
        if (warp == PX_LOADER || warp == PX_LOADER + 1)
          settle_loads(sm, warp != PX_LOADER, n, halves, fixes, mending);
        else if (warp == PX_ISSUER || warp == PX_ISSUER + 1)
          settle_products(sm, warp - PX_ISSUER, n, warp == PX_ISSUER ? units[0] : units[1], issued);
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
      }
      tiles += n;
      units[0] += n;
      if (rows > rows0) units[1] += n;
      halves += 2 * n;
    }
    if (lost && u1 > u0 && mine >= 0) a.prefix_ml[slot + mine] = make_float2(0.f, __int_as_float(0x7fc00000));
    // ---- the next item
    if (place + PX_ITEM_COST + x.units >= v1) break;
    place += x.units + PX_ITEM_COST;
    if (++item == x.tiles(members) * heads) {
      item = 0;
      int end = x.end;
      do {
        if (++g >= a.n_groups) break;
        const int start = end;
        end = max(start, clamp_start(a, g + 1));
        x = group_of(a, g, start, end);
      } while (x.units == 0);
      if (g >= a.n_groups) break;
    }
  }
  if (warp == PX_ISSUER) tmem_dealloc(tmem, PX_TMEM);
}

// cuTensorMapEncodeTiled of the driver that is there.
decltype(&cuTensorMapEncodeTiled) tensor_map_encode() {
  static const auto encode = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(p);
  }();
  return encode;
}

// The pages as a tensor [page][head][position][dim] of any order of the first three, dimensions by rising stride. Rows of 16
// bits come in boxes of 64 dims, in the layout of an MMA operand; codes as they are.
bool make_map(CUtensorMap *map, int *order, const kie_pages &pg, bool v, int rows) {
  const int64_t *st = v ? pg.v_stride : pg.k_stride;
  const int es = paged_dtype_bytes(pg.dtype);
  struct Dim {
    int what;  // 0 position, 1 head, 2 page
    cuuint64_t size, stride;
  } d[3] = {{0, (cuuint64_t)pg.block_size, (cuuint64_t)st[2] * es},
            {1, (cuuint64_t)pg.n_kv_heads, (cuuint64_t)st[1] * es},
            {2, (cuuint64_t)pg.n_blocks, (cuuint64_t)st[0] * es}};
  for (Dim &x : d)
    if (x.size == 1) x.stride = (cuuint64_t)pg.head_dim * es;  // not stepped over, whatever it is
  std::stable_sort(d, d + 3, [](const Dim &x, const Dim &y) { return x.stride < y.stride; });
  cuuint64_t size[4] = {(cuuint64_t)pg.head_dim}, stride[3];
  cuuint32_t box[4] = {pg.dtype == KIE_E4M3 ? (cuuint32_t)pg.head_dim : 64u}, step[4] = {1, 1, 1, 1};
  *order = d[0].what | d[1].what << 2 | d[2].what << 4;
  for (int i = 0; i < 3; ++i) {
    size[i + 1] = d[i].size;
    stride[i] = d[i].stride;
    box[i + 1] = d[i].what == 0 ? rows : 1;
  }
  const auto encode = tensor_map_encode();
  return encode && encode(map, pg.dtype == KIE_E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4,
                          v ? pg.v : pg.k, size, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          pg.dtype == KIE_E4M3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int KIND, int DH, bool SPLIT>
cudaError_t launch(const PrefixArgs &a, int dev, int sms, cudaStream_t stream) {
  const int bs = a.pages.block_size;
  PrefixMaps maps;
  maps.rows = bs % 64 == 0 ? 64 : bs % 32 == 0 ? 32 : 16;  // a box lies in one page
  if (!make_map(&maps.k, &maps.order[0], a.pages, false, maps.rows) || !make_map(&maps.v, &maps.order[1], a.pages, true, maps.rows))
    return cudaErrorInvalidPitchValue;
  static std::atomic<uint64_t> ready{0};  // devices whose limit of dynamic shared memory is raised
  const int smem = (int)sizeof(PxSmem<KIND, DH, SPLIT>);
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (!bit || !(ready.load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(prefix_kernel<KIND, DH, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_after_previous(prefix_kernel<KIND, DH, SPLIT>, sms, PxShape<KIND, DH, SPLIT>::THREADS, smem, stream, a, maps);
}

template <int DH>
cudaError_t launch_dh(const PrefixArgs &a, int dev, int sms, cudaStream_t stream) {
  const bool wide = a.q_dtype == KIE_F32;
  if (a.pages.dtype == KIE_BF16) return launch<PG_BF16, DH, false>(a, dev, sms, stream);
  if (a.pages.dtype == KIE_E4M3)
    return wide ? launch<PG_E4M3, DH, true>(a, dev, sms, stream) : launch<PG_E4M3, DH, false>(a, dev, sms, stream);
  return wide ? launch<PG_F16, DH, true>(a, dev, sms, stream) : launch<PG_F16, DH, false>(a, dev, sms, stream);
}

// ---- the join ------------------------------------------------------------------------------------------------

// The pieces of a query head, its own positions' first, then the prefix's in their order: a thread has four dimensions.
constexpr int PJ_THREADS = 128;
template <int DH>
__global__ void __launch_bounds__(PJ_THREADS) join_kernel(const PrefixArgs a) {
  begin_after_previous();
  constexpr int LANES = DH / 4;
  const int64_t at = ((int64_t)blockIdx.x * PJ_THREADS + threadIdx.x) / LANES;  // row * heads + head
  if (at >= (int64_t)a.n_seqs * a.n_heads) return;
  const int d = threadIdx.x % LANES * 4, b = (int)(at / a.n_heads), head = (int)(at % a.n_heads);
  const int group = a.n_heads / a.pages.n_kv_heads, h = head / group;
  const PrefixRow row = a.rows[b];
  const long long per = *a.per_block;
  float4 acc = __ldcg(reinterpret_cast<const float4 *>(a.own + at * DH + d));
  const float2 own = __ldcg(a.own_ml + at);
  float M = own.x, L = own.y;
  if (row.lo > 0) {
    const long long place = row.place + (long long)h * (row.units + PX_ITEM_COST) + PX_ITEM_COST;
    const auto block_of = [&](long long v) { return (int)((v | per) >> 32 ? v / per : (unsigned)v / (unsigned)per); };
    const int first = block_of(place), n = block_of(place + row.units - 1) - first + 1;
    const int64_t slot = row.slot + (int64_t)h * row.rows + (int64_t)PX_TILE * first;
    const int r = row.local + head - h * group;
    const float *o = a.prefix + slot * DH + (int64_t)(d >> 3) * row.rows * 8 + r * 8 + (d & 7);
    const float2 *ml = a.prefix_ml + slot + r;
    constexpr int BATCH = 8;  // 4 and 20 take 1 and 0.5 us more for 4 rows, 0.6 and 6 for 256 rows
    for (int i0 = 0; i0 < n; i0 += BATCH) {
      float2 w[BATCH];
      float4 y[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const int64_t i = min(i0 + k, n - 1);
        w[k] = __ldcg(ml + PX_TILE * i);
        y[k] = __ldcg(reinterpret_cast<const float4 *>(o + PX_TILE * DH * i));
      }
      float mn = M;
#pragma unroll
      for (int k = 0; k < BATCH; ++k)
        if (i0 + k < n) mn = fmaxf(mn, w[k].x);
      const float ref = mn == -INFINITY ? 0.f : mn, f0 = ex2(M - ref);
      L *= f0, acc.x *= f0, acc.y *= f0, acc.z *= f0, acc.w *= f0;
#pragma unroll
      for (int k = 0; k < BATCH; ++k)
        if (i0 + k < n) {
          const float f = ex2(w[k].x - ref);
          L = fmaf(w[k].y, f, L);
          acc.x = fmaf(y[k].x, f, acc.x), acc.y = fmaf(y[k].y, f, acc.y);
          acc.z = fmaf(y[k].z, f, acc.z), acc.w = fmaf(y[k].w, f, acc.w);
        }
      M = mn;
    }
  }
  const float inv = L == 0.f ? 0.f : __fdividef(1.f, L);
  const float v[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
  const int64_t to = b * a.out_stride[0] + head * a.out_stride[1] + d;
  const int size = paged_dtype_bytes(a.q_dtype);
  const bool vec = ((uintptr_t)a.out | (uintptr_t)(a.out_stride[0] * size) | (uintptr_t)(a.out_stride[1] * size)) % (4 * size) == 0;
  if (!vec) {
#pragma unroll
    for (int e = 0; e < 4; ++e) paged_store(a.out, to + e, a.q_dtype, v[e]);
  } else if (a.q_dtype == KIE_F32) {
    *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + to) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + to) =
        make_uint2(pack2(v[0], v[1], a.q_dtype), pack2(v[2], v[3], a.q_dtype));
  }
  if (d == 0 && a.lse) a.lse[at] = L == 0.f ? -INFINITY : (M + lg2(L)) * 0.6931471805599453f;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// The workspace: that of the rows' own positions, then what the launches pass on.
struct Parts {
  size_t per_block, blocks, row_lo, rows, prefix_ml, own_ml, own, prefix, all;
  Parts(int n_seqs, int n_heads, int n_kv_heads, int head_dim, int sms) {
    const size_t heads = (size_t)n_seqs * n_heads, slots = heads + (size_t)PX_TILE * sms;
    per_block = up256(kie_paged_attention_workspace_bytes(n_heads, n_kv_heads, head_dim, sms));
    blocks = per_block + 256;
    row_lo = up256(blocks + sms * sizeof(PrefixBlock));
    rows = up256(row_lo + (size_t)n_seqs * 4);
    prefix_ml = up256(rows + (size_t)n_seqs * sizeof(PrefixRow));
    own_ml = up256(prefix_ml + slots * 8);
    own = up256(own_ml + heads * 8);
    prefix = up256(own + heads * head_dim * 4);
    all = prefix + slots * head_dim * 4;
  }
};

template <int DH>
cudaError_t launch_all(const PrefixArgs &a, int dev, int sms, cudaStream_t stream) {
  const int plan_blocks = std::max(1, std::min(sms / 8, (a.n_seqs + PL_THREADS - 1) / PL_THREADS));
  static std::atomic<uint64_t> ready{0};  // devices whose limit of dynamic shared memory is raised
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  cudaError_t e = cudaSuccess;
  if (!bit || !(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (KIE_PAGED_MAX_GROUPS + 1) * 12);
    if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
  }
  if (e == cudaSuccess)
    e = launch_after_previous(plan_kernel, plan_blocks, PL_THREADS, (size_t)(a.n_groups + 1) * 12, stream, a, sms);
  if (e == cudaSuccess) e = launch_dh<DH>(a, dev, sms, stream);
  if (e == cudaSuccess) e = kie_launch_paged_own(a, dev, sms, stream);
  const int64_t threads = (int64_t)a.n_seqs * a.n_heads * (DH / 4);
  return e != cudaSuccess ? e
                          : launch_after_previous(join_kernel<DH>, (unsigned)((threads + PJ_THREADS - 1) / PJ_THREADS), PJ_THREADS, 0,
                                                  stream, a);
}

}  // namespace
}  // namespace kie

size_t kie_paged_prefix_workspace_bytes(int n_seqs, int n_heads, int n_kv_heads, int head_dim, int sms) {
  return kie::Parts(n_seqs, n_heads, n_kv_heads, head_dim, sms).all;
}

cudaError_t kie_launch_paged_prefix(const kie_paged_prefix_attention_args &args, unsigned long long wait_ns, int stop_block,
                                    int stop_half, int dev, int sms, cudaStream_t stream) {
  kie::PrefixArgs a;
  static_cast<kie_paged_attention_args &>(a) = kie::rows_in_lens(args.a);
  a.group_start = args.group_start;
  a.prefix_lens = args.prefix_lens;
  a.n_groups = args.n_groups;
  const kie::Parts p(a.n_seqs, a.n_heads, a.pages.n_kv_heads, a.pages.head_dim, sms);
  uint8_t *at = static_cast<uint8_t *>(a.workspace);
  a.per_block = reinterpret_cast<long long *>(at + p.per_block);
  a.blocks = reinterpret_cast<kie::PrefixBlock *>(at + p.blocks);
  a.row_lo = reinterpret_cast<int32_t *>(at + p.row_lo);
  a.rows = reinterpret_cast<kie::PrefixRow *>(at + p.rows);
  a.prefix_ml = reinterpret_cast<float2 *>(at + p.prefix_ml);
  a.own_ml = reinterpret_cast<float2 *>(at + p.own_ml);
  a.own = reinterpret_cast<float *>(at + p.own);
  a.prefix = reinterpret_cast<float *>(at + p.prefix);
  a.wait_ns = wait_ns;
  a.stop_block = stop_block;
  a.stop_half = stop_half;
  return a.pages.head_dim == 64 ? kie::launch_all<64>(a, dev, sms, stream) : kie::launch_all<128>(a, dev, sms, stream);
}
