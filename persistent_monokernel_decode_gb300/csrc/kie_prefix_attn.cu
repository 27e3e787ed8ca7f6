// The shared part of kie_paged_prefix_attention: attention of the rows of each group over the positions of their prefix.
// The rows' own positions, and the sum of both, are kie_paged_attn.cu's.
//
// For one KV head, the query heads of a group's rows are the rows of a matrix: with 5 query heads a KV head, 25 sequences
// fill the 128 rows of a tensor-core tile, so that what kie_paged_attn.cu has to do as matrix-vector products becomes
// S = Q K^T and O += P V on tcgen05. Work is a list of items (group, tile of its rows, KV head), each a row of units of 64
// positions; every block takes an equal run of the list and writes a piece (O, reference, sum of weights) for each item
// that it has part in. The kernel of the rows' own positions joins the pieces where it finishes a row: hundreds of blocks
// there read them side by side.
//
// In a block four warps load K and V tiles into a ring (cp.async, or through registers where E4M3 codes become fp16), one
// thread issues the MMAs, and four warps hold the softmax: thread = row = TMEM lane, so its maxima and sums need no
// shuffles. S is double-buffered in TMEM, so that the scores of the next tile are formed while this one's weights are;
// the weights go back over the scores, as the TMEM operand of the second product. As in kie_paged_attn.cu, the softmax's
// reference stays within 2^8 of the running maximum and O is only rescaled when a weight would pass 2^15, weights and fp32
// queries are two 16-bit parts, and the sum of weights is of the weights before they are rounded.
#include <float.h>

#include <algorithm>
#include <atomic>

#include "kie_device.cuh"
#include "kie_paged.cuh"
#include "kie_tc.cuh"

namespace kie {
namespace {

constexpr int PX_M = 128, PX_N = 64;       // rows of a tile, positions of a unit
constexpr int PX_SOFT = 4, PX_LOAD = 4;    // warps; one more issues the MMAs
constexpr int PX_THREADS = 32 * (PX_SOFT + PX_LOAD + 1);
constexpr int PX_LOADERS = 32 * PX_LOAD;
// Depth of what is kept per unit besides K and V. The loaders are at most NS <= 5 halves ahead of the oldest one in use, so
// at most three units ahead of the one whose weights are formed.
constexpr int PX_TILES = 4;
constexpr uint32_t PX_TMEM = 256;          // columns: S twice, O
constexpr unsigned long long PX_TIMEOUT_NS = 2000000000ull;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float P_BIAS = 7.f, P_STEP = 8.f;  // weights are 2^7 2^(v - reference), below 2^15
constexpr float MIN_LOG2_SCALE = -60.f, MAX_LOG2_SCALE = 127.f;  // of E4M3 values, as in kie_paged_attn.cu

enum { PG_F16 = 0, PG_BF16 = 1, PG_E4M3 = 2 };

template <int KIND, int DH, bool SPLIT>
struct PxShape {
  static constexpr int Q_BYTES = PX_M * DH * 2 * (SPLIT ? 2 : 1), SLOT = PX_N * DH * 2;
  // Two blocks fit an SM but where fp32 queries meet E4M3 pages of 128, whose scales are 1 KB too many
  static constexpr int BLOCKS = SPLIT && KIND == PG_E4M3 && DH == 128 ? 1 : 2;
  static constexpr int NS = DH == 64 || BLOCKS == 1 ? 5 : SPLIT ? 3 : KIND == PG_E4M3 ? 4 : 5;  // ring slots
};

template <int KIND, int DH, bool SPLIT>
struct PxSmem {
  using T = PxShape<KIND, DH, SPLIT>;
  uint8_t q[T::Q_BYTES];         // [part][64-dim block][row][128 B], 16-byte chunks swizzled by the row
  uint8_t ring[T::NS][T::SLOT];  // [64-dim block][position][128 B], the same
  float scale[KIND == PG_E4M3 ? PX_TILES : 1][3][KIND == PG_E4M3 ? PX_N : 1];  // of K, of V, log2 of V's
  uint32_t live[PX_TILES];       // bit i: positions 16 i .. 16 i + 15 lie on a page
  float rs[PX_M];                // score scale of a row, in log2 units
  uint64_t full[T::NS], empty[T::NS], unit[PX_TILES], s_full[2], p_full[2], pv_done;
  unsigned long long best;       // of the group's rows: reach, and the first row that has it
  uint32_t tmem;
  int failed;
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

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Waits for a phase of a barrier of this block, two seconds at most; false if that ran out, here or in another wait.
__device__ __forceinline__ bool px_wait(uint64_t *bar, uint32_t parity, int *failed) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (int spins = 1;; ++spins) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((spins & 63) == 0) {
      if (*static_cast<volatile int *>(failed)) return false;
      if (globaltimer() - t0 > PX_TIMEOUT_NS) {
        *static_cast<volatile int *>(failed) = 1;
        return false;
      }
    }
  }
}

// The same for a whole warp at once.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int *failed) {
  return __all_sync(0xffffffffu, px_wait(bar, parity, failed)) != 0;
}

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

// Sums over the block in thread order: v becomes the sum of the threads' before this one, *all of all.
__device__ __forceinline__ long long sum_before(long long v, long long *all) {
  __shared__ long long s_warp[PX_THREADS / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long up = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += x;
  }
  if (lane == 31) s_warp[warp] = up;
  __syncthreads();
  long long before = up - v, sum = 0;
  for (int w = 0; w < PX_THREADS / 32; ++w) {
    if (w < warp) before += s_warp[w];
    sum += s_warp[w];
  }
  __syncthreads();
  *all = sum;
  return before;
}

// ---- the three roles of a block, for units u0 .. u0 + n - 1 of an item -------------------------------------------
// `tiles` and `halves` count the units, and the halves of them in the ring, of the items before. The halves' order is that
// of their use: K0, K1, V0, K2, V1, .., V(n - 1).

// Slot of a half, and the parity of its round through the ring.
template <int NS>
struct Half {
  uint32_t slot, round;
  __device__ __forceinline__ explicit Half(uint32_t i) : slot(i % NS), round(i / NS & 1u) {}
};

template <int KIND, int DH, bool SPLIT>
__device__ __forceinline__ void load_item(const PrefixArgs &a, PxSmem<KIND, DH, SPLIT> &sm, int lt, int h, int source, int reach,
                                          int u0, int n, uint32_t tiles, uint32_t halves) {
  using T = PxShape<KIND, DH, SPLIT>;
  constexpr bool CODES = KIND == PG_E4M3;
  constexpr int NS = T::NS, ES = CODES ? 1 : 2, CH = DH * ES / 16;      // 16-byte chunks of a cache row
  constexpr int STEP = PX_LOADERS / CH, LOADS = PX_N / STEP;            // rows that the loaders take at once, and how often
  constexpr int LAG = NS > 3 ? 2 : 1;  // halves whose copies are on their way when the next one's begin
  const int warp = lt >> 5, lane = lt & 31, row0 = lt / CH, chunk = lt % CH;
  const int *pages = a.block_table + sequence_of(a, source) * a.table_stride;
  const unsigned bs = a.pages.block_size;
  const uint8_t *base[2] = {static_cast<const uint8_t *>(a.pages.k) + (int64_t)h * a.pages.k_stride[1] * ES + 16 * chunk,
                            static_cast<const uint8_t *>(a.pages.v) + (int64_t)h * a.pages.v_stride[1] * ES + 16 * chunk};
  const int64_t page_step[2] = {a.pages.k_stride[0] * ES, a.pages.v_stride[0] * ES};
  const int64_t row_step[2] = {a.pages.k_stride[2] * ES, a.pages.v_stride[2] * ES};

  // lane: page and place in it of 16 positions, of eight units from `batch` on and of the eight behind them
  int batch = u0, page_a, at_a, page_b, at_b;
  const auto fetch = [&](int unit, int *page, int *at) {
    const int pos = unit * PX_N + 16 * lane;
    const unsigned j = (unsigned)pos / bs;
    *at = pos - (int)(j * bs);
    *page = unit < u0 + n && pos < reach ? pages[j] : -1;
  };
  fetch(u0, &page_a, &at_a);
  fetch(u0 + 8, &page_b, &at_b);
  struct Places {
    int page[4], at[4];
    uint32_t live;
  };
  const auto places = [&](int unit) {  // of a unit's four groups of 16 positions; units come in order
    if (unit >= batch + 8) {
      batch += 8;
      page_a = page_b, at_a = at_b;
      fetch(batch + 8, &page_b, &at_b);
    }
    Places p;
    p.live = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p.page[i] = __shfl_sync(0xffffffffu, page_a, (unit - batch) * 4 + i);
      p.at[i] = __shfl_sync(0xffffffffu, at_a, (unit - batch) * 4 + i);
      if ((unsigned)p.page[i] < (unsigned)a.pages.n_blocks) p.live |= 1u << i;
    }
    return p;
  };
  // Row row0 + i STEP of a unit lies in its group (i STEP + row0) / 16; with rows of 64 codes that depends on the thread.
  const auto source_of = [&](const Places &p, int unit, int i, int v, bool *live) {
    const int row = row0 + i * STEP;
    int page = p.page[(i * STEP) >> 4], at = p.at[(i * STEP) >> 4];
    uint32_t bit = (p.live >> ((i * STEP) >> 4)) & 1u;
    if (STEP > 16 && row0 >= 16) {
      page = p.page[((i * STEP) >> 4) + 1], at = p.at[((i * STEP) >> 4) + 1];
      bit = (p.live >> (((i * STEP) >> 4) + 1)) & 1u;
    }
    *live = bit && unit * PX_N + row < reach;
    return base[v] + (*live ? page * page_step[v] + (at + (row & 15)) * row_step[v] : 0);
  };
  const auto wait_empty = [&](uint32_t half) {
    const Half<NS> x(half);
    return warp_wait(&sm.empty[x.slot], x.round ^ 1u, &sm.failed);
  };
  const auto announce = [&](uint32_t half) {  // this warp's part of it is in place
    fence_async_proxy();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.full[half % NS]);
  };

  uint32_t half = halves;
  if constexpr (!CODES) {
    const uint32_t ring = smem_u32(sm.ring);
    const auto copy = [&](const Places &p, int unit, int v) {
      if (!wait_empty(half)) return false;
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        bool live;
        const uint8_t *src = source_of(p, unit, i, v, &live);
        const int row = row0 + i * STEP;
        cp_async16(ring + (half % NS) * T::SLOT + (chunk >> 3) * (PX_N * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4), src, live);
      }
      cp_commit();
      if (half - halves >= LAG) {
        cp_wait<LAG>();
        announce(half - LAG);
      }
      ++half;
      return true;
    };
    Places before = {};
    bool ok = true;
    for (int u = 0; u <= n && ok; ++u) {
      Places p = {};
      if (u < n) {
        p = places(u0 + u);
        ok = copy(p, u0 + u, 0);
        if (warp == 0 && lane == 0) {
          sm.live[(tiles + u) % PX_TILES] = p.live;
          mbar_arrive(&sm.unit[(tiles + u) % PX_TILES]);
        }
      }
      if (u > 0) ok = ok && copy(before, u0 + u - 1, 1);
      before = p;
    }
    cp_wait<0>();
    if (ok)
      for (uint32_t i = max(halves, half - min(half, (uint32_t)LAG)); i < half; ++i) announce(i);
  } else {
    // E4M3: codes through registers, on their way while the half before them is converted
    uint4 code[2][LOADS];
    float ks = 0.f, vs = 0.f;  // scales of position lt of the unit, for the first PX_N loaders
    const auto request = [&](const Places &p, int unit, int v) {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        bool live;
        const uint8_t *src = source_of(p, unit, i, v, &live);
        code[v][i] = live ? *reinterpret_cast<const uint4 *>(src) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    const auto request_scales = [&](const Places &p, int unit) {
      if (lt >= PX_N) return;
      int page = p.page[0], at = p.at[0];
#pragma unroll
      for (int i = 1; i < 4; ++i)
        if (lt >> 4 == i) page = p.page[i], at = p.at[i];
      ks = vs = 0.f;
      if ((p.live >> (lt >> 4) & 1u) && unit * PX_N + lt < reach) {
        const int off = at + (lt & 15);
        ks = a.pages.k_scale[page * a.pages.k_scale_stride[0] + h * a.pages.k_scale_stride[1] + off * a.pages.k_scale_stride[2]];
        vs = a.pages.v_scale[page * a.pages.v_scale_stride[0] + h * a.pages.v_scale_stride[1] + off * a.pages.v_scale_stride[2]];
      }
    };
    const auto store = [&](int v) {
      if (!wait_empty(half)) return false;
      uint8_t *slot = sm.ring[half % NS];
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int row = row0 + i * STEP, c = 2 * (chunk & 3);
        uint8_t *to = slot + (chunk >> 2) * (PX_N * 128) + row * 128;
        const uint4 w = code[v][i];
        *reinterpret_cast<uint4 *>(to + ((c ^ (row & 7)) << 4)) =
            make_uint4(e4m3x2(w.x & 0xffffu), e4m3x2(w.x >> 16), e4m3x2(w.y & 0xffffu), e4m3x2(w.y >> 16));
        *reinterpret_cast<uint4 *>(to + (((c + 1) ^ (row & 7)) << 4)) =
            make_uint4(e4m3x2(w.z & 0xffffu), e4m3x2(w.z >> 16), e4m3x2(w.w & 0xffffu), e4m3x2(w.w >> 16));
      }
      announce(half);
      ++half;
      return true;
    };
    Places p = {};
    if (n > 0) {
      p = places(u0);
      request(p, u0, 0);
      request_scales(p, u0);
    }
    bool ok = true;
    for (int u = 0; u <= n && ok; ++u) {
      const Places mine = p;
      if (u < n) {
        ok = store(0);
        const uint32_t i = (tiles + u) % PX_TILES;
        if (ok && lt < PX_N) {
          sm.scale[i][0][lt] = ks;
          sm.scale[i][CODES ? 1 : 0][lt] = vs;
          sm.scale[i][CODES ? 2 : 0][lt] = log2_scale(vs);
          if (lt == 0) sm.live[i] = mine.live;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.unit[i]);
        }
        if (u + 1 < n) {
          p = places(u0 + u + 1);
          request(p, u0 + u + 1, 0);
          request_scales(p, u0 + u + 1);
        }
      }
      if (u > 0) ok = ok && store(1);
      if (u < n) request(mine, u0 + u, 1);
    }
  }
}

// One thread.
template <int KIND, int DH, bool SPLIT>
__device__ __forceinline__ void multiply_item(PxSmem<KIND, DH, SPLIT> &sm, uint32_t tmem, int n, uint32_t tiles, uint32_t halves) {
  constexpr int NS = PxShape<KIND, DH, SPLIT>::NS, KB = DH / 64;
  constexpr uint32_t S_DESC = px_idesc(PX_N, KIND == PG_BF16, false), O_DESC = px_idesc(DH, KIND == PG_BF16, true);
  const uint32_t q = smem_u32(sm.q);
  uint32_t half = halves;
  for (int j = 0; j <= n; ++j) {
    if (j < n) {  // S = Q K^T
      const uint32_t tile = tiles + j, to = tmem + (tile & 1u) * PX_N;
      const Half<NS> x(half);
      if (!px_wait(&sm.full[x.slot], x.round, &sm.failed)) return;
      if (j >= 2 && !px_wait(&sm.pv_done, tile & 1u, &sm.failed)) return;  // unit j - 2 is done with the buffer
      tc_fence_after();
      const uint32_t k = smem_u32(sm.ring[x.slot]);
#pragma unroll
      for (int p = 0; p < (SPLIT ? 2 : 1); ++p)
#pragma unroll
        for (int s = 0; s < DH / 16; ++s)
          tc_mma(to, px_desc(q + (p * KB + s / 4) * (PX_M * 128) + s % 4 * 32, 16), px_desc(k + s / 4 * (PX_N * 128) + s % 4 * 32, 16),
                 S_DESC, p || s ? 1u : 0u);
      tc_commit(&sm.empty[x.slot]);
      tc_commit(&sm.s_full[tile & 1u]);
      ++half;
    }
    if (j > 0) {  // O += P V
      const uint32_t tile = tiles + j - 1, p = tmem + (tile & 1u) * PX_N;
      const Half<NS> x(half);
      if (!px_wait(&sm.p_full[tile & 1u], tile >> 1 & 1u, &sm.failed)) return;
      if (!px_wait(&sm.full[x.slot], x.round, &sm.failed)) return;
      tc_fence_after();
      const uint32_t v = smem_u32(sm.ring[x.slot]);
#pragma unroll
      for (int s = 0; s < PX_N / 16; ++s)
#pragma unroll
        for (int part = 0; part < 2; ++part)
          tc_mma_ts(tmem + 2 * PX_N, p + s * 16 + part * 8, px_desc(v + s * 2048, PX_N * 128), O_DESC, j > 1 || s || part ? 1u : 0u);
      tc_commit(&sm.empty[x.slot]);
      tc_commit(&sm.pv_done);
      ++half;
    }
  }
}

// A thread is the row `row`, which attends to positions below lim; `rows`: whether the warp has any row at all. m, l: the
// reference (log2 units) and the sum of weights. O is complete on return; false if a wait ran out.
template <int KIND, int DH, bool SPLIT>
__device__ __forceinline__ bool soften_item(PxSmem<KIND, DH, SPLIT> &sm, uint32_t tmem, int row, bool rows, int lim, int u0, int n,
                                            uint32_t tiles, float *m_out, float *l_out) {
  const float rs = sm.rs[row];
  const uint32_t t_o = tmem + 2 * PX_N;
  const int lane = row & 31;
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < n; ++j) {
    const uint32_t tile = tiles + j, t_s = tmem + (tile & 1u) * PX_N;
    const int left = lim - (u0 + j) * PX_N;  // positions of the unit that the row attends to
    if (!warp_wait(&sm.unit[tile % PX_TILES], tile / PX_TILES & 1u, &sm.failed)) return false;
    if (!warp_wait(&sm.s_full[tile & 1u], tile >> 1 & 1u, &sm.failed)) return false;
    tc_fence_after();
    if (rows) {
      const uint32_t live = sm.live[tile % PX_TILES];
      float s[2][32];
      tmem_ld32(t_s, s[0]);
      tmem_ld32(t_s + 32, s[1]);
      tmem_wait_ld();
      if (KIND == PG_E4M3) {
        const float *ks = sm.scale[KIND == PG_E4M3 ? tile % PX_TILES : 0][0];
#pragma unroll
        for (int e = 0; e < PX_N; ++e) s[e / 32][e % 32] *= ks[KIND == PG_E4M3 ? e : 0];
      }
      if (!__all_sync(0xffffffffu, left >= PX_N && live == 15u)) {
#pragma unroll
        for (int e = 0; e < PX_N; ++e)
          if (e >= left || !(live >> (e / 16) & 1u)) s[e / 32][e % 32] = -INFINITY;
      }
      float top = -INFINITY;
      if (KIND == PG_E4M3) {
        const float *ls = sm.scale[KIND == PG_E4M3 ? tile % PX_TILES : 0][KIND == PG_E4M3 ? 2 : 0];
#pragma unroll
        for (int e = 0; e < PX_N; ++e) top = fmaxf(top, fmaf(s[e / 32][e % 32], rs, ls[KIND == PG_E4M3 ? e : 0]));
      } else {
#pragma unroll
        for (int e = 0; e < PX_N; ++e) top = fmaxf(top, s[e / 32][e % 32]);
        top *= rs;
      }
      const bool far = top > m + P_STEP;
      if (__any_sync(0xffffffffu, far)) {
        const float mn = far ? top : m, f = far && m != -INFINITY ? ex2(m - mn) : 1.f;
        m = mn;
        l *= f;
        if (j > 0) {
          if (!warp_wait(&sm.pv_done, (tile - 1) & 1u, &sm.failed)) return false;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < DH; c += 32) {
            float o[32];
            tmem_ld32(t_o + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; k += 16) {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[k + e] * f);
              tmem_st16(t_o + c + k, w);
            }
          }
        }
      }
      const float bias = P_BIAS - (m == -INFINITY ? 0.f : m);
      float part[2] = {0.f, 0.f};
#pragma unroll
      for (int c = 0; c < PX_N; c += 16) {  // the weights of 16 positions: eight columns of first parts, eight of second ones
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          float y[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int at = c + e + k;
            y[k] = ex2(fmaf(s[at / 32][at % 32], rs, bias));
            part[k] += y[k];
            if (KIND == PG_E4M3) y[k] *= sm.scale[KIND == PG_E4M3 ? tile % PX_TILES : 0][KIND == PG_E4M3 ? 1 : 0][KIND == PG_E4M3 ? at : 0];
          }
          const uint32_t hi = pack16<KIND>(y[0], y[1]);
          const float2 b = unpack16<KIND>(hi);
          w[e / 2] = hi;
          w[8 + e / 2] = pack16<KIND>(y[0] - b.x, y[1] - b.y);
        }
        tmem_st16(t_s + c, w);
      }
      l += part[0] + part[1];
      tmem_wait_st();
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.p_full[tile & 1u]);
  }
  // the last two: a barrier tells a phase from the one before it only, and so far no more than unit n - 3 is known to be done
  if (n > 1 && !warp_wait(&sm.pv_done, (tiles + n) & 1u, &sm.failed)) return false;
  if (n > 0 && !warp_wait(&sm.pv_done, (tiles + n - 1) & 1u, &sm.failed)) return false;
  *m_out = m;
  *l_out = l;
  return true;
}

// ---- the kernel ----------------------------------------------------------------------------------------------

template <int KIND, int DH, bool SPLIT>
__global__ void __launch_bounds__(PX_THREADS, PxShape<KIND, DH, SPLIT>::BLOCKS) prefix_kernel(const PrefixArgs a) {
  using T = PxShape<KIND, DH, SPLIT>;
  using Sm = PxSmem<KIND, DH, SPLIT>;
  constexpr int NS = T::NS, KB = DH / 64;  // 64-dim blocks of a row
  extern __shared__ __align__(1024) uint8_t px_raw[];
  Sm &sm = *reinterpret_cast<Sm *>(px_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int heads = a.pages.n_kv_heads, group = a.n_heads / heads, members = PX_M / group;
  wait_for_previous();

  // ---- where this block's run begins, and (each row by one block) what the join has to know of a row
  __shared__ long long s_place;  // of the item, in the list
  __shared__ int s_g, s_edge[2];
  long long total, per, v0;
  {
    int *starts = reinterpret_cast<int *>(px_raw);  // [n_groups + 1]; the ring and queries are not in use yet
    long long *base = reinterpret_cast<long long *>(px_raw + (KIE_PAGED_MAX_GROUPS + 4) * 4);
    const int G = a.n_groups;
    for (int g = tid; g <= G; g += PX_THREADS) starts[g] = clamp_start(a, g);
    __syncthreads();
    bool falls = false;
    for (int g = tid; g < G; g += PX_THREADS) falls |= starts[g + 1] < starts[g];
    if (__syncthreads_or(falls)) {
      if (tid == 0)
        for (int g = 0; g < G; ++g) starts[g + 1] = max(starts[g + 1], starts[g]);
      __syncthreads();
    }
    const int each = (G + PX_THREADS - 1) / PX_THREADS, g0 = min(tid * each, G), g1 = min(g0 + each, G);
    long long mine = 0;
    for (int g = g0; g < g1; ++g) mine += places_of(a, group_of(a, g, starts[g], starts[g + 1]), members);
    long long at = sum_before(mine, &total);
    per = max((total + gridDim.x - 1) / gridDim.x, (long long)PX_MIN_RUN);
    v0 = blockIdx.x * per;
    for (int g = g0; g < g1; ++g) {
      const long long n = places_of(a, group_of(a, g, starts[g], starts[g + 1]), members);
      base[g] = at;
      if (v0 >= at && v0 < at + n) s_g = g, s_place = at, s_edge[0] = starts[g], s_edge[1] = starts[g + 1];
      at += n;
    }
    __syncthreads();
    for (int b = blockIdx.x * PX_THREADS + tid; b < a.n_seqs; b += gridDim.x * PX_THREADS) {
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
    if (blockIdx.x == 0 && tid == 0) *a.per_block = per;
    __syncthreads();
  }
  if (v0 >= total) return;
  const long long v1 = min(v0 + per, total);

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&sm.full[i], PX_LOAD), mbar_init(&sm.empty[i], 1);
    for (int i = 0; i < PX_TILES; ++i) mbar_init(&sm.unit[i], KIND == PG_E4M3 ? PX_N / 32 : 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sm.s_full[i], 1), mbar_init(&sm.p_full[i], PX_SOFT);
    mbar_init(&sm.pv_done, 1);
    fence_barrier_init();
    sm.failed = 0;
  }
  if (warp == 0) {
    tmem_alloc(&sm.tmem, PX_TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem, t_o = tmem + 2 * PX_N;
  const uint32_t my_lanes = (uint32_t)((warp & 3) * 32) << 16;

  uint32_t tiles = 0, halves = 0;  // units of all items so far; halves of them (K or V) in the ring
  int g = s_g;
  Group x = group_of(a, g, s_edge[0], s_edge[1]);
  const bool bf16_q = a.q_dtype == KIE_BF16;
  const bool q_vec = [&] {
    const int size = paged_dtype_bytes(a.q_dtype);
    return ((uintptr_t)a.q | (uintptr_t)(a.q_stride[0] * size) | (uintptr_t)(a.q_stride[1] * size)) % (DH / 32 * size) == 0;
  }();

  long long place = s_place;
  int item;  // of the group: tile * heads + head
  {
    const int span = x.units + PX_ITEM_COST;
    item = (int)((v0 - place) / span);
    place += (long long)item * span;
  }
  for (;;) {
    // ---- an item, or this block's part of it: units [u0, u1)
    const int t = item / heads, h = item % heads, first = x.start + t * members;
    const int rows = min(members, x.end - first) * group;
    const int u0 = (int)max(0ll, v0 - place - PX_ITEM_COST), u1 = (int)min((long long)x.units, v1 - place - PX_ITEM_COST);
    if (u1 > u0) {
      // the group's longest row (the first of them): its pages are read
      if (tid == 0) sm.best = 0;
      __syncthreads();
      unsigned long long mine = 0;
      for (int b = x.start + tid; b < x.end; b += PX_THREADS)
        mine = max(mine, (unsigned long long)min(x.prefix, length_of(a, b)) << 32 | (uint32_t)~b);
#pragma unroll
      for (int o = 16; o; o >>= 1) mine = max(mine, __shfl_xor_sync(0xffffffffu, mine, o));
      if (lane == 0) atomicMax(&sm.best, mine);
      // queries: a warp takes a row at a time, a lane DH / 32 neighbouring elements of it
      for (int r = warp; r < PX_M; r += PX_THREADS / 32) {
        constexpr int E = DH / 32;
        float q[E];
        const int64_t at = (int64_t)(first + r / group) * a.q_stride[0] + (int64_t)(h * group + r % group) * a.q_stride[1] + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) q[e] = 0.f;
        if (r < rows) {
          if (a.q_dtype == KIE_F32) {
            const float *p = static_cast<const float *>(a.q) + at;
            if (q_vec && E == 4) {
              const float4 w = *reinterpret_cast<const float4 *>(p);
              q[0] = w.x, q[1] = w.y, q[E - 2] = w.z, q[E - 1] = w.w;
            } else {
#pragma unroll
              for (int e = 0; e < E; ++e) q[e] = p[e];
            }
          } else {
            const uint16_t *p = static_cast<const uint16_t *>(a.q) + at;
            uint32_t w[E / 2];
            if (q_vec && E == 4) {
              const uint2 y = *reinterpret_cast<const uint2 *>(p);
              w[0] = y.x, w[E / 2 - 1] = y.y;
            } else if (q_vec) {
              w[0] = *reinterpret_cast<const uint32_t *>(p);
            } else {
#pragma unroll
              for (int e = 0; e < E / 2; ++e) w[e] = p[2 * e] | (uint32_t)p[2 * e + 1] << 16;
            }
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
              const float2 f = bf16_q ? unpack16<PG_BF16>(w[e]) : unpack16<PG_F16>(w[e]);
              q[2 * e] = f.x, q[2 * e + 1] = f.y;
            }
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
          rs *= __int_as_float((127 - e2) << 23);
        }
        if (lane == 0) sm.rs[r] = rs;
        uint32_t hi[E / 2], lo[E / 2];
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          const float u = q[2 * e] * up, w = q[2 * e + 1] * up;
          if (!SPLIT) {
            hi[e] = pack16<KIND>(u, w);
            lo[e] = 0u;
          } else {
            // The first part is cut off, not rounded, and a remainder of 0 becomes the least there is: both parts then
            // have the sign of the query, and an infinity in K gives the score that it should instead of NaN.
            const float f[2] = {u, w};
            uint16_t parts[2][2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const __half b = __float2half_rz(f[k]);
              const float rest = f[k] - __half2float(b);
              __half c = __float2half_rn(rest);
              const uint16_t sign = (__float_as_uint(f[k]) >> 16) & 0x8000u;
              uint16_t low = __half_as_ushort(c);
              if ((low & 0x7fffu) == 0) low = sign | 1u;
              if ((__half_as_ushort(b) & 0x7fffu) == 0) low = 0;
              parts[0][k] = __half_as_ushort(b);
              parts[1][k] = low;
            }
            hi[e] = parts[0][0] | (uint32_t)parts[0][1] << 16;
            lo[e] = parts[1][0] | (uint32_t)parts[1][1] << 16;
          }
        }
        const int byte = lane * E * 2;  // of the row; 128 bytes to a block
        uint8_t *to = sm.q + (byte >> 7) * (PX_M * 128) + r * 128 + ((((byte >> 4) & 7) ^ (r & 7)) << 4) + (byte & 15);
#pragma unroll
        for (int p = 0; p < (SPLIT ? 2 : 1); ++p) {
          const uint32_t(&w)[E / 2] = p ? lo : hi;
          if (E == 4)
            *reinterpret_cast<uint2 *>(to + p * KB * PX_M * 128) = make_uint2(w[0], w[E / 2 - 1]);
          else
            *reinterpret_cast<uint32_t *>(to + p * KB * PX_M * 128) = w[0];
        }
      }
      fence_async_proxy();
      __syncthreads();
      const int reach = (int)(sm.best >> 32), source = (int)~(uint32_t)sm.best;
      const int u_end = min(u1, (reach + PX_N - 1) / PX_N), n = max(0, u_end - u0);  // units with positions

      if (warp >= PX_SOFT && warp < PX_SOFT + PX_LOAD) {
        load_item<KIND, DH, SPLIT>(a, sm, tid - 32 * PX_SOFT, h, source, reach, u0, n, tiles, halves);
      } else if (warp == PX_SOFT + PX_LOAD) {
        if (lane == 0) multiply_item<KIND, DH, SPLIT>(sm, tmem, n, tiles, halves);
        __syncwarp();
      } else {
        const int lim = tid < rows ? min(x.prefix, length_of(a, first + tid / group)) : 0;
        float m = -INFINITY, l = 0.f;
        const bool ok = soften_item<KIND, DH, SPLIT>(sm, tmem + my_lanes, tid, warp * 32 < rows, lim, u0, n, tiles, &m, &l);
        // the piece: eight dimensions of a row at a time, rows side by side
        const int64_t slot = (int64_t)first * a.n_heads + h * rows + (int64_t)PX_M * blockIdx.x;
        float *to = a.prefix + slot * DH + 8 * tid;
        if (ok && n > 0) tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < DH; c += 32) {
          float o[32];
          if (ok && n > 0) {
            tmem_ld32(t_o + my_lanes + c, o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0.f;
          }
          if (tid < rows) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              float4 *p = reinterpret_cast<float4 *>(to + (int64_t)(c + e) * rows);
              p[0] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
              p[1] = make_float4(o[e + 4], o[e + 5], o[e + 6], o[e + 7]);
            }
          }
        }
        // a wait that ran out shows as NaN in every result that it concerns
        if (tid < rows) a.prefix_ml[slot + tid] = make_float2(ok ? m - P_BIAS : 0.f, ok ? l : __int_as_float(0x7fc00000));
        tc_fence_before();
      }
      tiles += n;
      halves += 2 * n;
      __syncthreads();
      tc_fence_after();
    }
    // ---- the next item
    if (place + PX_ITEM_COST + x.units >= v1) break;
    place += x.units + PX_ITEM_COST;
    if (++item == x.tiles(members) * heads) {
      item = 0;
      int end = x.end;
      do {
        ++g;  // the list has places left, so another group with units follows
        const int start = end;
        end = max(start, clamp_start(a, g + 1));
        x = group_of(a, g, start, end);
      } while (x.units == 0);
    }
  }
  let_next_begin();
  if (warp == 0) tmem_dealloc(tmem, PX_TMEM);
}

template <int KIND, int DH, bool SPLIT>
cudaError_t launch(const PrefixArgs &a, int dev, int sms, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};  // devices whose limit of dynamic shared memory is raised
  using T = PxShape<KIND, DH, SPLIT>;
  static_assert(sizeof(PxSmem<KIND, DH, SPLIT>) >= (KIE_PAGED_MAX_GROUPS + 4) * 4 + KIE_PAGED_MAX_GROUPS * 8, "the list's arrays");
  // no more than T::BLOCKS to an SM: a third one's TMEM would have to wait
  const int smem = (int)std::max<size_t>(sizeof(PxSmem<KIND, DH, SPLIT>), 80 * 1024);
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (!bit || !(ready.load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(prefix_kernel<KIND, DH, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_after_previous(prefix_kernel<KIND, DH, SPLIT>, sms * T::BLOCKS, PX_THREADS, smem, stream, a);
}

template <int DH>
cudaError_t launch_dh(const PrefixArgs &a, int dev, int sms, cudaStream_t stream) {
  const bool wide = a.q_dtype == KIE_F32;
  if (a.pages.dtype == KIE_BF16) return launch<PG_BF16, DH, false>(a, dev, sms, stream);
  if (a.pages.dtype == KIE_E4M3)
    return wide ? launch<PG_E4M3, DH, true>(a, dev, sms, stream) : launch<PG_E4M3, DH, false>(a, dev, sms, stream);
  return wide ? launch<PG_F16, DH, true>(a, dev, sms, stream) : launch<PG_F16, DH, false>(a, dev, sms, stream);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// The workspace: that of the rows' own positions, then what the two kernels pass on.
struct Parts {
  size_t per_block, row_lo, rows, ml, o, all;
  Parts(int n_seqs, int n_heads, int n_kv_heads, int head_dim, int sms) {
    const size_t slots = (size_t)n_seqs * n_heads + (size_t)PX_M * 2 * sms;
    per_block = up256(kie_paged_attention_workspace_bytes(n_heads, n_kv_heads, head_dim, sms));
    row_lo = per_block + 256;
    rows = up256(row_lo + (size_t)n_seqs * 4);
    ml = up256(rows + (size_t)n_seqs * sizeof(PrefixRow));
    o = up256(ml + slots * 8);
    all = o + slots * head_dim * 4;
  }
};

}  // namespace
}  // namespace kie

size_t kie_paged_prefix_workspace_bytes(int n_seqs, int n_heads, int n_kv_heads, int head_dim, int sms) {
  return kie::Parts(n_seqs, n_heads, n_kv_heads, head_dim, sms).all;
}

cudaError_t kie_launch_paged_prefix(const kie_paged_prefix_attention_args &args, int dev, int sms, cudaStream_t stream) {
  kie::PrefixArgs a;
  static_cast<kie_paged_attention_args &>(a) = kie::rows_in_lens(args.a);
  a.group_start = args.group_start;
  a.prefix_lens = args.prefix_lens;
  a.n_groups = args.n_groups;
  const kie::Parts p(a.n_seqs, a.n_heads, a.pages.n_kv_heads, a.pages.head_dim, sms);
  uint8_t *at = static_cast<uint8_t *>(a.workspace);
  a.per_block = reinterpret_cast<long long *>(at + p.per_block);
  a.row_lo = reinterpret_cast<int32_t *>(at + p.row_lo);
  a.rows = reinterpret_cast<kie::PrefixRow *>(at + p.rows);
  a.prefix_ml = reinterpret_cast<float2 *>(at + p.ml);
  a.prefix = reinterpret_cast<float *>(at + p.o);
  const cudaError_t e = a.pages.head_dim == 64 ? kie::launch_dh<64>(a, dev, sms, stream) : kie::launch_dh<128>(a, dev, sms, stream);
  return e != cudaSuccess ? e : kie_launch_paged_suffix(a, dev, sms, stream);
}
