// Attention of one new token per sequence over a paged K/V cache, split over the cache's length and joined.
//
// The work is a list of items (query row, KV head), each a row of units of 64 (E4M3: 128) positions. Every block of the
// grid takes an equal run of the list, whatever items it belongs to, so a ragged batch and a single long sequence load
// the GPU alike; a block keeps the whole items of its run to itself and publishes the pieces of the (at most two)
// items that it shares with its neighbours. The last block to publish a piece of an item joins them all (in two levels
// where they are many), in the order of the pieces: no block waits for another, and the result does not depend on
// which one is last.
//
// Inside a block each of four warps takes a quarter of a unit, one tile. Both products run as mma.sync m16n8k16 in the
// transposed form, so that no row of an instruction is wasted on the at most 8 query heads of a KV head: S^T = K Q^T
// (16 positions x 8 heads) and O^T += V^T P^T (16 dimensions x 8 heads). K is the A operand as it lies in shared memory
// (ldmatrix), V through ldmatrix.trans; the weights P pass from accumulator to B operand with movmatrix. Where 16 bits
// do not hold a B value exactly (fp32 queries; the weights), its remainder goes through a second mma. The running sum
// and output of a warp's positions stay in registers.
//
// No tcgen05: an MMA of 128 rows would have 5 of 128 filled, and at 20 operations a byte of K/V the arithmetic is far
// from the bound (tensor pipe 14 % busy with bf16, 27 % with E4M3). Bound by HBM where there is much to read: 256
// sequences of 4,096 positions (bf16, 16 heads over 4 of 128, 2.15 GB) take 309-313 us, 6.9 TB/s, 1.02 of the measured
// copy rate. E4M3 is paced by its instructions instead (its loop has no memory stall left; a quarter of its tensor work is
// the second part of queries that 16-bit types leave zero): 61 ragged sequences, 189 MB, take 39.3 us, 4.8 TB/s; 1.1 GB
// with 20 heads 172 us, 6.4 TB/s. Where there is little to read it is bound by its chain of latencies: launch,
// lengths, page ids, K, V, the join of the warps, and for shared items the arrival and the join of the pieces (one
// sequence of 128 positions 6.0 us, of 1,152 9.8 us, of 8,704 14.0 us).
//
// The reference of the softmax is not the running maximum but a value that stays within 2^8 of it: weights up to 2^15
// fit in fp16, so it is only moved (with the shuffles and the rescaling that this costs) when a weight passes that.
#include <float.h>

#include <atomic>
#include <type_traits>

#include "kie_device.cuh"
#include "kie_paged.cuh"

namespace kie {
namespace {

constexpr int PA_WARPS = 4;
constexpr int PA_THREADS = PA_WARPS * 32;
constexpr int PA_MAX_BLOCKS_PER_SM = 3;
constexpr int PA_RING_BYTES = 192 * 1024;   // the rings of an SM's blocks
constexpr int PA_ROWS = PAGED_MAX_GROUP;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
// Weights are kept as 2^7 2^(v - ref): an fp16 pair holds them to 2^-25, which is 2^-32 of the largest.
constexpr float P_BIAS = 7.f, P_LIMIT = 32768.f;
// The scales of E4M3 value rows count into the reference down to MIN_LOG2_SCALE (log2), so that after a move the plain
// weights, which the sum adds up, are at most 2^67. Rows of smaller scales that come later may outgrow the rest without
// their weighted values showing it: the reference also moves when a lane's plain weights of a tile pass P_PLAIN. The sums of
// 2^30 positions then stay below 2^121.
// An infinite scale counts as 2^127: the reference stays finite, and with it the sum and the lse, which do not depend on V.
constexpr float MIN_LOG2_SCALE = -60.f, MAX_LOG2_SCALE = 127.f, P_PLAIN = 0x1p90f;

enum { PG_F16 = 0, PG_BF16 = 1, PG_E4M3 = 2 };

// A warp's tile: 16 positions (32 of E4M3), as one half of K rows and one of V rows of 32 * DH bytes each.
template <int KIND, int DH>
struct PaTile {
  static constexpr int ES = KIND == PG_E4M3 ? 1 : 2, SUBS = KIND == PG_E4M3 ? 2 : 1;  // 16-position parts
  static constexpr int POS = 16 * SUBS, UNIT = POS * PA_WARPS;
  static constexpr int ROW = DH * ES, CH = ROW / 16, HALF = POS * ROW;  // bytes; 16-byte chunks of a row
  // Blocks of an SM: a third helps where its 168 registers a thread are enough (256 x 4,096 positions, 16 heads over 4:
  // 311 us against 316 with two); E4M3 needs more (191 against 186), and rows of 64 gain nothing (171 against 167).
  static constexpr int BLOCKS = KIND != PG_E4M3 && DH == 128 ? 3 : 2;
  static constexpr int NS = PA_RING_BYTES / BLOCKS / PA_WARPS / HALF;   // ring slots, a half each
  static constexpr int LOADS = HALF / 512;                              // chunks each lane copies
};

// A block's shared memory: the warps' rings (the slot last used also joins the four warps), the E4M3 scales of each
// slot, which positions of it are live, and the warps' references and sums.
template <int KIND, int DH>
struct PaSmem {
  using T = PaTile<KIND, DH>;
  uint8_t ring[PA_WARPS][T::NS][T::HALF];
  float scale[PA_WARPS][KIND == PG_E4M3 ? T::NS : 1][32];
  float4 m[PA_ROWS], l[PA_ROWS];  // of a row: the four warps'
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

// Flushing results and arguments below 2^-126 to 0 (a weight that small counts for nothing) saves the rescaling around
// each of these.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float log2_scale(float x) { return fminf(fmaxf(lg2(fabsf(x)), MIN_LOG2_SCALE), MAX_LOG2_SCALE); }

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

// What query row b attends: positions [lo, len) of its sequence, in n units of UNIT positions from `from` on, a multiple of
// 16 (at least one unit, so that a row of no positions still writes its zeros). Rows of a step (a.seqs) end with their own
// position: their positions stand in a.lens here, and those of no sequence find no pages.
struct Span {
  int lo, len, from, n;
};
template <int UNIT, class Args>
__device__ __forceinline__ Span span_of(const Args &a, int b) {
  Span s;
  s.len = row_len(a, b);
  if constexpr (std::is_same<Args, PrefixArgs>::value)
    s.lo = __ldcg(a.row_lo + b);  // the positions before are the group's
  else
    s.lo = a.window > 0 ? max(0, s.len - a.window) : 0;
  s.from = s.lo & ~15;
  s.n = max(1, (int)((unsigned)(s.len - s.from + UNIT - 1) / UNIT));
  return s;
}

// Places in the list are numbered through, an item taking PA_ITEM_COST places before those of its units: starting an
// item (its queries, the join of the warps, the output) takes a block about as long as that many units.
// A run is at least PA_MIN_RUN places, or a whole item where items are short (PA_WHOLE places on average at most): to
// share an item costs about 2 us in the end, which is worth four units. (One sequence of 128 positions: 7.3 us whole,
// 8.3 us shared by two blocks. One of 1,152: 11.1 us in runs of 3 places, 11.6 in runs of 4, 12.0 in runs of 5.)
constexpr int PA_ITEM_COST = 2, PA_MIN_RUN = 3, PA_WHOLE = PA_ITEM_COST + 4;

// Unit `unit` of item (b, h), at place v of this block's run.
template <int UNIT>
struct Cursor {
  Span s;
  int b, h, unit, v;
  template <class Args>
  __device__ __forceinline__ void next(const Args &a) {
    ++v;
    if (++unit < s.n) return;
    unit = 0;
    v += PA_ITEM_COST;
    if (++h < a.pages.n_kv_heads) return;
    h = 0;
    if (++b < a.n_seqs) s = span_of<UNIT>(a, b);
  }
};

// a / b, with a 32-bit division where it does (a 64-bit one takes a few hundred cycles).
__device__ __forceinline__ long long divide(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// The number of places of this block's run (*end; 0 behind the list's end), the cursor at its first unit, and the
// places of a full run (*per_block). Every thread gets the same; two block barriers. The cursor may stand at or past
// *end: no units.
template <int UNIT, class Args>
__device__ __forceinline__ void locate(const Args &a, Cursor<UNIT> *c, int *end, long long *per_block) {
  __shared__ long long s_warp[PA_WARPS];
  __shared__ int s_b, s_h;
  __shared__ int s_off;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (a.n_seqs + PA_THREADS - 1) / PA_THREADS;
  const int b0 = min(tid * per, a.n_seqs), b1 = min(b0 + per, a.n_seqs);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += span_of<UNIT>(a, b).n + PA_ITEM_COST;
  long long up = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += x;
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
  const long long items = (long long)a.n_seqs * heads, mean = divide(all + items - 1, items);
  *per_block = max(divide(all + gridDim.x - 1, gridDim.x), mean <= PA_WHOLE ? mean : PA_MIN_RUN);
  const long long v0 = blockIdx.x * *per_block;
  *end = (int)max(0ll, min(*per_block, all - v0));
  if (v0 >= before && v0 < before + mine * heads) {
    long long at = before;
    int b = b0;
    for (;; ++b) {
      const long long n = (long long)(span_of<UNIT>(a, b).n + PA_ITEM_COST) * heads;
      if (v0 < at + n) break;
      at += n;
    }
    s_b = b;
    long long off = v0 - at;  // into the sequence's items
    const int n = span_of<UNIT>(a, b).n + PA_ITEM_COST;
    int h = 0;
    for (; off >= n; off -= n) ++h;
    s_h = h;
    s_off = (int)off;
  }
  __syncthreads();
  c->v = 0;
  if (v0 >= all) return;
  c->b = s_b;
  c->s = span_of<UNIT>(a, s_b);
  c->h = s_h;
  c->unit = max(0, s_off - PA_ITEM_COST);
  c->v = max(0, PA_ITEM_COST - s_off);
}

// ---- workspace ----------------------------------------------------------------------------------------------

// Per block: three arrival words, then four pieces: o [group][dh], then (m, l) [group] (rounded to 16 bytes). A block
// continues at most one item that an earlier block started and starts at most one that it does not end:
//   word / piece CONT, START: the arrivals of the group of blocks that begins with this one, as a continuation or as
//   the item's start; this block's piece of either.
//   word ITEM: arrivals of an item's groups, at the block that starts it; pieces JOINED + CONT / START: a joined group.
enum { CONT = 0, START = 1, ITEM = 2, JOINED = 2 };
constexpr int PA_WORDS = 3, PA_PIECES = 4;
constexpr int PA_ONE_LEVEL = 24;  // up to this many pieces are joined at once, more in groups of about their root

__host__ __device__ __forceinline__ size_t pa_piece_floats(int group, int dh) { return ((size_t)group * (dh + 2) + 3) / 4 * 4; }
__host__ __device__ __forceinline__ size_t pa_header_bytes(int blocks) {
  return ((size_t)blocks * PA_WORDS * 8 + 255) / 256 * 256;
}

struct Workspace {
  unsigned long long *words;
  float *pieces;
  size_t piece;  // floats
  __device__ __forceinline__ Workspace(const kie_paged_attention_args &a, int dh)
      : words(static_cast<unsigned long long *>(a.workspace)),
        pieces(reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + pa_header_bytes(gridDim.x))),
        piece(pa_piece_floats(a.n_heads / a.pages.n_kv_heads, dh)) {}
  __device__ __forceinline__ unsigned long long *word(int block, int which) const { return words + block * PA_WORDS + which; }
  __device__ __forceinline__ float *at(int block, int which) const { return pieces + ((size_t)block * PA_PIECES + which) * piece; }
};

// One more arrival at *word; true for the n-th, which leaves the word at 0. A word holds the call's number above 8 bits
// of count: whatever it held before the call (an older call's number, other data) counts as no arrivals, so the
// workspace needs no clearing; a replayed graph, whose number stays the same, finds the zeros of its last replay.
__device__ __forceinline__ bool arrive(unsigned long long *word, unsigned long long call, int n) {
  if (n == 1) return true;
  unsigned long long seen = 0ull;  // what the last call left
  while ((seen >> 8) != call) {    // a failed exchange finds other data once, or another block's first arrival
    unsigned long long was;
    asm volatile("atom.acquire.gpu.global.cas.b64 %0, [%1], %2, %3;"
                 : "=l"(was)
                 : "l"(word), "l"(seen), "l"((call << 8) | 1ull)
                 : "memory");
    if (was == seen) return false;
    seen = was;
  }
  asm volatile("atom.acquire.gpu.global.add.u64 %0, [%1], %2;" : "=l"(seen) : "l"(word), "l"(1ull) : "memory");
  if ((int)(seen & 255ull) + 1 < n) return false;
  *word = 0ull;
  return true;
}

// The block's earlier writes to the workspace are seen by the block that arrives last. Every thread must call.
__device__ __forceinline__ bool block_arrive(unsigned long long *word, unsigned long long call, int n) {
  __shared__ bool s_last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();  // release: cumulative over the writes of the block's threads, ordered before it by the barrier
    s_last = arrive(word, call, n);
  }
  __syncthreads();
  const bool last = s_last;
  __syncthreads();
  return last;
}

// A thread's share of a joined item: four dimensions d .. d + 3 of the rows r0, r0 + STEP, .. (ROWS of them at most).
template <int DH>
struct JoinShare {
  static constexpr int LANES = DH / 4, STEP = PA_THREADS / LANES, ROWS = PA_ROWS / STEP;
  int r0 = threadIdx.x / LANES, d = threadIdx.x % LANES * 4;
};

// Pieces in their order: the first, and the others `step` floats apart.
struct Pieces {
  const float *first, *rest;
  size_t step;
  __device__ __forceinline__ const float *operator[](int i) const { return i == 0 ? first : rest + (size_t)(i - 1) * step; }
};

// The thread's share of n pieces, joined in order: put(r, d, sum, M, L) gets their sum at the largest
// reference M. The loads of BATCH pieces are in flight at a time.
template <int DH, class P>
__device__ __forceinline__ void join_pieces(const Pieces &piece, int n, int group, const P &put) {
  using S = JoinShare<DH>;
  constexpr int R = S::ROWS, BATCH = 8 / R;
  const S me;
  float top[R], sum[R];
  float4 acc[R];
#pragma unroll
  for (int q = 0; q < R; ++q) {
    top[q] = -INFINITY;
    sum[q] = 0.f;
    acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (me.r0 >= group) return;
  for (int i0 = 0; i0 < n; i0 += BATCH) {
    float2 ml[BATCH][R];
    float4 y[BATCH][R];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const float *p = piece[min(i0 + k, n - 1)];
#pragma unroll
      for (int q = 0; q < R; ++q) {
        const int r = min(me.r0 + q * S::STEP, group - 1);
        ml[k][q] = __ldcg(reinterpret_cast<const float2 *>(p + group * DH + 2 * r));
        y[k][q] = __ldcg(reinterpret_cast<const float4 *>(p + r * DH + me.d));
      }
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
      float mn = top[q];
#pragma unroll
      for (int k = 0; k < BATCH; ++k)
        if (i0 + k < n) mn = fmaxf(mn, ml[k][q].x);
      const float ref = mn == -INFINITY ? 0.f : mn, f0 = ex2(top[q] - ref);
      sum[q] *= f0, acc[q].x *= f0, acc[q].y *= f0, acc[q].z *= f0, acc[q].w *= f0;
#pragma unroll
      for (int k = 0; k < BATCH; ++k)
        if (i0 + k < n) {
          const float f = ex2(ml[k][q].x - ref);
          sum[q] = fmaf(ml[k][q].y, f, sum[q]);
          acc[q].x = fmaf(y[k][q].x, f, acc[q].x), acc[q].y = fmaf(y[k][q].y, f, acc[q].y);
          acc[q].z = fmaf(y[k][q].z, f, acc[q].z), acc[q].w = fmaf(y[k][q].w, f, acc[q].w);
        }
      top[q] = mn;
    }
  }
#pragma unroll
  for (int q = 0; q < R; ++q)
    if (me.r0 + q * S::STEP < group) put(me.r0 + q * S::STEP, me.d, acc[q], top[q], sum[q]);
}

// Four dimensions of a query head's output from its weighted sum, and its lse from the reference M (log2 units) and the
// sum of weights L: zeros and -inf where nothing was attended. vec: the output is aligned for one store of four.
template <int DH, class Args>
__device__ __forceinline__ void finish4(const Args &a, bool vec, int b, int64_t head, int d, float4 acc, float M, float L) {
  if constexpr (std::is_same<Args, PrefixArgs>::value) {  // the piece that the join takes
    const int64_t at = b * (int64_t)a.n_heads + head;
    *reinterpret_cast<float4 *>(a.own + at * DH + d) = acc;
    if (d == 0) a.own_ml[at] = make_float2(M, L);
    return;
  }
  const float inv = L == 0.f ? 0.f : rcp(L);
  const float v[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
  const int64_t to = b * a.out_stride[0] + head * a.out_stride[1] + d;
  if (!vec) {
#pragma unroll
    for (int e = 0; e < 4; ++e) paged_store(a.out, to + e, a.q_dtype, v[e]);
  } else if (a.q_dtype == KIE_F32) {
    *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + to) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + to) =
        make_uint2(pack2(v[0], v[1], a.q_dtype), pack2(v[2], v[3], a.q_dtype));
  }
  if (d == 0 && a.lse) a.lse[(int64_t)b * a.n_heads + head] = L == 0.f ? -INFINITY : (M + lg2(L)) * LN2;
}
__device__ __forceinline__ bool out_vec(const kie_paged_attention_args &a) {
  const int size = paged_dtype_bytes(a.q_dtype);
  return ((uintptr_t)a.out | (uintptr_t)(a.out_stride[0] * size) | (uintptr_t)(a.out_stride[1] * size)) % (4 * size) == 0;
}

template <int DH>
__device__ __forceinline__ void put_piece(float *p, int group, int r, int d, float4 acc, float M, float L) {
  *reinterpret_cast<float4 *>(p + r * DH + d) = acc;
  if (d == 0) *reinterpret_cast<float2 *>(p + group * DH + 2 * r) = make_float2(M, L);
}

// After this block has written its piece of item (b, h), whose `units` units begin at place v of the list: whoever of
// the blocks that share it comes last joins the pieces.
template <int DH, class Args>
__device__ __forceinline__ void publish(const Args &a, unsigned long long call, int b, int h, long long v,
                                        int units, long long per_block) {
  const Workspace ws(a, DH);
  const int first = (int)divide(v, per_block), last = (int)divide(v + units - 1, per_block);
  const int group = a.n_heads / a.pages.n_kv_heads, n = last - first + 1;
  const bool vec = out_vec(a);
  const auto finish = [&](int r, int d, float4 acc, float M, float L) {
    finish4<DH>(a, vec, b, (int64_t)h * group + r, d, acc, M, L);
  };
  const size_t step = PA_PIECES * ws.piece;
  if (n <= PA_ONE_LEVEL) {
    if (block_arrive(ws.word(first, START), call, n))
      join_pieces<DH>(Pieces{ws.at(first, START), ws.at(first + 1, CONT), step}, n, group, finish);
    return;
  }
  const int fan = (int)ceilf(sqrtf((float)n));
  const int g0 = ((int)blockIdx.x - first) / fan * fan, size = min(fan, n - g0), at = first + g0, kind = g0 ? CONT : START;
  if (!block_arrive(ws.word(at, kind), call, size)) return;
  float *to = ws.at(at, JOINED + kind);
  join_pieces<DH>(Pieces{ws.at(at, kind), ws.at(at + 1, CONT), step}, size, group,
                  [&](int r, int d, float4 acc, float M, float L) { put_piece<DH>(to, group, r, d, acc, M, L); });
  const int groups = (n + fan - 1) / fan;
  if (block_arrive(ws.word(first, ITEM), call, groups))
    join_pieces<DH>(Pieces{ws.at(first, JOINED + START), ws.at(first + fan, JOINED + CONT), fan * step}, groups, group, finish);
}

// ---- the kernel ---------------------------------------------------------------------------------------------

// The pairs of elements at + off(0 .. N - 1) of a query head, as they are: two words each of fp32, else one. Nothing
// waits for the loads here, so that they can be issued long before their use.
template <int N, int WORDS, class F>
__device__ __forceinline__ void request_pairs(const kie_paged_attention_args &a, int64_t at, const F &off,
                                              uint32_t (&w)[N * WORDS]) {
  const int size = paged_dtype_bytes(a.q_dtype);
  const bool pair = ((uintptr_t)a.q | (uintptr_t)(a.q_stride[0] * size) | (uintptr_t)(a.q_stride[1] * size)) % (2 * size) == 0;
  if (WORDS == 2 && a.q_dtype == KIE_F32) {
    const uint32_t *q = static_cast<const uint32_t *>(a.q) + at;
    if (pair) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint2 x = *reinterpret_cast<const uint2 *>(q + off(i));
        w[i * WORDS] = x.x, w[i * WORDS + WORDS - 1] = x.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i * WORDS] = q[off(i)], w[i * WORDS + WORDS - 1] = q[off(i) + 1];
    }
  } else {
    const uint16_t *q = static_cast<const uint16_t *>(a.q) + at;
    if (pair) {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i * WORDS] = *reinterpret_cast<const uint32_t *>(q + off(i));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i * WORDS] = q[off(i)] | (uint32_t)q[off(i) + 1] << 16;
    }
  }
}

// Where column d of a warp's output row r lies in the joining area: the accumulators' four column pairs of a lane
// quad go to different banks.
template <int KIND>
__device__ __forceinline__ int join_col(int r, int d) {
  return d ^ (((r >> 1) & 3) << (KIND == PG_E4M3 ? 4 : 3));
}

template <int KIND, int DH, bool SPLIT, class Args>
__global__ void __launch_bounds__(PA_THREADS, PaTile<KIND, DH>::BLOCKS)
paged_attn_kernel(const Args a, unsigned long long call) {
  using T = PaTile<KIND, DH>;
  using Sm = PaSmem<KIND, DH>;
  constexpr int NS = T::NS, CH = T::CH, ROW = T::ROW, ES = T::ES, SUBS = T::SUBS, LOADS = T::LOADS;
  constexpr int KSTEPS = DH / 16, MT = DH / 16;
  constexpr uint32_t FULL = SUBS == 2 ? 0xffffffffu : 0xffffu;
  static_assert(T::HALF >= PA_ROWS * DH * 4, "the joining area is one slot");
  extern __shared__ __align__(1024) uint8_t pa_raw[];
  Sm &sm = *reinterpret_cast<Sm *>(pa_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = a.n_heads / a.pages.n_kv_heads;
  const unsigned bs = a.pages.block_size;
  const int bs_shift = (bs & (bs - 1)) ? -1 : __ffs(bs) - 1;

  // Beside a prefix the kernel before this one is at work on it, and what came before that is complete: its blocks let this
  // one begin when they have seen to that. The join has to find both complete, so the last block waits, in the end.
  constexpr bool BESIDE = std::is_same<Args, PrefixArgs>::value;
  if (BESIDE)
    __threadfence();  // nothing that older kernels left in this SM's L1 is read
  else
    wait_for_previous();
  Cursor<T::UNIT> c;
  int end;
  long long per_block;
  locate(a, &c, &end, &per_block);
  if (c.v >= end) {
    if (BESIDE && blockIdx.x == gridDim.x - 1) wait_for_previous();
    return;
  }

  // Chunk ch of row r of a half lies at chunk ch ^ swz(r): the eight rows of an 8 x 8 matrix fall in different banks.
  const auto swz = [](int row) { return CH >= 8 ? row & 7 : (row >> 1) & 3; };

  // ---- producer side: the warp's tile of unit `p`, K half first, then V. A lane copies chunks lane + 32 i.
  Cursor<T::UNIT> p = c;
  uint32_t p_live = 0;
  int p_base = 0, p_page[SUBS], p_id[SUBS];  // lane j: the pages of the warp's tile of unit p_base + j; of p's tile
  const int row0 = lane / CH;  // row of the lane's first chunk; the next are 32 / CH rows on
  const uint32_t dst_lane = (lane * 16) ^ (swz(row0) << 4);
  // strides in bytes: below 2^32, of positions below 2^27, so that an address is the base and two 32 x 32-bit products
  const uint32_t k_page = (uint32_t)a.pages.k_stride[0] * ES, k_row = (uint32_t)a.pages.k_stride[2] * ES;
  const uint32_t v_page = (uint32_t)a.pages.v_stride[0] * ES, v_row = (uint32_t)a.pages.v_stride[2] * ES;
  const uint8_t *k_base, *v_base;  // the lane's first chunk in page 0 of p's head
  auto set_head = [&]() {
    const int at = (lane % CH) * 16;
    const uint64_t k_head = (uint64_t)p.h * (uint32_t)a.pages.k_stride[1] * ES, v_head = (uint64_t)p.h * (uint32_t)a.pages.v_stride[1] * ES;
    k_base = static_cast<const uint8_t *>(a.pages.k) + k_head + (uint64_t)row0 * k_row + at;
    v_base = static_cast<const uint8_t *>(a.pages.v) + v_head + (uint64_t)row0 * v_row + at;
  };
  const uint32_t ring0 = smem_u32(sm.ring[warp]);
  auto first_pos = [&](const Cursor<T::UNIT> &x) { return x.s.from + (x.unit * PA_WARPS + warp) * T::POS; };
  auto fetch_pages = [&]() {  // requested before the issue that uses them
    p_base = p.unit;
    int seq = p.b;
    if (a.seqs && p.v < end) seq = a.seqs[p.b];
#pragma unroll
    for (int i = 0; i < SUBS; ++i) {
      const int pos = first_pos(p) + lane * T::UNIT + 16 * i;
      p_page[i] = -1;
      if (p.v < end && pos < p.s.len && (unsigned)seq < (unsigned)a.n_table)
        p_page[i] = a.block_table[seq * a.table_stride + (bs_shift >= 0 ? (unsigned)pos >> bs_shift : (unsigned)pos / bs)];
    }
  };
  auto issue = [&](int slot, bool is_v) {
    const int pos = first_pos(p);
    if (!is_v) {
      const int hi = p.s.len - pos, lo = p.s.lo - pos;
      p_live = hi >= T::POS ? FULL : hi > 0 ? (1u << hi) - 1u : 0u;
      if (lo > 0) p_live &= lo >= 32 ? 0u : ~((1u << lo) - 1u);
#pragma unroll
      for (int i = 0; i < SUBS; ++i) {
        p_id[i] = __shfl_sync(0xffffffffu, p_page[i], p.unit - p_base);
        if ((unsigned)p_id[i] >= (unsigned)a.pages.n_blocks) p_live &= ~(0xffffu << (16 * i));
      }
      if (p.v >= end) p_live = 0u;  // behind the run
      if (lane == 0) sm.live[warp][slot] = p_live;
    }
    if (p_live) {
      const uint32_t row = is_v ? v_row : k_row, step = row * (32 / CH);
      const uint32_t dst = ring0 + slot * T::HALF + dst_lane;
#pragma unroll
      for (int s = 0; s < SUBS; ++s) {
        const unsigned at = pos + 16 * s, off = bs_shift >= 0 ? at & (bs - 1) : at % bs;
        const uint32_t live = (p_live >> (16 * s)) & 0xffffu;
        const uint32_t page = live ? p_id[s] : 0;  // an address inside the pages even where nothing is read
        const uint8_t *src = (is_v ? v_base : k_base) + (uint64_t)page * (is_v ? v_page : k_page) + (uint64_t)off * row;
        constexpr int N = LOADS / SUBS;
        if (live == 0xffffu) {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            cp_async16((dst ^ (swz((i + s * N) * (32 / CH)) << 4)) + (i + s * N) * 512, src + (uint64_t)step * i);
          }
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) {
            cp_async16((dst ^ (swz((i + s * N) * (32 / CH)) << 4)) + (i + s * N) * 512, src + (uint64_t)step * i,
                       (p_live >> (row0 + (i + s * N) * (32 / CH))) & 1u);
          }
        }
      }
      if (KIND == PG_E4M3) {  // a row's scale to each lane
        const int64_t *ss = is_v ? a.pages.v_scale_stride : a.pages.k_scale_stride;
        const unsigned at = pos + lane, off = bs_shift >= 0 ? at & (bs - 1) : at % bs;
        const bool live = (p_live >> lane) & 1u;
        const int64_t page = live ? (lane < 16 ? p_id[0] : p_id[SUBS - 1]) : 0;
        cp_async4(&sm.scale[warp][KIND == PG_E4M3 ? slot : 0][lane],
                  (is_v ? a.pages.v_scale : a.pages.k_scale) + page * ss[0] + p.h * ss[1] + off * ss[2],
                  live);
      }
    }
    if (is_v) {
      if (p.v < end) p.next(a);
      if (p.unit == 0) set_head();
      if (p.unit == 0 || p.unit == p_base + 32) fetch_pages();
    }
  };

  // the first item's queries, and its pages, on their way together
  const int g = lane >> 2, t = lane & 3;
  uint32_t raw[2 * KSTEPS * (SPLIT ? 2 : 1)];
  auto request_q = [&](int b, int h) {
    // E4M3 rows come as four codes to a lane, so that the k order of a step is 4t .. 4t + 3
    request_pairs<2 * KSTEPS, SPLIT ? 2 : 1>(
        a, b * a.q_stride[0] + (int64_t)(h * group + min(g, group - 1)) * a.q_stride[1],
        [&](int i) { return 16 * (i >> 1) + (KIND == PG_E4M3 ? 4 * t + 2 * (i & 1) : 2 * t + 8 * (i & 1)); }, raw);
  };
  request_q(c.b, c.h);
  set_head();
  fetch_pages();
#pragma unroll 1
  for (int x = 0; x < NS - 1; ++x) {
    issue(x, x & 1);
    cp_commit();
  }

  // ---- consumer side. Lane (g, t) holds, of the accumulators, heads 2t and 2t + 1; of the B operands, head g.
  const uint32_t k_at = ((lane & 15) * ROW) + (((lane >> 4) ^ swz(lane & 7)) << 4);  // ldmatrix row of the lane
  const uint32_t v_at = ((((lane >> 4) << 3) + (lane & 7)) * ROW) + ((((lane >> 3) & 1) ^ swz(lane & 7)) << 4);
  uint32_t qb[KSTEPS][SPLIT ? 4 : 2];
  float rs[2], m[2], bias[2], l[2], o[MT][4];  // rs: score scale in log2 units; bias: P_BIAS - m
  int ring = 0;  // slot of the next half

  for (;;) {  // an item, or this block's part of it
    const int units = min(c.s.n - c.unit, end - c.v);
    {  // its query heads as B fragments
      float down = 1.f;
      if (!SPLIT) {
#pragma unroll
        for (int i = 0; i < 2 * KSTEPS; ++i) qb[i >> 1][i & 1] = g < group ? raw[SPLIT ? 0 : i] : 0u;
      } else {  // bring the head's largest element to [2^13, 2^14) by a power of two
        float2 f[2 * KSTEPS];
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * KSTEPS; ++i) {
          const uint32_t w = raw[SPLIT ? 2 * i : i];
          f[i] = a.q_dtype == KIE_F32   ? make_float2(__uint_as_float(w), __uint_as_float(raw[SPLIT ? 2 * i + 1 : i]))
                 : a.q_dtype == KIE_F16 ? __half22float2(*reinterpret_cast<const __half2 *>(&w))
                                        : make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
          if (g >= group) f[i] = make_float2(0.f, 0.f);
          top = fmaxf(top, fmaxf(fabsf(f[i].x), fabsf(f[i].y)));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        int e2 = 0;
        if (top > 0.f && top <= FLT_MAX) e2 = max(-120, min(120, 140 - (int)(__float_as_uint(top) >> 23)));
        const float up = __int_as_float((127 + e2) << 23);
        down = __int_as_float((127 - e2) << 23);
#pragma unroll
        for (int i = 0; i < 2 * KSTEPS; ++i) {
          const float x = f[i].x * up, y = f[i].y * up;
          const uint32_t w = pack16<KIND>(x, y);
          qb[i >> 1][i & 1] = w;
          qb[i >> 1][SPLIT ? 2 + (i & 1) : 0] = rest16<KIND>(x, y, w);
        }
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

    for (int u = 0; u < units; ++u) {
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
          for (int e = 0; e < 4; ++e) {
            // an infinity in K makes the product with the queries' second part infinite or NaN: the first alone counts then
            if (SPLIT && KIND == PG_F16 && !(fabsf(x[1][e]) <= FLT_MAX)) x[1][e] = 0.f;
            s[i][e] = (x[0][e] + x[1][e]) * ks[e >> 1];
          }
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
        if (KIND == PG_E4M3) far = far || part[0] > P_PLAIN || part[1] > P_PLAIN;
        if (__any_sync(0xffffffffu, far)) {  // move the references to the maxima so far
          float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < SUBS; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((live >> (16 * i + g + 8 * (e >> 1))) & 1u)
                top[e & 1] = fmaxf(top[e & 1], fmaf(s[i][e], rs[e & 1], KIND == PG_E4M3 ? log2_scale(vs[i][e >> 1]) : 0.f));
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

      ring = ring + 1 == NS ? 0 : ring + 1;
    }

    // ---- the item's end, or the run's: join the four warps through the slot just used
    const bool starts = c.unit == 0, ends = c.unit + units == c.s.n;
    const int used = ring == 0 ? NS - 1 : ring - 1, b = c.b, h = c.h, n = c.s.n;
    const long long v = blockIdx.x * per_block + c.v - c.unit;  // place of the item's first unit
    c.unit += units - 1;
    c.v += units - 1;
    c.next(a);
    const bool done = c.v >= end;
    if (!done) request_q(c.b, c.h);  // the next item's queries arrive while this one is finished
    {
      __syncwarp();  // every lane is done with the slot
      float *join = reinterpret_cast<float *>(sm.ring[warp][used]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], x);
        const int r = 2 * t + k;
        if (g == 0) {
          reinterpret_cast<float *>(&sm.m[r])[warp] = m[k] - P_BIAS;
          reinterpret_cast<float *>(&sm.l[r])[warp] = l[k];
        }
#pragma unroll
        for (int n = 0; n < MT; ++n) {
          if (KIND == PG_E4M3) {
            *reinterpret_cast<float2 *>(&join[r * DH + join_col<KIND>(r, 16 * n + 2 * g)]) = make_float2(o[n][k], o[n][2 + k]);
          } else {
            join[r * DH + join_col<KIND>(r, 16 * n + g)] = o[n][k];
            join[r * DH + join_col<KIND>(r, 16 * n + g + 8)] = o[n][2 + k];
          }
        }
      }
      __syncthreads();
      const bool whole = ends && starts;
      float *piece = Workspace(a, DH).at(blockIdx.x, starts ? START : CONT);
      const bool vec = out_vec(a);
      const JoinShare<DH> me;
#pragma unroll
      for (int q = 0; q < JoinShare<DH>::ROWS; ++q) {
        const int r = me.r0 + q * JoinShare<DH>::STEP;
        if (r >= group) break;
        const float4 wm = sm.m[r], wl = sm.l[r];
        const float M = fmaxf(fmaxf(wm.x, wm.y), fmaxf(wm.z, wm.w)), ref = M == -INFINITY ? 0.f : M;
        const float f[PA_WARPS] = {ex2(wm.x - ref), ex2(wm.y - ref), ex2(wm.z - ref), ex2(wm.w - ref)};
        const float L = fmaf(wl.w, f[3], fmaf(wl.z, f[2], fmaf(wl.y, f[1], wl.x * f[0])));
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < PA_WARPS; ++w) {
          const float4 y = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(sm.ring[w][used]) + r * DH +
                                                             join_col<KIND>(r, me.d));
          acc.x = fmaf(y.x, f[w], acc.x), acc.y = fmaf(y.y, f[w], acc.y);
          acc.z = fmaf(y.z, f[w], acc.z), acc.w = fmaf(y.w, f[w], acc.w);
        }
        if (whole)
          finish4<DH>(a, vec, b, (int64_t)h * group + r, me.d, acc, M, L);
        else
          put_piece<DH>(piece, group, r, me.d, acc, M, L);
      }
      if (!whole)
        publish<DH>(a, call, b, h, v, n, per_block);
      __syncthreads();  // the next half may land in the slot, and the next item's sums in theirs
      if (done) break;
    }
  }
  if (!BESIDE) let_next_begin();
  cp_wait<0>();
  if (BESIDE && blockIdx.x == gridDim.x - 1) wait_for_previous();
}

// 56 bits, never 0, that no other call of the process has (steps through the odd numbers) and other data hardly holds.
unsigned long long call_number() {
  static std::atomic<uint64_t> calls{0x9e3779b97f4a7dull};
  return calls.fetch_add(0x3c6ef372fe94faull, std::memory_order_relaxed) & ((1ull << 56) - 1);
}

template <int KIND, int DH, bool SPLIT, class Args>
cudaError_t launch(const Args &a, int dev, int sms, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};  // devices whose limit of dynamic shared memory is raised
  const int smem = sizeof(PaSmem<KIND, DH>);
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (!bit || !(ready.load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(paged_attn_kernel<KIND, DH, SPLIT, Args>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_after_previous(paged_attn_kernel<KIND, DH, SPLIT, Args>, sms * PaTile<KIND, DH>::BLOCKS, PA_THREADS, smem, stream, a,
                               call_number());
}

template <int DH, class Args>
cudaError_t launch_dh(const Args &a, int dev, int sms, cudaStream_t stream) {
  if (a.pages.dtype == KIE_BF16) return launch<PG_BF16, DH, false>(a, dev, sms, stream);
  if (a.pages.dtype == KIE_E4M3) return launch<PG_E4M3, DH, true>(a, dev, sms, stream);
  return a.q_dtype == KIE_F32 ? launch<PG_F16, DH, true>(a, dev, sms, stream) : launch<PG_F16, DH, false>(a, dev, sms, stream);
}

}  // namespace
}  // namespace kie

size_t kie_paged_attention_workspace_bytes(int n_heads, int n_kv_heads, int head_dim, int sms) {
  const size_t blocks = (size_t)sms * kie::PA_MAX_BLOCKS_PER_SM;
  return kie::pa_header_bytes(blocks) + blocks * kie::PA_PIECES * kie::pa_piece_floats(n_heads / n_kv_heads, head_dim) * 4;
}

cudaError_t kie_launch_paged_attention(const kie_paged_attention_args &args, int dev, int sms, cudaStream_t stream) {
  const kie_paged_attention_args a = kie::rows_in_lens(args);
  return a.pages.head_dim == 64 ? kie::launch_dh<64>(a, dev, sms, stream) : kie::launch_dh<128>(a, dev, sms, stream);
}

cudaError_t kie_launch_paged_own(const kie::PrefixArgs &a, int dev, int sms, cudaStream_t stream) {
  return a.pages.head_dim == 64 ? kie::launch_dh<64>(a, dev, sms, stream) : kie::launch_dh<128>(a, dev, sms, stream);
}
