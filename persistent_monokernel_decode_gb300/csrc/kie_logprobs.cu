// Log probabilities of tokens, entropies and the largest logits (kie_paged.cu holds the C entry).
//
// A row is streamed once. Each thread keeps a reference r within a few of the maximum of what it has seen, s = sum exp(x - r)
// and t = sum exp(x - r) (x - r), and the threads' sums are joined at the row's maximum m: ln p = x - m - ln s, and the
// entropy is ln s - t / s, which stays accurate where x itself is large. Rows too few to fill the GPU are split over a
// cluster of up to eight blocks, which meet at the cluster's barrier and pass their results through distributed shared
// memory. 8,191 rows of 32,000 bf16 logits take 91 us without alternatives (5.8 TB/s), 123 with the 20 largest: bound by the
// loads under way (of 4,096 rows DRAM is 66 % busy and the SMs 52 %, with 8 instructions an element of 16 bits, two fp32
// operations to an instruction; with alternatives 49 %, 59 % and 12), then by the end of a row; four rows take 7 us, a chain
// of the launch, the loads, the cluster's barriers and the ranking.
// Holding the row, so that the maximum is known before the sums, took more: in registers, unrolled, 22 instructions an
// element and 280 us for 8,191 rows of 32,000 bf16 logits; in shared memory 13 and 159 us, three rows to an SM being too few.
//
// The `top` largest: the maxima of groups of threads give a bound that at least `top` elements reach, the `top`-th
// largest of them; a row of random logits has about 1.6 times as many that do. Those, as keys of value and index, are
// collected in any order and then put into their places by counting, for each, the keys above it, so results do not depend
// on the order. Rows with more than LP_KEYS of them (equal logits, fewer tokens left than are asked for) look for one
// maximum after the other instead, in as many passes (8,191 rows of 32,000 with 5 tokens left, 20 largest: 5.7 ms).
#include <cooperative_groups.h>

#include "kie_device.cuh"
#include "kie_paged.cuh"

namespace kie {
namespace {

namespace cg = cooperative_groups;

// Threads of a block: small ones where there are rows enough, so that the waits at the end of a row concern few warps at a
// time (8,191 rows of 32,000 bf16 logits, 20 largest, at the time: 122 us with 128 threads, 131 with 256).
constexpr int LP_FEW = 256, LP_MANY = 128;
constexpr int LP_AHEAD = 4;  // 16-byte pieces of a row that a thread has on their way
constexpr float LP_STEP = 4.f;  // the reference moves when the maximum passes it by more
constexpr int LP_GROUPS = 64;  // of threads
constexpr int LP_KEYS = 512, LP_LIST = 1024;
constexpr int LP_CLUSTER = 8;
constexpr float LP_LEAST = -1e4f;  // a distance from the maximum with a weight of 0 that may be multiplied with it
constexpr float LOG2E = 1.4426950408889634f;

using Key = unsigned long long;

// A logit as an unsigned integer of the same order, NaN above +inf and -0 as 0.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t order) {
  return order == 0xffffffffu ? __uint_as_float(0x7fc00000u) : __uint_as_float(order & 0x80000000u ? order ^ 0x80000000u : ~order);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes of a row: N elements of type X.
template <int X>
struct Piece {
  static constexpr int N = X == KIE_F32 ? 4 : 8, SIZE = 16 / N;
  static constexpr uint32_t NONE = X == KIE_F32 ? 0xff800000u : X == KIE_F16 ? 0xfc00fc00u : 0xff80ff80u;  // -inf, or two
  uint32_t w[4];
  __device__ __forceinline__ float get(int e) const {
    if (X == KIE_F32) return __uint_as_float(w[e & 3]);
    if (X == KIE_F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[(e >> 1) & 3]));
      return e & 1 ? f.y : f.x;
    }
    return __uint_as_float(e & 1 ? w[(e >> 1) & 3] & 0xffff0000u : w[(e >> 1) & 3] << 16);
  }
  // Elements at .. at + N - 1 of a row of V one by one, those outside it as -inf.
  static __device__ __noinline__ uint4 gather(const uint8_t *row, int at, int V) {
    uint32_t w[4] = {NONE, NONE, NONE, NONE};
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if (at + e < 0 || at + e >= V) continue;
      const uint8_t *p = row + (int64_t)(at + e) * SIZE;
      if (X == KIE_F32)
        w[e & 3] = *reinterpret_cast<const uint32_t *>(p);
      else
        w[(e >> 1) & 3] = __byte_perm(w[(e >> 1) & 3], *reinterpret_cast<const uint16_t *>(p), e & 1 ? 0x5410 : 0x3254);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // Against a row's maximum from LOW up, what pair() makes of -inf has a weight of 0.
  static constexpr float LOW = X == KIE_F16 ? -65000.f : -1e37f;
  // The elements, two by two, none below a finite value.
  __device__ __forceinline__ float2 pair(int k) const {
    if (X == KIE_F32) return make_float2(fmaxf(get(2 * k), -1e38f), fmaxf(get(2 * k + 1), -1e38f));
    if (X == KIE_F16) return __half22float2(__hmax2(*reinterpret_cast<const __half2 *>(&w[k & 3]), __float2half2_rn(-65504.f)));
    const __nv_bfloat162 b = __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&w[k & 3]), __float2bfloat162_rn(-1e38f));
    const uint32_t u = *reinterpret_cast<const uint32_t *>(&b);
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  // This one's elements or y's, whichever is larger at each place, NaN if one is.
  __device__ __forceinline__ void raise(const Piece &y) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (X == KIE_F32) {
        float f = __uint_as_float(w[k]);
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(f) : "f"(__uint_as_float(y.w[k])));
        w[k] = __float_as_uint(f);
      } else if (X == KIE_F16) {
        const __half2 h = __hmax2_nan(*reinterpret_cast<const __half2 *>(&w[k]), *reinterpret_cast<const __half2 *>(&y.w[k]));
        w[k] = *reinterpret_cast<const uint32_t *>(&h);
      } else {
        const __nv_bfloat162 h =
            __hmax2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&w[k]), *reinterpret_cast<const __nv_bfloat162 *>(&y.w[k]));
        w[k] = *reinterpret_cast<const uint32_t *>(&h);
      }
    }
  }
  // The largest element, NaN if there is one.
  __device__ __forceinline__ float most() const {
    if (X == KIE_F32) {
      float m = get(0);
#pragma unroll
      for (int e = 1; e < 4; ++e) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(get(e)));
      return m;
    }
    if (X == KIE_F16) {
      const __half2 *h = reinterpret_cast<const __half2 *>(w);
      const __half2 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
      return __half2float(__hmax_nan(__low2half(m), __high2half(m)));
    }
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(w);
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
    return __bfloat162float(__hmax_nan(__low2bfloat16(m), __high2bfloat16(m)));
  }
};

// Two fp32 operations at a time.
__device__ __forceinline__ unsigned long long two(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 both(unsigned long long r) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(r));
  return f;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

struct LpSmem {
  alignas(16) uint32_t group[LP_GROUPS];  // maxima
  uint32_t list[LP_LIST];     // rounds of threads that have elements which reach the bound, or may: thread | round << 8
  int n_list;
  float2 sums[LP_FEW / 32];
  uint32_t bound;
  Key warp_best[LP_FEW / 32];
  // of the cluster, in its first block:
  float2 block_sums[LP_CLUSTER];
  Key block_best[LP_CLUSTER];
  int n_keys;
  Key keys[LP_KEYS];
};

// One row to a cluster (or a block), per_block pieces of it to each block.
template <int X, bool CLUSTER>
__global__ void __launch_bounds__(CLUSTER ? LP_FEW : LP_MANY, CLUSTER ? 4 : 10) token_logprobs_kernel(const kie_token_logprobs_args a, int per_block) {
  using P = Piece<X>;
  constexpr int LP_THREADS = CLUSTER ? LP_FEW : LP_MANY, LP_WARPS = LP_THREADS / 32, LP_GROUP = LP_THREADS / LP_GROUPS;
  __shared__ LpSmem sm;
  const cg::cluster_group cl = cg::this_cluster();
  const int blocks = CLUSTER ? cl.num_blocks() : 1, block = CLUSTER ? cl.block_rank() : 0;
  const int64_t row = CLUSTER ? blockIdx.x / blocks : blockIdx.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, V = a.vocab, top = a.top;
  const auto meet = [&] {
    if (CLUSTER)
      cl.sync();
    else
      __syncthreads();
  };
  LpSmem &first = CLUSTER ? *cl.map_shared_rank(&sm, 0) : sm;

  const uint8_t *base = static_cast<const uint8_t *>(a.logits) + row * a.row_stride * P::SIZE;
  const int skew = (int)((uintptr_t)base & 15) / P::SIZE;  // elements from the last 16-byte boundary to the row
  // piece v of the row holds elements v N - skew ..; this block has [v0, v1); pieces [whole0, whole1) lie inside the row
  const int pieces = (V + skew + P::N - 1) / P::N, v0 = min(block * per_block, pieces), v1 = min(v0 + per_block, pieces);
  const int whole0 = skew ? 1 : 0, whole1 = (V + skew) / P::N;
  const uint4 *const from = reinterpret_cast<const uint4 *>(base - skew * P::SIZE);
  // Thread i takes every LP_THREADS-th of the places [u0 + i, u1): the pieces from the first whole one on, and behind them
  // the row's first piece where it is none.
  const int u0 = max(v0, whole0), u1 = v1 + (v0 == 0 && whole0 && v1 > 0 ? 1 : 0);
  const auto piece_of = [&](int u) { return u == v1 ? 0 : u; };
  const auto fetch = [&](int u) {
    uint4 w = make_uint4(P::NONE, P::NONE, P::NONE, P::NONE);
    if (u < min(v1, whole1))
      w = __ldcg(from + u);
    else if (u < u1)
      w = P::gather(base, piece_of(u) * P::N - skew, V);
    P x;
    x.w[0] = w.x, x.w[1] = w.y, x.w[2] = w.z, x.w[3] = w.w;
    return x;
  };
  if (tid == 0) sm.n_keys = sm.n_list = 0;
  begin_after_previous();
  float asked = 0.f;
  int token = -1;
  if (tid == 0 && block == 0 && a.logprob) {
    token = a.tokens[row];
    if ((unsigned)token < (unsigned)V) {
      const uint8_t *p = base + (int64_t)token * P::SIZE;
      asked = X == KIE_F32   ? *reinterpret_cast<const float *>(p)
              : X == KIE_F16 ? __half2float(*reinterpret_cast<const __half *>(p))
                             : __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(p));
    }
  }

  // ---- the thread's pieces: their maximum and sums
  float ref = 0.f, most = -INFINITY, next_most = -INFINITY;  // the largest maximum of a round, and the second
  int most_round = 0;
  bool any = false, far = false;  // there is a reference; it, or an element, is too large for differences in fp32
  unsigned long long s2[2] = {0, 0}, t2[2] = {0, 0}, minus = 0;
  const unsigned long long unit = two(LOG2E, LOG2E);
  const auto take = [&](const P(&x)[LP_AHEAD], int round) {
    P up = x[0];
#pragma unroll
    for (int k = 1; k < LP_AHEAD; ++k) up.raise(x[k]);
    const float high = up.most();
    if (!(high <= most)) {
      next_most = most;
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(most) : "f"(high));  // a NaN stays, and from the next round on next_most is one too
      most_round = round;
    } else if (high > next_most) {
      next_most = high;
    }
    if (!(high <= ref + LP_STEP) || !any) {  // seldom but for the first time
      far = far || (!(fabsf(high) < 1e37f) && high != -INFINITY);
      if (high != -INFINITY && !far) {
        // t + s (old - new reference), s, both times f. s times a distance whose f is 0 shall be finite
        const float by = any ? fmaxf(ref - high, LP_LEAST) : 0.f, f = ex2(by * LOG2E);
        const unsigned long long f2 = two(f, f), by2 = two(by, by);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          t2[k] = mul2(fma2(s2[k], by2, t2[k]), f2);
          s2[k] = mul2(s2[k], f2);
        }
        ref = high;
        minus = two(-ref, -ref);
        any = true;
      }
    }
#pragma unroll
    for (int k = 0; k < LP_AHEAD; ++k)
#pragma unroll
      for (int e = 0; e < P::N / 2; ++e) {
        const float2 f = x[k].pair(e);
        const unsigned long long d = add2(two(f.x, f.y), minus);
        const float2 g = both(mul2(d, unit));
        const unsigned long long w = two(ex2(g.x), ex2(g.y));
        s2[e & 1] = add2(s2[e & 1], w);
        t2[e & 1] = fma2(w, d, t2[e & 1]);
      }
  };
  const int rounds = max(0, min(v1, whole1) - u0) / (LP_AHEAD * LP_THREADS);  // without an end in them
  {
    const uint4 *at = from + u0 + tid;
#pragma unroll 1
    for (int r = 0; r < rounds; ++r, at += LP_AHEAD * LP_THREADS) {
      P x[LP_AHEAD];
#pragma unroll
      for (int k = 0; k < LP_AHEAD; ++k) {
        const uint4 w = __ldcg(at + k * LP_THREADS);
        x[k].w[0] = w.x, x[k].w[1] = w.y, x[k].w[2] = w.z, x[k].w[3] = w.w;
      }
      take(x, r);
    }
  }
  const int all_rounds = (max(0, u1 - u0) + LP_AHEAD * LP_THREADS - 1) / (LP_AHEAD * LP_THREADS);
#pragma unroll 1
  for (int r = rounds; r < all_rounds; ++r) {
    P x[LP_AHEAD];
#pragma unroll
    for (int k = 0; k < LP_AHEAD; ++k) x[k] = fetch(u0 + tid + (r * LP_AHEAD + k) * LP_THREADS);
    take(x, r);
  }
  const uint32_t mine = order_of(most);
  // ---- the row's maximum, and a bound that the `top` largest reach
  uint32_t group = mine;
#pragma unroll
  for (int o = LP_GROUP / 2; o; o >>= 1) group = max(group, __shfl_xor_sync(0xffffffffu, group, o));
  if (tid % LP_GROUP == 0) sm.group[tid / LP_GROUP] = group;
  meet();
  uint32_t best = 0;
  if constexpr (CLUSTER) {
    uint32_t all[LP_CLUSTER], y[LP_CLUSTER];  // lane i: groups i and i + 32 of each block
#pragma unroll
    for (int b = 0; b < LP_CLUSTER; ++b) {  // no condition: the loads are on their way together
      const uint32_t *g = cl.map_shared_rank(&sm, min(b, blocks - 1))->group;
      all[b] = g[lane], y[b] = g[lane + 32];
    }
#pragma unroll
    for (int b = 0; b < LP_CLUSTER; ++b) {
      all[b] = b < blocks ? max(all[b], y[b]) : 0u;
      best = max(best, all[b]);
    }
    if (top > 0 && warp == 0) {
      uint32_t bound = 0;  // its upper 16 bits: of bf16 logits all there is
#pragma unroll 1
      for (uint32_t bit = 0x80000000u; bit > 0x8000u; bit >>= 1) {
        int n = 0;
#pragma unroll
        for (int b = 0; b < LP_CLUSTER; ++b) n += __popc(__ballot_sync(0xffffffffu, all[b] >= (bound | bit)));
        if (n >= top) bound |= bit;
      }
      if (lane == 0) sm.bound = bound;
    }
  } else {
    best = max(sm.group[lane], sm.group[lane + 32]);
    if (top > 0) {  // the group with top - 1 others above it
      constexpr int PARTS = LP_THREADS / LP_GROUPS;
      const int g = tid / PARTS, part = tid % PARTS;
      const uint32_t own = sm.group[g];
      int above = 0;
#pragma unroll 4
      for (int k = 0; k < LP_GROUPS / PARTS; k += 4) {
        const int at = part * (LP_GROUPS / PARTS) + k;
        const uint4 y = *reinterpret_cast<const uint4 *>(&sm.group[at]);
        above += (y.x > own || (y.x == own && at < g)) + (y.y > own || (y.y == own && at + 1 < g)) +
                 (y.z > own || (y.z == own && at + 2 < g)) + (y.w > own || (y.w == own && at + 3 < g));
      }
#pragma unroll
      for (int o = 1; o < PARTS; o <<= 1) above += __shfl_xor_sync(0xffffffffu, above, o);
      if (above == top - 1) sm.bound = own;
    }
  }
  best = __reduce_max_sync(0xffffffffu, best);
  const float m = value_of(best), base_m = m == -INFINITY ? 0.f : m;
  // ---- the sums at the row's maximum
  float s = 0.f, t = 0.f;
  // once more where differences may leave the range, where there is an infinity or NaN, and where -inf has counted
  if (!(base_m >= P::LOW && base_m < 1e37f) || far) {
#pragma unroll 1
    for (int u = u0 + tid; u < u1; u += LP_THREADS) {
      const P x = fetch(u);
#pragma unroll
      for (int e = 0; e < P::N; ++e) {
        const float d = fmaxf(x.get(e) - base_m, LP_LEAST), w = ex2(d * LOG2E);
        s += w;
        t = fmaf(w, d, t);
      }
    }
  } else if (any) {
    const float2 f = both(add2(s2[0], s2[1])), g = both(add2(t2[0], t2[1]));
    const float by = ref - base_m, factor = ex2(by * LOG2E);
    s = f.x + f.y;
    t = fmaf(s, fmaxf(by, LP_LEAST), g.x + g.y) * factor;
    s *= factor;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o), t += __shfl_xor_sync(0xffffffffu, t, o);
  if (lane == 0) sm.sums[warp] = make_float2(s, t);
  __syncthreads();
  // ---- the elements that reach the bound: the rounds that have some are read again, half a piece to a lane, four rounds of
  // a thread to a warp
  if (top > 0) {
    const uint32_t bound = sm.bound;
    const float least = value_of(bound);
    if (mine >= bound) {
      const bool more = !(next_most < least);  // which rounds is not known
      for (int r = more ? 0 : most_round; r < (more ? all_rounds : most_round + 1); ++r) {
        const int at = atomicAdd(&sm.n_list, 1);
        if (at >= LP_LIST) break;
        sm.list[at] = tid | r << 8;
      }
    }
    __syncthreads();
    const int n_list = sm.n_list;
    static_assert(LP_AHEAD * 2 * 4 == 32 && LP_THREADS <= 256, "a round is eight lanes' work; a thread's number takes 8 bits");
    if (n_list > LP_LIST) {
      if (tid == 0) atomicAdd(&first.n_keys, LP_KEYS + 1);
    } else {
#pragma unroll 1
      for (int e = warp * 4 + (lane >> 3); e < n_list; e += 8 * LP_WARPS) {
        P x[2];
        int u[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t who = sm.list[min(e + i * 4 * LP_WARPS, n_list - 1)];
          u[i] = e + i * 4 * LP_WARPS < n_list ? u0 + ((who >> 8) * LP_AHEAD + (lane >> 1 & 3)) * LP_THREADS + (who & 255u) : u1;
          x[i] = fetch(u[i]);
        }
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          P h = x[0];
          const int v = u[0];
          x[0] = x[1], u[0] = u[1];
          if (lane & 1) h.w[0] = h.w[2], h.w[1] = h.w[3];
          h.w[2] = h.w[0], h.w[3] = h.w[1];
          if (h.most() < least || v >= u1) continue;
          const int id0 = piece_of(v) * P::N - skew + (lane & 1) * (P::N / 2);
#pragma unroll 1
          for (int k = 0; k < P::N / 2; ++k) {
            const float y = h.get(0);
            const int id = id0 + k;
            if (P::SIZE == 4)  // the next one
              h.w[0] = h.w[1];
            else
              h.w[0] = h.w[0] >> 16 | h.w[1] << 16, h.w[1] >>= 16;
            if (y < least || id < 0 || id >= V) continue;
            const int at = atomicAdd(&first.n_keys, 1);
            if (at >= LP_KEYS) break;
            first.keys[at] = (Key)order_of(y) << 32 | (uint32_t)~id;
          }
        }
      }
    }
  }
  if (warp == 0) {
    float2 y = lane < LP_WARPS ? sm.sums[lane] : make_float2(0.f, 0.f);
#pragma unroll
    for (int o = LP_WARPS / 2; o; o >>= 1)
      y.x += __shfl_xor_sync(0xffffffffu, y.x, o), y.y += __shfl_xor_sync(0xffffffffu, y.y, o);
    if (lane == 0) first.block_sums[block] = y;
  }
  meet();
  // ---- results, by the first block
  const int n = first.n_keys;
  const bool many = n > LP_KEYS;
  float ls = 0.f;
  if (block == 0) {
    float ss = 0.f, tt = 0.f;
    for (int b = 0; b < blocks; ++b) ss += sm.block_sums[b].x, tt += sm.block_sums[b].y;
    // nothing left: ln p = -inf, entropy 0; NaN or +inf: NaN
    const bool none = m == -INFINITY, bad = !(m < INFINITY);
    ls = none ? INFINITY : bad ? __uint_as_float(0x7fc00000u) : logf(ss);
    if (tid == 0) {
      if (a.entropy) a.entropy[row] = none ? 0.f : ls - tt / ss;
      if (a.logprob) a.logprob[row] = (unsigned)token >= (unsigned)V ? 0.f : asked - base_m - ls;
    }
    if (!many)
      for (int i = warp; i < n; i += LP_WARPS) {  // the place of a key: as many are above it
        const Key key = sm.keys[i];
        int above = 0;
        for (int k = 0; k < n; k += 32) above += __popc(__ballot_sync(0xffffffffu, k + lane < n && sm.keys[k + lane] > key));
        if (above >= top || lane) continue;
        a.top_ids[row * top + above] = (int)~(uint32_t)key;
        a.top_logprobs[row * top + above] = value_of((uint32_t)(key >> 32)) - base_m - ls;
      }
  }
  if (many) {  // the same in every block
    Key last = ~0ull;
    for (int k = 0; k < top; ++k) {
      Key next = 0;
#pragma unroll 1
      for (int u = u0 + tid; u < u1; u += LP_THREADS) {
        const P x = fetch(u);
#pragma unroll
        for (int e = 0; e < P::N; ++e) {
          const int id = piece_of(u) * P::N - skew + e;
          const Key key = (Key)order_of(x.get(e)) << 32 | (uint32_t)~id;
          if ((k == 0 || key < last) && key > next && id >= 0 && id < V) next = key;  // a NaN at id 0 is the largest key there is
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) next = max(next, __shfl_xor_sync(0xffffffffu, next, o));
      if (lane == 0) sm.warp_best[warp] = next;
      __syncthreads();
      if (tid == 0) {
        for (int w = 0; w < LP_WARPS; ++w) next = max(next, sm.warp_best[w]);
        first.block_best[block] = next;
      }
      meet();
      last = 0;
      for (int b = 0; b < blocks; ++b) last = max(last, first.block_best[b]);
      if (block == 0 && tid == 0) {
        a.top_ids[row * top + k] = (int)~(uint32_t)last;
        a.top_logprobs[row * top + k] = value_of((uint32_t)(last >> 32)) - base_m - ls;
      }
      meet();  // read before the next round writes
    }
  }
  if (CLUSTER) cl.sync();  // the first block's memory is read until here
}

template <int X>
cudaError_t launch(const kie_token_logprobs_args &a, int sms, cudaStream_t stream) {
  using P = Piece<X>;
  const int pieces = a.vocab / P::N + 2;  // of a row at most
  // Rows that leave SMs idle are split, as long as every thread of a block has a piece.
  int blocks = 1;
  while (blocks < LP_CLUSTER && (int64_t)a.n_rows * blocks * 2 <= sms && pieces >= 2 * blocks * LP_FEW) blocks *= 2;
  const int per_block = (pieces + blocks - 1) / blocks;
  auto *const kernel = blocks > 1 ? token_logprobs_kernel<X, true> : token_logprobs_kernel<X, false>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.n_rows * blocks));
  cfg.blockDim = dim3(blocks > 1 ? LP_FEW : LP_MANY);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = blocks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = blocks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, per_block);
}

}  // namespace
}  // namespace kie

cudaError_t kie_launch_token_logprobs(const kie_token_logprobs_args &a, int sms, cudaStream_t stream) {
  return a.dtype == KIE_F32   ? kie::launch<KIE_F32>(a, sms, stream)
         : a.dtype == KIE_F16 ? kie::launch<KIE_F16>(a, sms, stream)
                              : kie::launch<KIE_BF16>(a, sms, stream);
}
