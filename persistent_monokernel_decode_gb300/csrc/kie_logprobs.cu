// Log probabilities of tokens, entropies and the largest logits (kie_paged.cu holds the C entry).
//
// A row is read once, into shared memory: a block holds up to 64 KB of it, brought by bulk copies, and longer rows, or rows
// too few to fill the GPU, are split over a cluster of up to eight blocks that meet at the cluster's barrier and pass their
// results through distributed shared memory. (Rows of more than 512 KB are read again for each pass.) Passes over the row
// are short loops: held in registers and unrolled, as it was first, the row took 22 instructions an element and most of the
// time to fetch them. With the maximum of the row as the reference, s = sum exp(x - m) and t = sum exp(x - m) (x - m):
// ln p = x - m - ln s, and the entropy is ln s - t / s, which stays accurate where x itself is large.
//
// The `top` largest: the maxima of groups of threads give a bound that at least `top` elements reach, the `top`-th
// largest of them; a row of random logits has about 1.6 times as many that do. Those, as keys of value and index, are
// collected in any order and then put into their places by counting, for each, the keys above it, so results do not depend
// on the order. Rows with more than LP_KEYS of them (equal logits, fewer tokens left than are asked for) look for one
// maximum after the other instead.
#include <cooperative_groups.h>

#include <limits.h>

#include <algorithm>
#include <atomic>

#include "kie_device.cuh"
#include "kie_paged.cuh"

namespace kie {
namespace {

namespace cg = cooperative_groups;

#ifndef LPT
#define LPT 256
#endif
constexpr int LP_THREADS = LPT, LP_WARPS = LP_THREADS / 32;
constexpr int LP_PIECES = 4096;  // 16-byte pieces of a row that a block holds: three blocks to an SM
constexpr int LP_GROUPS = 32, LP_GROUP = LP_THREADS / LP_GROUPS;  // of threads
constexpr int LP_KEYS = 512;
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
  __device__ void gather(const uint8_t *row, int at, int V) {
    constexpr uint32_t NONE = X == KIE_F32 ? 0xff800000u : X == KIE_F16 ? 0xfc00fc00u : 0xff80ff80u;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = NONE;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if (at + e < 0 || at + e >= V) continue;
      const uint8_t *p = row + (int64_t)(at + e) * SIZE;
      if (X == KIE_F32)
        w[e & 3] = *reinterpret_cast<const uint32_t *>(p);
      else
        w[(e >> 1) & 3] = __byte_perm(w[(e >> 1) & 3], *reinterpret_cast<const uint16_t *>(p), e & 1 ? 0x5410 : 0x3254);
    }
  }
  // The elements, two by two, none below a finite value whose weight is 0 (against a maximum above -10^37).
  __device__ __forceinline__ float2 pair(int k) const {
    if (X == KIE_F32) return make_float2(fmaxf(get(2 * k), -1e38f), fmaxf(get(2 * k + 1), -1e38f));
    if (X == KIE_F16) return __half22float2(__hmax2(*reinterpret_cast<const __half2 *>(&w[k & 3]), __float2half2_rn(-65504.f)));
    const __nv_bfloat162 b = __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&w[k & 3]), __float2bfloat162_rn(-1e38f));
    const uint32_t u = *reinterpret_cast<const uint32_t *>(&b);
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  // The largest element, NaN if there is one.
  __device__ __forceinline__ float top() const {
    if (X == KIE_F32) {
      float m;
      asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(get(0)), "f"(get(1)));
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(get(2)));
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(get(3)));
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
  uint64_t full;
  int failed;
  uint32_t group[LP_GROUPS];  // maxima
  float2 sums[LP_WARPS];
  uint32_t bound;
  Key warp_best[LP_WARPS];
  // of the cluster, in its first block:
  float2 block_sums[LP_CLUSTER];
  Key block_best[LP_CLUSTER];
  int n_keys;
  Key keys[LP_KEYS];
};

constexpr unsigned long long LP_TIMEOUT_NS = 2000000000ull;

// One row to a cluster (or a block), loaded in `rounds` parts of LP_PIECES pieces: one, unless the row is very long.
template <int X, bool CLUSTER>
__global__ void __launch_bounds__(LP_THREADS, 3) token_logprobs_kernel(const kie_token_logprobs_args a, int per_block, int rounds) {
  using P = Piece<X>;
  extern __shared__ __align__(128) uint8_t lp_raw[];
  __shared__ LpSmem sm;
  P *const held = reinterpret_cast<P *>(lp_raw);
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
  if (tid == 0) {
    mbar_init(&sm.full, 1);
    fence_barrier_init();
    sm.n_keys = 0;
    sm.failed = 0;
  }
  begin_after_previous();
  __syncthreads();
  int loads = 0, held0 = 0, n_held = 0;  // pieces held0 .. of the row are there
  const auto load = [&](int round) {
    if (loads) {  // everybody is done with the last part
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncthreads();
    }
    held0 = v0 + round * LP_PIECES;
    n_held = max(0, min(v1 - held0, LP_PIECES));
    const int b = max(held0, whole0), e = min(held0 + n_held, whole1), bytes = max(0, e - b) * 16;
    if (tid == 0) {
      mbar_arrive_expect_tx(&sm.full, bytes);
      for (int at = 0; at < bytes; at += 16384)
        bulk_g2s(lp_raw + (b - held0) * 16 + at, base + ((int64_t)b * P::N - skew) * P::SIZE + at, min(16384, bytes - at), &sm.full,
                 l2_evict_first_policy());
    }
    if (held0 == 0 && whole0 == 1 && n_held > 0 && tid == 32) held[0].gather(base, -skew, V);
    if (whole1 < pieces && whole1 >= max(held0, whole0) && whole1 < held0 + n_held && tid == 64)
      held[whole1 - held0].gather(base, whole1 * P::N - skew, V);
    if (!mbar_try_wait(&sm.full, loads & 1)) {
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait(&sm.full, loads & 1))
        if (globaltimer() - t0 > LP_TIMEOUT_NS) {
          sm.failed = 1;
          break;
        }
    }
    ++loads;
    if (whole0 == 1 || whole1 < pieces) __syncthreads();  // the pieces put together by hand
  };
  load(0);
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

  // ---- the maximum, and a bound that the `top` largest reach
  uint32_t mine = 0;
  for (int r = 0; r < rounds; ++r) {
    if (r) load(r);
#pragma unroll 4
    for (int i = tid; i < n_held; i += LP_THREADS) mine = max(mine, order_of(held[i].top()));
  }
  uint32_t group = mine;
#pragma unroll
  for (int o = LP_GROUP / 2; o; o >>= 1) group = max(group, __shfl_xor_sync(0xffffffffu, group, o));
  if (tid % LP_GROUP == 0) sm.group[tid / LP_GROUP] = group;
  meet();
  uint32_t best = 0, all[CLUSTER ? LP_CLUSTER : 1];  // lane i: group i of each block
#pragma unroll
  for (int b = 0; b < (CLUSTER ? LP_CLUSTER : 1); ++b) {
    all[b] = 0;
    if (b < blocks) all[b] = CLUSTER ? cl.map_shared_rank(&sm, b)->group[lane] : sm.group[lane];
    best = max(best, all[b]);
  }
  best = __reduce_max_sync(0xffffffffu, best);
  const float m = value_of(best), ref = m == -INFINITY ? 0.f : m;
  if (top > 0 && warp == 0) {
    uint32_t bound = 0;  // its upper 16 bits: of bf16 logits all there is
#pragma unroll 1
    for (uint32_t bit = 0x80000000u; bit > 0x8000u; bit >>= 1) {
      int n = 0;
#pragma unroll
      for (int b = 0; b < (CLUSTER ? LP_CLUSTER : 1); ++b) n += __popc(__ballot_sync(0xffffffffu, all[b] >= (bound | bit)));
      if (n >= top) bound |= bit;
    }
    if (lane == 0) sm.bound = bound;
  }
  // ---- the sums
  float s, t;
  if (fabsf(ref) < 1e37f) {
    unsigned long long s2[2] = {0, 0}, t2[2] = {0, 0};
    const unsigned long long minus = two(-ref, -ref), unit = two(LOG2E, LOG2E);
    for (int r = 0; r < rounds; ++r) {
      if (rounds > 1) load(r);
#pragma unroll 2
      for (int i = tid; i < n_held; i += LP_THREADS) {
        const P x = held[i];
#pragma unroll
        for (int k = 0; k < P::N / 2; ++k) {
          const float2 f = x.pair(k);
          const unsigned long long d = add2(two(f.x, f.y), minus);
          const float2 g = both(mul2(d, unit));
          const unsigned long long w = two(ex2(g.x), ex2(g.y));
          s2[k & 1] = add2(s2[k & 1], w);
          t2[k & 1] = fma2(w, d, t2[k & 1]);
        }
      }
    }
    const float2 f = both(add2(s2[0], s2[1])), g = both(add2(t2[0], t2[1]));
    s = f.x + f.y, t = g.x + g.y;
  } else {  // differences may leave the range, or there is an infinity or NaN
    s = t = 0.f;
    for (int r = 0; r < rounds; ++r) {
      if (rounds > 1) load(r);
#pragma unroll 1
      for (int i = tid; i < n_held; i += LP_THREADS) {
        const P x = held[i];
#pragma unroll
        for (int e = 0; e < P::N; ++e) {
          const float d = fmaxf(x.get(e) - ref, LP_LEAST), w = ex2(d * LOG2E);
          s += w;
          t = fmaf(w, d, t);
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o), t += __shfl_xor_sync(0xffffffffu, t, o);
  if (lane == 0) sm.sums[warp] = make_float2(s, t);
  __syncthreads();
  // ---- the elements that reach the bound
  const uint32_t bound = sm.bound;
  const float least = value_of(bound);
  for (int r = 0; top > 0 && r < rounds; ++r) {
    if (rounds > 1) load(r);
    bool room = mine >= bound;
#pragma unroll 1
    for (int i = tid; i < n_held && room; i += LP_THREADS) {
      const P x = held[i];
      if (x.top() < least) continue;
#pragma unroll
      for (int e = 0; e < P::N; ++e) {
        const float y = x.get(e);
        const int id = (held0 + i) * P::N - skew + e;
        if (y < least || id < 0 || id >= V || !room) continue;
        const int at = atomicAdd(&first.n_keys, 1);
        room = at < LP_KEYS;
        if (room) first.keys[at] = (Key)order_of(y) << 32 | (uint32_t)~id;
      }
    }
  }
  if (warp == 0) {
    float2 y = lane < LP_WARPS ? sm.sums[lane] : make_float2(0.f, 0.f);
#pragma unroll
    for (int o = LP_WARPS / 2; o; o >>= 1)
      y.x += __shfl_xor_sync(0xffffffffu, y.x, o), y.y += __shfl_xor_sync(0xffffffffu, y.y, o);
    // a copy that did not come shows as NaN
    if (lane == 0) first.block_sums[block] = sm.failed ? make_float2(__uint_as_float(0x7fc00000u), 0.f) : y;
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
      if (a.logprob) a.logprob[row] = (unsigned)token >= (unsigned)V ? 0.f : asked - ref - ls;
    }
    if (!many)
      for (int i = tid; i < n; i += LP_THREADS) {
        const Key key = sm.keys[i];
        int above = 0;
#pragma unroll 4
        for (int k = 0; k < n; ++k) above += sm.keys[k] > key;
        if (above >= top) continue;
        a.top_ids[row * top + above] = (int)~(uint32_t)key;
        a.top_logprobs[row * top + above] = value_of((uint32_t)(key >> 32)) - ref - ls;
      }
  }
  if (many) {  // the same in every block
    Key last = ~0ull;
    for (int k = 0; k < top; ++k) {
      Key next = 0;
      for (int r = 0; r < rounds; ++r) {
        if (rounds > 1) load(r);
#pragma unroll 1
        for (int i = tid; i < n_held; i += LP_THREADS) {
          const P x = held[i];
#pragma unroll
          for (int e = 0; e < P::N; ++e) {
            const int id = (held0 + i) * P::N - skew + e;
            const Key key = (Key)order_of(x.get(e)) << 32 | (uint32_t)~id;
            if (key < last && key > next && id >= 0 && id < V) next = key;
          }
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
        a.top_logprobs[row * top + k] = value_of((uint32_t)(last >> 32)) - ref - ls;
      }
      meet();  // read before the next round writes
    }
  }
  if (CLUSTER) cl.sync();  // the first block's memory is read until here
}

template <int X>
cudaError_t launch(const kie_token_logprobs_args &a, int dev, int sms, cudaStream_t stream) {
  using P = Piece<X>;
  const int pieces = a.vocab / P::N + 2;  // of a row at most
  // A block to a row, or as many as it takes to hold it. Rows that leave SMs idle are split further, as long as every thread
  // of a block has a piece.
  int blocks = 1;
  while (blocks < LP_CLUSTER &&
         (blocks * LP_PIECES < pieces || ((int64_t)a.n_rows * blocks * 2 <= sms && pieces >= 2 * blocks * LP_THREADS)))
    blocks *= 2;
  const int per_block = (pieces + blocks - 1) / blocks, rounds = (per_block + LP_PIECES - 1) / LP_PIECES;
  if ((int64_t)a.n_rows * blocks > INT_MAX) return cudaErrorInvalidValue;
  auto *const kernel = blocks > 1 ? token_logprobs_kernel<X, true> : token_logprobs_kernel<X, false>;
  static std::atomic<uint64_t> ready[2];  // devices whose limit of dynamic shared memory is raised
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (!bit || !(ready[blocks > 1].load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, LP_PIECES * 16);
    if (e != cudaSuccess) return e;
    ready[blocks > 1].fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.n_rows * blocks));
  cfg.blockDim = dim3(LP_THREADS);
  cfg.dynamicSmemBytes = std::min(per_block, LP_PIECES) * 16;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = blocks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = blocks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, per_block, rounds);
}

}  // namespace
}  // namespace kie

cudaError_t kie_launch_token_logprobs(const kie_token_logprobs_args &a, int dev, int sms, cudaStream_t stream) {
  return a.dtype == KIE_F32   ? kie::launch<KIE_F32>(a, dev, sms, stream)
         : a.dtype == KIE_F16 ? kie::launch<KIE_F16>(a, dev, sms, stream)
                              : kie::launch<KIE_BF16>(a, dev, sms, stream);
}
