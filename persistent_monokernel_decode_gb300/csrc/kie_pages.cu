// Pages that several sequences share: forks, compaction and copies (kie_paged.cu holds the C entries).
//
// Forks and compaction are short chains of passes over small integer arrays, each of which needs the whole of the one
// before. Small ones are one launch of one block. Larger ones are two: what has to know everything comes first (each block
// of a fork plans for itself and copies its share of the rows; a compaction is one cluster of eight blocks, which meet at the
// cluster's hardware barrier, about a microsecond, and pass their counts through distributed shared memory), the rest, on
// every SM, in a second. Additions to a page's count commute and every list is written at ranks from scans, so results do not
// depend on the order in which blocks run. Bound by latency throughout.
#include <cooperative_groups.h>
#include <limits.h>

#include <algorithm>
#include <atomic>

#include "kie_device.cuh"
#include "kie_paged.cuh"

namespace kie {
namespace {

namespace cg = cooperative_groups;

constexpr int PS_THREADS = 1024, PS_WARPS = PS_THREADS / 32;
constexpr int PS_CLUSTER = 8;  // the portable most
// Up to these sizes (entries of the table, pages of the cache) one block does it all: a fork of 32 rows over a table of 2,336
// entries takes 8.2 us so and 8.8 in two launches, of 64 rows over 4,672 entries 9.9 and 9.8, of 128 over 16,512 13.9 and
// 8.9; a compaction of 512 pages 4.6 and 6.2, of 4,096 pages 6.7 and 7.2, of 16,384 16.0 and 8.2.
constexpr int PS_SMALL_TABLE = 4096, PS_SMALL_CACHE = 2048;

// Exclusive prefix of the flags over the block's threads, in thread order; *all gets their number. Every thread calls.
__device__ __forceinline__ int rank_of(bool flag, int *all) {
  __shared__ int s_warp[PS_WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned m = __ballot_sync(0xffffffffu, flag);
  __syncthreads();  // the last call's readers are done
  if (lane == 0) s_warp[warp] = __popc(m);
  __syncthreads();
  const int n = s_warp[lane];
  int up = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += x;
  }
  *all = __shfl_sync(0xffffffffu, up, 31);
  return __shfl_sync(0xffffffffu, up - n, warp) + __popc(m & ((1u << lane) - 1u));
}

// The sum of v over the block. Every thread calls.
__device__ __forceinline__ int block_sum(int v) {
  __shared__ int s_sum[PS_WARPS];
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, s_sum[threadIdx.x & 31]);
}

// The sum of every block's value (*all), and of those before this one. places, in shared memory, one for each block of the
// cluster, is not used again; it is written by the others, so that nobody reads from a block that may have ended. Every
// thread calls, in every block.
__device__ __forceinline__ int before_in_cluster(const cg::cluster_group &cl, int *places, int mine, int *all) {
  const int lane = threadIdx.x & 31, blocks = cl.num_blocks();
  if ((int)threadIdx.x < blocks) cl.map_shared_rank(places, threadIdx.x)[cl.block_rank()] = mine;
  cl.sync();
  const int v = lane < blocks ? places[lane] : 0;
  *all = __reduce_add_sync(0xffffffffu, v);
  return __reduce_add_sync(0xffffffffu, lane < (int)cl.block_rank() ? v : 0);
}

// f(j, from[j]) for j < n, the loads of four at a time on their way together: a warp.
template <class F>
__device__ __forceinline__ void for_each(const int *from, int n, const F &f) {
  for (int j0 = threadIdx.x & 31; j0 < n; j0 += 128) {
    int v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __ldcg(from + min(j0 + 32 * k, n - 1));
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (j0 + 32 * k < n) f(j0 + 32 * k, v[k]);
  }
}

// The i-th of `parts` equal ranges of n, its bounds multiples of 32.
__device__ __forceinline__ int range_begin(int n, int i, int parts) {
  const int per = ((n + parts - 1) / parts + 31) / 32 * 32;
  return (int)min((long long)i * per, (long long)n);
}

// ---- forks ---------------------------------------------------------------------------------------------------

__device__ __forceinline__ int parent_of(const ForkArgs &a, int r) {
  if (a.done) return a.done[r] ? -1 : r;
  const int p = a.parents[r];
  return p >= a.n_seqs ? r : max(p, -1);
}

// Pages of a row of length len, and whether the last is only filled in part.
__device__ __forceinline__ int pages_of(const ForkArgs &a, int len, bool *part) {
  const int n = len > 0 ? (int)(((unsigned)len + a.block_size - 1) / (unsigned)a.block_size) : 0;
  *part = len > 0 && len % a.block_size != 0 && n <= a.max_blocks;
  return min(n, a.max_blocks);
}

// What each row continues is the contents before the call, and rows change places: new table rows are staged in the
// workspace until every block has read the old ones.
// Returns the number of new pages that were taken, -1 if there are not enough.
__device__ __forceinline__ int plan_fork(const ForkArgs &a, int block, int blocks) {
  extern __shared__ int ps_raw[];
  const int R = a.n_seqs, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // of row p: how many rows continue it; which of them keeps its open page (-1: p itself, R: none); of row r: the rank of
  // its new page (-1: it needs none)
  const int n_free = min(max(*a.n_free, 0), a.free_capacity);
  int *kids = ps_raw, *keeper = ps_raw + R, *rank = ps_raw + 2 * R;
  for (int r = tid; r < R; r += PS_THREADS) kids[r] = 0, keeper[r] = R;
  __syncthreads();
  for (int r = tid; r < R; r += PS_THREADS) {
    const int p = parent_of(a, r);
    if (p < 0) continue;
    atomicAdd(&kids[p], 1);
    atomicMin(&keeper[p], p == r ? -1 : r);
  }
  __syncthreads();
  int total = 0;
  for (int r0 = 0; r0 < R; r0 += PS_THREADS) {
    const int r = r0 + tid;
    bool need = false;
    if (r < R) {
      const int p = parent_of(a, r);
      if (p >= 0 && p != r && keeper[p] != r) pages_of(a, a.lens[p], &need);
    }
    int all;
    const int k = rank_of(need, &all);
    if (r < R) rank[r] = need ? total + k : -1;
    total += all;
  }
  __syncthreads();
  const bool ok = total <= n_free;
  for (int r = block * PS_THREADS + tid; r < R; r += blocks * PS_THREADS) {
    const int p = ok ? parent_of(a, r) : r, len = p >= 0 ? a.lens[p] : 0;
    a.lens_out[r] = len;
    if (!a.copy_src) continue;
    const bool need = ok && rank[r] >= 0;
    a.copy_src[r] = need ? a.block_table[p * a.table_stride + len / a.block_size] : -1;
    a.copy_dst[r] = need ? a.free_blocks[n_free - 1 - rank[r]] : -1;
    a.copy_rows[r] = need ? len % a.block_size : 0;
  }
  if (block == 0 && tid == 0 && a.ok) *a.ok = ok;
  if (!ok) {  // the same in every block
    if (block == 0 && tid == 0) *a.n_free_out = *a.n_free;
    return -1;
  }
  int *staged = static_cast<int *>(a.workspace);
  for (int r = block * PS_WARPS + warp; r < R; r += blocks * PS_WARPS) {
    const int p = parent_of(a, r);
    bool part;
    if (p >= 0 && p != r) {
      const int n = pages_of(a, a.lens[p], &part);
      int *to = staged + (int64_t)r * a.max_blocks;
      for_each(a.block_table + p * a.table_stride, n, [&](int j, int x) { to[j] = x; });
      if (rank[r] >= 0 && lane == ((n - 1) & 31)) to[n - 1] = a.free_blocks[n_free - 1 - rank[r]];  // the lane that wrote it
    }
    if (kids[r] == 1) continue;  // its pages have as many holders as before
    const int n = pages_of(a, a.lens[r], &part);
    for_each(a.block_table + r * a.table_stride, n, [&](int j, int x) {
      const int change = (part && j == n - 1 ? min(kids[r], 1) : kids[r]) - 1;
      if (change && (unsigned)x < (unsigned)a.n_blocks) atomicAdd(&a.shares[x], change);
    });
  }
  if (block == 0 && tid == 0) *a.n_free_out = n_free - total;  // for now
  return total;
}

// After every block's plan_fork: pages that nobody holds any more go on the list, by the first cluster, and the rows change,
// by the others where there are any.
__device__ __forceinline__ void finish_fork(const ForkArgs &a, int left) {
  const cg::cluster_group cl = cg::this_cluster();
  const int R = a.n_seqs, tid = threadIdx.x, warp = tid >> 5;
  const int block = blockIdx.x, parts = cl.num_blocks(), first = gridDim.x > parts ? parts : 0, blocks = gridDim.x - first;
  int *staged = static_cast<int *>(a.workspace);
  for (int r = block < first ? R : (block - first) * PS_WARPS + warp; r < R; r += blocks * PS_WARPS) {
    const int p = parent_of(a, r);
    if (p < 0 || p == r) continue;
    bool part;
    int *to = a.block_table + r * a.table_stride;
    for_each(staged + (int64_t)r * a.max_blocks, pages_of(a, a.lens[p], &part), [&](int j, int x) { to[j] = x; });
  }
  if (block >= parts) return;
  __shared__ int s_freed[PS_CLUSTER];
  const int x0 = range_begin(a.n_blocks, block, parts), x1 = range_begin(a.n_blocks, block + 1, parts);
  int mine = 0, freed;
#pragma unroll 8
  for (int x = x0 + tid; x < x1; x += PS_THREADS) mine += __ldcg(&a.shares[x]) < 0;
  mine = block_sum(mine);
  long long to = left + before_in_cluster(cl, s_freed, mine, &freed);
  if (mine)
    for (int c0 = x0; c0 < x1; c0 += 4 * PS_THREADS) {
      bool free[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int x = c0 + k * PS_THREADS + tid;
        free[k] = x < x1 && __ldcg(&a.shares[x]) < 0;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int x = c0 + k * PS_THREADS + tid;
        int all;
        const int place = rank_of(free[k], &all);
        if (free[k]) {
          a.shares[x] = 0;
          if (to + place < a.free_capacity) a.free_blocks[to + place] = x;
        }
        to += all;
      }
    }
  if (block == 0 && tid == 0) *a.n_free_out = (int)min((long long)left + freed, (long long)a.free_capacity);
}

// One block.
__global__ void __launch_bounds__(PS_THREADS) paged_fork_kernel(const ForkArgs a) {
  begin_after_previous();
  const int total = plan_fork(a, 0, 1);
  __syncthreads();
  if (total >= 0) finish_fork(a, min(max(*a.n_free, 0), a.free_capacity) - total);
}

// The same in two launches, the second in clusters.
__global__ void __launch_bounds__(PS_THREADS) paged_fork_plan_kernel(const ForkArgs a) {
  begin_after_previous();
  plan_fork(a, blockIdx.x, gridDim.x);
}
__global__ void __launch_bounds__(PS_THREADS) paged_fork_finish_kernel(const ForkArgs a) {
  cg::this_cluster().sync();  // every block has begun, and others may write to its shared memory
  begin_after_previous();
  if (a.ok && !*a.ok) return;
  finish_fork(a, __ldcg(a.n_free_out));  // the cluster's barriers lie between this and its change
}


// ---- compaction ----------------------------------------------------------------------------------------------

// The rows' pages as they are numbered now.
__device__ __forceinline__ void rewrite_rows(const kie_paged_compact_args &a) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = a.n_blocks;
  const int block = blockIdx.x, blocks = gridDim.x;
  for (int r = block * PS_WARPS + warp; r < a.n_seqs; r += blocks * PS_WARPS) {
    const int len = a.lens[r];
    const int pages = len > 0 ? min((int)(((unsigned)len + a.block_size - 1) / (unsigned)a.block_size), a.max_blocks) : 0;
    int *row = a.block_table + r * a.table_stride;
    for (int j0 = lane; j0 < pages; j0 += 128) {
      int x[4], to[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = j0 + 32 * k < pages ? row[j0 + 32 * k] : -1;
#pragma unroll
      for (int k = 0; k < 4; ++k) to[k] = (unsigned)x[k] < (unsigned)n ? __ldcg(&a.page_map[x[k]]) : -1;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (to[k] >= 0 && to[k] != x[k]) row[j0 + 32 * k] = to[k];
    }
  }
}

// Live pages at and behind the number of live pages move into the free ones before it, both in the order of their ids. Each
// block keeps, for its range of pages, a bit to each in shared memory (set: free) and how many free ones lie before every 32:
// the list of free pages is read once, and everything else follows from the bits.
__global__ void __launch_bounds__(PS_THREADS) paged_compact_kernel(const kie_paged_compact_args a, int per, bool rows_too) {
  begin_after_previous();
  extern __shared__ int ps_raw[];
  __shared__ int s_free[PS_CLUSTER], s_below[PS_CLUSTER];
  const cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = a.n_blocks, most = n / 2;
  const int blocks = cl.num_blocks(), block = cl.block_rank(), all_tid = block * PS_THREADS + tid, all = blocks * PS_THREADS;
  const int x0 = (int)min((long long)block * per, (long long)n), x1 = (int)min((long long)x0 + per, (long long)n);
  cl.barrier_arrive();  // waited for before the first access to another block's memory: all of them have begun then
  const int words = per / 32;
  unsigned *bits = reinterpret_cast<unsigned *>(ps_raw);
  int *before = ps_raw + words;
  for (int w = tid; w < words; w += PS_THREADS) bits[w] = 0u;
  __syncthreads();
  const int n_free = min(max(*a.n_free, 0), a.free_capacity);
  // Every block reads the whole list for its own pages (an eighth of the bits set through distributed shared memory, by the
  // block that reads them, took 9 us where this takes 3)
  for (int i0 = tid; i0 < n_free; i0 += 8 * PS_THREADS) {
    int x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = i0 + k * PS_THREADS < n_free ? a.free_blocks[i0 + k * PS_THREADS] : -1;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (x[k] >= x0 && x[k] < x1) atomicOr(&bits[(x[k] - x0) >> 5], 1u << (x[k] & 31));
  }
  __syncthreads();
  // free pages before each word of this block, and in it
  int in_block = 0;
  for (int w0 = 0; w0 < words; w0 += PS_THREADS) {
    const int w = w0 + tid, c = w < words ? __popc(bits[w]) : 0;
    int up = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += y;
    }
    __shared__ int s_warp[PS_WARPS];
    __syncthreads();
    if (lane == 31) s_warp[warp] = up;
    __syncthreads();
    const int part = s_warp[lane];
    const int earlier = __reduce_add_sync(0xffffffffu, lane < warp ? part : 0), sum = __reduce_add_sync(0xffffffffu, part);
    if (w < words) before[w] = in_block + earlier + up - c;
    in_block += sum;
  }
  cl.barrier_wait();
  int free;
  const int first = before_in_cluster(cl, s_free, in_block, &free);  // of the blocks before
  const int live = n - free;
  __syncthreads();
  const auto free_before = [&](int x) {  // of a page of this block
    const int w = (x - x0) >> 5;
    return first + before[w] + __popc(bits[w] & ((1u << (x & 31)) - 1u));
  };
  // free pages below `live`: as many pages move
  int moves;
  before_in_cluster(cl, s_below, live > x0 && live <= x1 ? (live < x1 ? free_before(live) : first + in_block) : 0, &moves);
#pragma unroll 4
  for (int x = x0 + tid; x < x1; x += PS_THREADS) {
    const bool unused = bits[(x - x0) >> 5] >> (x & 31) & 1u;
    const int k = free_before(x);
    if (unused && x < live) a.dst[k] = x;
    if (!unused && x >= live) a.src[x - k - (live - moves)] = x;  // x - k live pages lie before it, live - moves of them stay
    if (unused || x < live) a.page_map[x] = unused ? -1 : x;
    if (unused && x >= live) a.shares[x] = 0;
  }
  for (int i = moves + all_tid; i < most; i += all) a.src[i] = a.dst[i] = -1;
  for (int i = all_tid; i < min(free, a.free_capacity); i += all) a.free_blocks[i] = n - 1 - i;
  cl.sync();
  for (int i0 = all_tid; i0 < moves; i0 += 4 * all) {
    int from[4], to[4], s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = min(i0 + k * all, moves - 1);
      from[k] = __ldcg(&a.src[i]), to[k] = __ldcg(&a.dst[i]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] = a.shares[from[k]];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i0 + k * all < moves) a.page_map[from[k]] = to[k], a.shares[to[k]] = s[k], a.shares[from[k]] = 0;
  }
  if (all_tid == 0) *a.n_free_out = min(free, a.free_capacity);
  if (!rows_too) return;
  __syncthreads();  // one block
  rewrite_rows(a);
}

// The rest: by every block of a grid.
__global__ void __launch_bounds__(PS_THREADS) paged_compact_rows_kernel(const kie_paged_compact_args a) {
  begin_after_previous();
  rewrite_rows(a);
}

// ---- copies --------------------------------------------------------------------------------------------------

constexpr int PC_THREADS = 128, PC_AHEAD = 4;

// A block copies what one pair of pages holds of one layer's K or V, 16 bytes to a thread at a time, four of them on their
// way together. Bound by HBM: 256 pages of 64 positions on E4M3 in 24 layers, 830 MB, take 126 us, 6.6 TB/s, 0.97 of the
// measured copy rate (one load at a time and 256 threads 141 us; eight at a time 129 us, and 5.5 us instead of 4.8 for the 24
// half-filled pages of a beam search's step, whose blocks are then mostly address arithmetic).
__global__ void __launch_bounds__(PC_THREADS) paged_copy_kernel(const kie_paged_copy_args a) {
  begin_after_previous();
  const kie_pages &pg = a.pages;
  const unsigned unit = blockIdx.x, pair = unit / (2u * a.n_layers), rest = unit % (2u * a.n_layers);
  const bool is_v = rest & 1u;
  const int64_t layer = rest >> 1;
  const int src = a.src[pair], dst = a.dst[pair];
  const int rows = a.rows ? min(a.rows[pair], pg.block_size) : pg.block_size;
  if ((unsigned)src >= (unsigned)pg.n_blocks || (unsigned)dst >= (unsigned)pg.n_blocks || src == dst || rows <= 0) return;
  const int es = paged_dtype_bytes(pg.dtype), shift = __ffs(pg.head_dim * es / 16) - 1;  // 2^shift chunks of a row
  const int64_t *st = is_v ? pg.v_stride : pg.k_stride;
  uint8_t *base = static_cast<uint8_t *>(is_v ? pg.v : pg.k) + layer * (is_v ? a.v_layer_stride : a.k_layer_stride) * es;
  const uint8_t *from = base + src * st[0] * es;
  uint8_t *to = base + dst * st[0] * es;
  const unsigned all = pg.n_kv_heads * rows << shift;
  for (unsigned i0 = threadIdx.x; i0 < all; i0 += PC_AHEAD * PC_THREADS) {
    uint4 x[PC_AHEAD];
    int64_t at[PC_AHEAD];
#pragma unroll
    for (int k = 0; k < PC_AHEAD; ++k) {
      const unsigned i = i0 + k * PC_THREADS, row = i >> shift, h = row / (unsigned)rows;
      at[k] = (h * st[1] + (row - h * rows) * st[2]) * es + 16 * (i & ((1u << shift) - 1u));
      if (i < all) x[k] = __ldcg(reinterpret_cast<const uint4 *>(from + at[k]));
    }
#pragma unroll
    for (int k = 0; k < PC_AHEAD; ++k)
      if (i0 + k * PC_THREADS < all) *reinterpret_cast<uint4 *>(to + at[k]) = x[k];
  }
  if (pg.dtype != KIE_E4M3) return;
  const int64_t *ss = is_v ? pg.v_scale_stride : pg.k_scale_stride;
  float *scale = (is_v ? pg.v_scale : pg.k_scale) + layer * (is_v ? a.v_scale_layer_stride : a.k_scale_layer_stride);
  for (int i = threadIdx.x; i < pg.n_kv_heads * rows; i += PC_THREADS) {
    const int64_t at = i / rows * ss[1] + i % rows * ss[2];
    scale[dst * ss[0] + at] = scale[src * ss[0] + at];
  }
}

// Raises a kernel's limit of dynamic shared memory, once on each device.
template <class K>
cudaError_t allow_smem(K kernel, std::atomic<uint64_t> *ready, int dev, size_t most) {
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit && (ready->load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e == cudaSuccess) ready->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <class K, class... A>
cudaError_t launch_clusters(K kernel, int clusters, size_t smem, cudaStream_t stream, const A &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(PS_CLUSTER * clusters);
  cfg.blockDim = dim3(PS_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = PS_CLUSTER;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace
}  // namespace kie

cudaError_t kie_launch_paged_fork(const kie::ForkArgs &a, int dev, int sms, cudaStream_t stream) {
  using namespace kie;
  static std::atomic<uint64_t> ready[2];
  const size_t smem = (size_t)3 * a.n_seqs * 4, most = 3 * KIE_PAGED_MAX_FORK * 4;
  if ((int64_t)a.n_seqs * a.max_blocks <= PS_SMALL_TABLE && a.n_blocks <= PS_SMALL_CACHE) {
    const cudaError_t e = allow_smem(paged_fork_kernel, &ready[0], dev, most);
    return e != cudaSuccess ? e : launch_after_previous(paged_fork_kernel, 1, PS_THREADS, smem, stream, a);
  }
  cudaError_t e = allow_smem(paged_fork_plan_kernel, &ready[1], dev, most);
  // A block for every eight rows, though its warps take 32 neighbouring ones: three of four blocks only plan, or find nothing
  // to do. Spreading the rows over all of them has not been measured.
  const int blocks = std::max(1, std::min(sms, (a.n_seqs + PS_WARPS / 4 - 1) / (PS_WARPS / 4)));
  if (e == cudaSuccess) e = launch_after_previous(paged_fork_plan_kernel, blocks, PS_THREADS, smem, stream, a);
  return e != cudaSuccess ? e : launch_clusters(paged_fork_finish_kernel, std::max(1, blocks / PS_CLUSTER), 0, stream, a);
}

cudaError_t kie_launch_paged_compact(const kie_paged_compact_args &a, int dev, int sms, cudaStream_t stream) {
  using namespace kie;
  static std::atomic<uint64_t> ready{0};
  const auto pages = [](int n, int blocks) { return ((n + blocks - 1) / blocks + 31) / 32 * 32; };  // of a block
  cudaError_t e = allow_smem(paged_compact_kernel, &ready, dev, (size_t)pages(KIE_PAGED_MAX_COMPACT, PS_CLUSTER) / 32 * 8);
  if (e != cudaSuccess) return e;
  if ((int64_t)a.n_seqs * a.max_blocks <= PS_SMALL_TABLE && a.n_blocks <= PS_SMALL_CACHE)
    return launch_after_previous(paged_compact_kernel, 1, PS_THREADS, (size_t)pages(a.n_blocks, 1) / 32 * 8, stream, a,
                                 pages(a.n_blocks, 1), true);
  const int per = pages(a.n_blocks, PS_CLUSTER);
  e = launch_clusters(paged_compact_kernel, 1, (size_t)per / 32 * 8, stream, a, per, false);
  const int blocks = std::max(1, std::min(sms, (a.n_seqs + PS_WARPS / 4 - 1) / (PS_WARPS / 4)));
  return e != cudaSuccess ? e : launch_after_previous(paged_compact_rows_kernel, blocks, PS_THREADS, 0, stream, a);
}

cudaError_t kie_launch_paged_copy(const kie_paged_copy_args &a, cudaStream_t stream) {
  return kie::launch_after_previous(kie::paged_copy_kernel, (unsigned)a.n_pairs * 2u * a.n_layers, kie::PC_THREADS, 0, stream, a);
}
