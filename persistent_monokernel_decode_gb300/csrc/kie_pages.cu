// Pages that several sequences share: forks, compaction and copies (kie_paged.cu holds the C entries).
//
// Forks and compaction are short chains of passes over small integer arrays, each of which needs the whole of the one
// before. They run as one launch of one thread-block cluster: the blocks meet at the cluster's hardware barrier, a few
// hundred nanoseconds, where a second launch would cost more than a microsecond and a grid-wide barrier would need all
// blocks resident. Counts pass between the blocks through distributed shared memory. Additions to a page's count commute
// and every list is written at ranks from scans, so results do not depend on the order in which blocks run.
#include <cooperative_groups.h>
#include <limits.h>

#include <atomic>

#include "kie_device.cuh"
#include "kie_paged.cuh"

namespace kie {
namespace {

namespace cg = cooperative_groups;

constexpr int PS_THREADS = 1024, PS_WARPS = PS_THREADS / 32;
constexpr int PS_CLUSTER = 8;  // the portable most

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

// The sum of every block's value (*all), and of those before this one. Every thread calls, in every block.
__device__ __forceinline__ int before_in_cluster(const cg::cluster_group &cl, int mine, int *all) {
  __shared__ int s_value;
  if (threadIdx.x == 0) s_value = mine;
  cl.sync();
  int before = 0, sum = 0;
  for (unsigned i = 0; i < cl.num_blocks(); ++i) {
    const int v = *cl.map_shared_rank(&s_value, i);
    if (i < cl.block_rank()) before += v;
    sum += v;
  }
  cl.sync();  // the values are read before they change, or their block ends
  *all = sum;
  return before;
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
__global__ void __launch_bounds__(PS_THREADS) paged_fork_kernel(const ForkArgs a) {
  begin_after_previous();
  extern __shared__ int ps_raw[];
  const cg::cluster_group cl = cg::this_cluster();
  const int R = a.n_seqs, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int blocks = cl.num_blocks(), block = cl.block_rank();
  // of row p: how many rows continue it; which of them keeps its open page (-1: p itself, R: none); of row r: the rank of
  // its new page (-1: it needs none)
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
  const int n_free = min(max(*a.n_free, 0), a.free_capacity);
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
    return;
  }
  int *staged = static_cast<int *>(a.workspace);
  for (int r = block * PS_WARPS + warp; r < R; r += blocks * PS_WARPS) {
    const int p = parent_of(a, r);
    bool part;
    if (p >= 0 && p != r) {
      const int *from = a.block_table + p * a.table_stride;
      const int n = pages_of(a, a.lens[p], &part);
      for (int j = lane; j < n; j += 32)
        staged[(int64_t)r * a.max_blocks + j] = rank[r] >= 0 && j == n - 1 ? a.free_blocks[n_free - 1 - rank[r]] : from[j];
    }
    if (kids[r] == 1) continue;  // its pages have as many holders as before
    const int n = pages_of(a, a.lens[r], &part);
    for (int j = lane; j < n; j += 32) {
      const int x = a.block_table[r * a.table_stride + j];
      const int change = (part && j == n - 1 ? min(kids[r], 1) : kids[r]) - 1;
      if (change && (unsigned)x < (unsigned)a.n_blocks) atomicAdd(&a.shares[x], change);
    }
  }
  cl.sync();
  for (int r = block * PS_WARPS + warp; r < R; r += blocks * PS_WARPS) {
    const int p = parent_of(a, r);
    if (p < 0 || p == r) continue;
    bool part;
    const int n = pages_of(a, a.lens[p], &part);
    for (int j = lane; j < n; j += 32) a.block_table[r * a.table_stride + j] = __ldcg(staged + (int64_t)r * a.max_blocks + j);
  }
  // pages that nobody holds any more, in the order of their ids
  const int x0 = range_begin(a.n_blocks, block, blocks), x1 = range_begin(a.n_blocks, block + 1, blocks);
  int mine = 0, freed;
  for (int x = x0 + tid; x - tid < x1; x += PS_THREADS) mine += __syncthreads_count(x < x1 && __ldcg(&a.shares[x]) < 0);
  long long to = (long long)n_free - total + before_in_cluster(cl, mine, &freed);
  if (mine)
    for (int x = x0 + tid; x - tid < x1; x += PS_THREADS) {
      const bool free = x < x1 && __ldcg(&a.shares[x]) < 0;
      int all;
      const int k = rank_of(free, &all);
      if (free) {
        a.shares[x] = 0;
        if (to + k < a.free_capacity) a.free_blocks[to + k] = x;
      }
      to += all;
    }
  if (block == 0 && tid == 0) *a.n_free_out = (int)min((long long)n_free - total + freed, (long long)a.free_capacity);
}

// ---- compaction ----------------------------------------------------------------------------------------------

// Live pages at and behind the number of live pages move into the free ones before it, both in the order of their ids.
__global__ void __launch_bounds__(PS_THREADS) paged_compact_kernel(const kie_paged_compact_args a) {
  begin_after_previous();
  const cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = a.n_blocks, most = n / 2;
  const int blocks = cl.num_blocks(), block = cl.block_rank(), all_tid = block * PS_THREADS + tid, all = blocks * PS_THREADS;
  const int x0 = range_begin(n, block, blocks), x1 = range_begin(n, block + 1, blocks);
  for (int x = x0 + tid; x < x1; x += PS_THREADS) a.page_map[x] = 0;
  cl.sync();
  const int n_free = min(max(*a.n_free, 0), a.free_capacity);
  for (int i = all_tid; i < n_free; i += all) {
    const int x = a.free_blocks[i];
    if ((unsigned)x < (unsigned)n) a.page_map[x] = -1;
  }
  cl.sync();
  int mine = 0, live;
  for (int x = x0 + tid; x - tid < x1; x += PS_THREADS) mine += __syncthreads_count(x < x1 && __ldcg(&a.page_map[x]) == 0);
  int first = before_in_cluster(cl, mine, &live);  // live pages before this block's
  mine = 0;
  for (int x = x0 + tid; x - tid < x1; x += PS_THREADS)
    mine += __syncthreads_count(x < x1 && x < live && __ldcg(&a.page_map[x]) == 0);
  int low;
  before_in_cluster(cl, mine, &low);  // live pages that stay
  const int moves = live - low;
  for (int x = x0 + tid; x - tid < x1; x += PS_THREADS) {
    const bool used = x < x1 && __ldcg(&a.page_map[x]) == 0;
    int in_chunk;
    const int k = first + rank_of(used, &in_chunk);
    if (x < x1 && !used && x < live) a.dst[x - k] = x;
    if (used && x >= live) a.src[k - low] = x;
    first += in_chunk;
  }
  for (int i = moves + all_tid; i < most; i += all) a.src[i] = a.dst[i] = -1;
  cl.sync();
  for (int i = all_tid; i < moves; i += all) {
    const int from = __ldcg(&a.src[i]), to = __ldcg(&a.dst[i]);
    a.shares[to] = a.shares[from];
    a.page_map[from] = to;
  }
  for (int x = all_tid; x < live; x += all)
    if (__ldcg(&a.page_map[x]) == 0) a.page_map[x] = x;  // the holes, at -1, stay so
  cl.sync();
  for (int x = live + all_tid; x < n; x += all) a.shares[x] = 0;
  for (int i = all_tid; i < min(n - live, a.free_capacity); i += all) a.free_blocks[i] = n - 1 - i;
  for (int r = block * PS_WARPS + warp; r < a.n_seqs; r += blocks * PS_WARPS) {
    const int len = a.lens[r];
    const int pages = len > 0 ? min((int)(((unsigned)len + a.block_size - 1) / (unsigned)a.block_size), a.max_blocks) : 0;
    for (int j = lane; j < pages; j += 32) {
      int *at = a.block_table + r * a.table_stride + j;
      const int x = *at;
      if ((unsigned)x >= (unsigned)n) continue;
      const int to = __ldcg(&a.page_map[x]);
      if (to >= 0 && to != x) *at = to;
    }
  }
  if (all_tid == 0) *a.n_free_out = min(n - live, a.free_capacity);
}

// ---- copies --------------------------------------------------------------------------------------------------

constexpr int PC_THREADS = 256;

// A block copies what one pair of pages holds of one layer's K or V: 16 bytes to a thread at a time.
__global__ void __launch_bounds__(PC_THREADS) paged_copy_kernel(const kie_paged_copy_args a) {
  begin_after_previous();
  const kie_pages &pg = a.pages;
  const unsigned unit = blockIdx.x, pair = unit / (2u * a.n_layers), rest = unit % (2u * a.n_layers);
  const bool is_v = rest & 1u;
  const int64_t layer = rest >> 1;
  const int src = a.src[pair], dst = a.dst[pair];
  const int rows = a.rows ? min(a.rows[pair], pg.block_size) : pg.block_size;
  if ((unsigned)src >= (unsigned)pg.n_blocks || (unsigned)dst >= (unsigned)pg.n_blocks || src == dst || rows <= 0) return;
  const int es = paged_dtype_bytes(pg.dtype), chunks = pg.head_dim * es / 16;
  const int64_t *st = is_v ? pg.v_stride : pg.k_stride;
  uint8_t *base = static_cast<uint8_t *>(is_v ? pg.v : pg.k) + layer * (is_v ? a.v_layer_stride : a.k_layer_stride) * es;
  const int all = pg.n_kv_heads * rows * chunks;
  for (int i = threadIdx.x; i < all; i += PC_THREADS) {
    const int c = i % chunks, row = i / chunks % rows, h = i / chunks / rows;
    const int64_t at = h * st[1] + row * st[2];
    *reinterpret_cast<uint4 *>(base + (dst * st[0] + at) * es + 16 * c) =
        *reinterpret_cast<const uint4 *>(base + (src * st[0] + at) * es + 16 * c);
  }
  if (pg.dtype != KIE_E4M3) return;
  const int64_t *ss = is_v ? pg.v_scale_stride : pg.k_scale_stride;
  float *scale = (is_v ? pg.v_scale : pg.k_scale) + layer * (is_v ? a.v_scale_layer_stride : a.k_scale_layer_stride);
  for (int i = threadIdx.x; i < pg.n_kv_heads * rows; i += PC_THREADS) {
    const int64_t at = i / rows * ss[1] + i % rows * ss[2];
    scale[dst * ss[0] + at] = scale[src * ss[0] + at];
  }
}

template <class K, class A>
cudaError_t launch_cluster(K kernel, size_t smem, cudaStream_t stream, const A &args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(PS_CLUSTER);
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
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

}  // namespace
}  // namespace kie

cudaError_t kie_launch_paged_fork(const kie::ForkArgs &a, int dev, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};  // devices whose limit of dynamic shared memory is raised
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (!bit || !(ready.load(std::memory_order_relaxed) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kie::paged_fork_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               3 * KIE_PAGED_MAX_FORK * 4);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  return kie::launch_cluster(kie::paged_fork_kernel, (size_t)3 * a.n_seqs * 4, stream, a);
}

cudaError_t kie_launch_paged_compact(const kie_paged_compact_args &a, cudaStream_t stream) {
  return kie::launch_cluster(kie::paged_compact_kernel, 0, stream, a);
}

cudaError_t kie_launch_paged_copy(const kie_paged_copy_args &a, cudaStream_t stream) {
  return kie::launch_after_previous(kie::paged_copy_kernel, (unsigned)a.n_pairs * 2u * a.n_layers, kie::PC_THREADS, 0, stream, a);
}
