// Shared by the paged-cache operators: rounding to the cache and activation types, and the launch functions that the C entry
// points (kie_paged.cu) call.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kie.h"

namespace kie {

constexpr int PAGED_MAX_GROUP = 8;   // query heads per KV head
constexpr int PAGED_ROWS = 16;       // block_size is a multiple: a 16-position tile never crosses a page

__host__ __device__ __forceinline__ int paged_dtype_bytes(int dtype) {
  return dtype == KIE_F32 ? 4 : dtype == KIE_E4M3 ? 1 : 2;
}

// An fp32 value as an element of an activation tensor (uniform dtype), rounded to nearest even.
__device__ __forceinline__ void paged_store(void *p, int64_t i, int dtype, float v) {
  if (dtype == KIE_F32)
    static_cast<float *>(p)[i] = v;
  else if (dtype == KIE_F16)
    static_cast<__half *>(p)[i] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ uint32_t pack2(float a, float b, int dtype) {
  if (dtype == KIE_F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Eight consecutive elements at p + i; VEC: p + i is aligned for 16-byte accesses.
template <bool VEC>
__device__ __forceinline__ void store8(void *p, int64_t i, int dtype, const float (&v)[8]) {
  if (!VEC) {
#pragma unroll
    for (int e = 0; e < 8; ++e) paged_store(p, i + e, dtype, v[e]);
    return;
  }
  if (dtype == KIE_F32) {
    float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
  *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) =
      make_uint4(pack2(v[0], v[1], dtype), pack2(v[2], v[3], dtype), pack2(v[4], v[5], dtype), pack2(v[6], v[7], dtype));
}

// The paged-cache kernels are launched so that their blocks may take their places while the kernel before them on the
// stream (one of them, as a rule: each of a step's operators needs the one before) still ends. The first thing a block
// does is to wait, on the device, until everything before it is complete and visible. It saves 0.3 to 0.4 us of each
// (extend of 256 requests 3.8 -> 3.4 us, append of 32 rows 2.4 -> 2.0 us, attention of 64 sequences of 64 6.0 -> 5.7).
// The short kernels let the next one in at once; the attention at the end of each block, for the next one's blocks would
// crowd on the SMs that were free first (the same attention: 8.0 us).
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void begin_after_previous() {
  wait_for_previous();
  let_next_begin();
}

template <class K, class... A>
cudaError_t launch_after_previous(K kernel, unsigned grid, unsigned threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace kie

namespace kie {

// A fork, or (done given, in the place of parents) the release of rows whose pages are shared.
struct ForkArgs : kie_paged_fork_args {
  const uint8_t *done;
};

// Attention of groups with a common prefix is four launches (kie_prefix_attn.cu): a plan; the prefixes; the rows' own
// positions (kie_paged_attn.cu), beside them; and the join. The prefixes are a list of items (group, tile of its rows, KV head)
// of PX_ITEM_COST places and one for each unit of positions. Block i takes the places from i * per_block on and leaves a piece
// of each item whose units it had: the weighted sum of V, unnormalised, for `rows` rows, at prefix[slot * DH], dimensions in
// groups of eight [DH / 8][rows][8], and at prefix_ml[slot + row] the reference (log2 units) and the sum of weights; slot =
// row.slot + head * row.rows + PX_TILE * i. The rows' own positions are a piece [DH] for each query head, at own and own_ml.
// Device time of 4 beams / 64 samples / 256 rows / 61 rows on E4M3 (the cases at the head of kie_prefix_attn.cu) 16.0 / 34.9 /
// 64.7 / 38.0 us; an item's cost as 1 place 16.4 / 35.4 / 64.5 / 38.3, as 4 16.1 / 36.2 / 64.4 / 38.6; runs of 1 place at
// least 17.1 for 4 beams, of 4 17.7, of 8 22.6, and the others as they are (E4M3 38.7 with 8).
constexpr int PX_ITEM_COST = 2, PX_MIN_RUN = 2, PX_TILE = 256;
struct PrefixRow {
  long long place;  // of the first head's item in the list
  int lo, units;    // positions that the group reads for the row; units of an item
  int slot, rows, local, unused;  // the row's query heads are rows local .. of the tile
};
// Where a block begins: its first item, of the group's `item`-th, at `place`, and the group's rows. place < 0: nothing to do.
struct PrefixBlock {
  long long place;
  int g, item, start, end;
};
struct PrefixArgs : kie_paged_attention_args {
  const int32_t *group_start, *prefix_lens;
  int n_groups;
  long long *per_block;
  PrefixBlock *blocks;
  PrefixRow *rows;
  int32_t *row_lo;  // lo of each row
  float *prefix, *own;
  float2 *prefix_ml, *own_ml;
  unsigned long long wait_ns;  // how long a wait may take
  int stop_block, stop_half;   // a test's: this block (-1: none) loads nothing from its stop_half-th half of a unit on
};

// The kernels find the rows' ends in lens, be they lengths or a step's positions, and the number of table rows in n_table.
inline kie_paged_attention_args rows_in_lens(kie_paged_attention_args a) {
  if (a.seqs)
    a.lens = a.positions;
  else
    a.n_table = a.n_seqs;
  return a;
}

// Positions of query row b. Rows of a step (a.seqs) end with their own position.
__device__ __forceinline__ int row_len(const kie_paged_attention_args &a, int b) {
  const int own = a.seqs ? 1 : 0;
  return min(max(a.lens[b], -own), a.max_blocks * a.pages.block_size - own) + own;
}

}  // namespace kie

cudaError_t kie_launch_paged_fork(const kie::ForkArgs &a, int dev, int sms, cudaStream_t stream);
cudaError_t kie_launch_paged_compact(const kie_paged_compact_args &a, int dev, int sms, cudaStream_t stream);
cudaError_t kie_launch_paged_copy(const kie_paged_copy_args &a, cudaStream_t stream);
cudaError_t kie_launch_token_logprobs(const kie_token_logprobs_args &a, int sms, cudaStream_t stream);
cudaError_t kie_launch_paged_own(const kie::PrefixArgs &a, int dev, int sms, cudaStream_t stream);
cudaError_t kie_launch_paged_prefix(const kie_paged_prefix_attention_args &a, unsigned long long wait_ns, int stop_block,
                                    int stop_half, int dev, int sms, cudaStream_t stream);
size_t kie_paged_prefix_workspace_bytes(int n_seqs, int n_heads, int n_kv_heads, int head_dim, int sms);
cudaError_t kie_launch_paged_attention(const kie_paged_attention_args &a, int dev, int sms, cudaStream_t stream);
size_t kie_paged_attention_workspace_bytes(int n_heads, int n_kv_heads, int head_dim, int sms);
