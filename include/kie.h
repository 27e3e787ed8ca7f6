/*
 * kie.h -- C ABI of the GB300 (sm_103a) persistent decode monokernel.
 *
 * The library runs batch-1 greedy decode of a dense Llama-style decoder (fp16 weights and KV cache, fp32
 * arithmetic) as ONE persistent cooperative kernel per call, one CTA per SM, that loops over all requested
 * tokens and all layers without returning to the host. This is the "monokernel" of the Kog Inference
 * Engine pages ("Inside the monokernel: a single resident GPU program that never returns control"): the
 * host launches once, the device embeds, projects, attends, samples and feeds the next token back itself.
 *
 * Where the calls come from: the pages define no programming interface (the creeta article, section "Before
 * adopting", only says the engine can stand in for a vLLM deployment). The create / prefill / decode / destroy
 * shape below is this library's own statement of the batch-1 decode problem; each declaration names the part
 * of the pages its work follows, or says that it has none.
 *
 * Conventions for every entry point:
 *   - Return value: KIE_OK (0) or a negative KIE_ERR_* code. kie_last_error() gives a message.
 *   - Weights are IEEE binary16 bit patterns (uint16_t), row-major [out_features, in_features].
 *   - Pointers are HOST pointers unless the name or comment says "_dev" / "device".
 *   - A kie_ctx is not thread-safe: calls on one ctx must be serialised by the caller. All GPU work of a
 *     ctx is issued on the stream given at creation (NULL = the legacy default stream).
 *   - Positions are 0-based; the first prompt token is at position 0.
 */
#ifndef KIE_H
#define KIE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
  KIE_OK = 0,
  KIE_ERR_INVALID = -1,  /* bad argument, unsupported dimension, or call out of order */
  KIE_ERR_OOM = -2,      /* a device allocation failed */
  KIE_ERR_CAPACITY = -3, /* position + n would exceed max_seq */
  KIE_ERR_CUDA = -4,     /* a CUDA runtime call failed (message in kie_last_error) */
  KIE_ERR_LAUNCH = -5,   /* the cooperative grid (one CTA per SM) could not be made co-resident */
  KIE_ERR_TIMEOUT = -6   /* a device-side wait gave up; the kernel exited cleanly, the ctx is reset */
};

/* Model shape. Supported: head_dim in {64, 128}; n_heads % n_kv_heads == 0; d_model, ffn_dim and
 * n_heads*head_dim multiples of 8; n_layers >= 1; vocab >= 2. rope_theta is the RoPE base, rms_eps the
 * RMSNorm epsilon. */
typedef struct {
  int n_layers, d_model, n_heads, n_kv_heads, head_dim, ffn_dim, vocab, max_seq;
  float rope_theta, rms_eps;
} kie_config;

/* Host weights (fp16 bits). Per-layer fields are arrays of n_layers host pointers. Shapes:
 * embed, lm_head [vocab, d_model]; final_norm, attn_norm[l], ffn_norm[l] [d_model];
 * wq [n_heads*head_dim, d_model]; wk, wv [n_kv_heads*head_dim, d_model]; wo [d_model, n_heads*head_dim];
 * w_gate, w_up [ffn_dim, d_model]; w_down [d_model, ffn_dim].
 * Ownership: read during kie_create only; the caller may free them afterwards. */
typedef struct {
  const uint16_t *embed, *lm_head, *final_norm;
  const uint16_t *const *attn_norm, *const *wq, *const *wk, *const *wv, *const *wo;
  const uint16_t *const *ffn_norm, *const *w_gate, *const *w_up, *const *w_down;
} kie_weights;

typedef struct kie_ctx kie_ctx;

/* Device buffer sizes a ctx needs (bytes), for callers that allocate device memory themselves. */
typedef struct {
  size_t weights_bytes;   /* repacked weights + embedding table (+ the prefill's tensor-core tiles, dense models) */
  size_t kv_bytes;        /* K/V cache [n_layers][2][n_kv_heads][max_seq][head_dim] fp16 */
  size_t workspace_bytes; /* activations, split-attention partials, RoPE table, logits, control words */
  int n_cta;              /* CTAs of the persistent grid the layout was planned for */
} kie_buffer_sizes;

/* Sizes for `cfg` on the current device (n_cta = its SM count when the argument is 0).
 * Errors: KIE_ERR_INVALID for an unsupported cfg; KIE_ERR_CUDA if the device cannot be queried. */
int kie_query_buffers(const kie_config *cfg, int n_cta, kie_buffer_sizes *out);

/* Create a ctx: validates cfg, repacks the weights (QKV fused with RoPE pairs made adjacent, gate/up
 * interleaved, RMSNorm gains folded into the next matrix, rows tiled per CTA -- the fusion list of the
 * "inside the monokernel" section of the monokernel pages), uploads them, builds the RoPE table and
 * zeroes the KV cache. `stream` is a cudaStream_t or NULL. The ctx allocates its own device memory
 * (cudaMalloc) and frees it in kie_destroy. On error *out is NULL. */
int kie_create(const kie_config *cfg, const kie_weights *w, void *stream, kie_ctx **out);

/* As kie_create, but the device memory is provided by the caller (e.g. allocated with PyTorch) and stays
 * owned by the caller: it must outlive the ctx. Each buffer must be 256-byte aligned and at least the size
 * kie_query_buffers returned (for n_cta = 0). kie_create_with_buffers still allocates one temporary
 * staging buffer of the largest repacked matrix while it runs, and frees it before returning. */
int kie_create_with_buffers(const kie_config *cfg, const kie_weights *w, void *stream, void *weights_dev,
                            size_t weights_bytes, void *kv_dev, size_t kv_bytes, void *workspace_dev,
                            size_t workspace_bytes, kie_ctx **out);

/* Prompt ingestion. The pages do not describe prefill (their measurements start at decode); this call exists
 * so that decode has a KV cache and current logits to start from.
 * Append n prompt tokens (host int32 ids in [0, vocab)) to the KV cache at positions pos..pos+n-1 and keep the
 * logits of the last one (so the next decode can start). The tokens go through each layer together, in chunks
 * of up to 128: the projections are tensor-core GEMMs (tcgen05) over a second copy of the dense weights in the
 * tensor cores' tile layout, with each fp32 activation split into fp16 high and low parts (fp32-class results);
 * the causal attention over the cache runs on the tensor cores too, in 512-position pieces. The result does not depend on
 * how a prompt is split over calls (bit for bit). Synchronous. Errors: INVALID (n < 1, bad id), CAPACITY, CUDA,
 * TIMEOUT (a bounded device wait of the GEMM ran out; the sequence is reset). */
int kie_prefill(kie_ctx *ctx, const int32_t *tokens, int n);

/* The monokernel's token loop ("Inside the monokernel", creeta: one resident launch embeds, runs every layer,
 * samples greedily on the device and feeds the token back, with no host round trip between tokens).
 * Greedy decode of n tokens in ONE launch (the hot path). Token i is the argmax of the current logits
 * (lowest id on ties); the kernel then runs the forward of that token at the next position, whose logits
 * are the current ones for token i+1. So n tokens cost n forwards, and decode(a) then decode(b) gives the
 * same tokens as decode(a+b). Requires a prior prefill (INVALID otherwise). `out_tokens` is a host array of
 * n int32; the call synchronises the stream. Errors: INVALID, CAPACITY, CUDA, LAUNCH, TIMEOUT. */
int kie_decode(kie_ctx *ctx, int n, int32_t *out_tokens);

/* As kie_decode, but writes the n tokens to DEVICE memory `out_tokens_dev` and returns right after the
 * launch is enqueued on the ctx stream (no synchronisation). Device-side errors are reported by the next
 * kie_sync(). */
int kie_decode_async(kie_ctx *ctx, int n, int32_t *out_tokens_dev);

/* Wait for the ctx stream and report the status word of the last launch (KIE_OK or KIE_ERR_TIMEOUT). */
int kie_sync(kie_ctx *ctx);

/* No counterpart on the pages: a testing aid of this library (teacher forcing keeps one permitted divergence
 * of a near-tied greedy choice from cascading when the GPU is compared with a CPU reference).
 * Teacher forcing, for tests: for i in [0, n): out_tokens[i] = argmax of the current logits (what greedy
 * decode would emit), then the forward consumes forced[i] (not the argmax) at the next position; if
 * out_logits is not NULL it receives the logits of that forward ([n, vocab] fp32, host). Synchronous.
 * Requires a prior prefill. */
int kie_decode_forced(kie_ctx *ctx, int n, const int32_t *forced, int32_t *out_tokens, float *out_logits);

/* Scores a given continuation: for each of the n host tokens, what kie_token_logprobs (below) reads off the logits before
 * it, those after all tokens ahead of it; then the sequence has taken all n in, as if kie_decode had emitted them.
 * logprob [n] and, if not NULL, entropy [n]; top_ids, top_logprobs [n][top], 0 <= top <= min(vocab, KIE_MAX_TOP), NULL if
 * top is 0. The logits stay on the device. Host arrays, synchronous; requires a prior prefill. */
int kie_decode_score(kie_ctx *ctx, int n, const int32_t *tokens, int top, float *logprob, float *entropy, int32_t *top_ids,
                     float *top_logprobs);

/* No counterpart on the pages: a testing aid for sparse-MoE models (below). The expert selection is itself a
 * floating-point decision (a top_k over router logits) that a CPU reference and the GPU take from logits rounded
 * differently; to compare every step, the reference's own selections can be imposed on the GPU.
 * As kie_decode_forced, plus: forced_experts (host int32 [n][n_layers][top_k], or NULL) replaces the selection
 * of every layer of every forward by the given expert ids (the routing weights stay the softmax of the GPU's
 * router logits over the given experts, in the given order); out_experts (host int32 [n][n_layers][top_k], or
 * NULL) receives the GPU's own selection (descending router logit, the lowest id first among equal ones; ranked
 * on the logits before their common positive RMS factor, so sums whose scaled values round to the same float may
 * rank either way), computed whether or not it is overridden. It may also start a sequence (no prior prefill: the forwards then
 * ingest the forced tokens like a prompt, and out_tokens[0] is -1). Errors: INVALID (a dense model with
 * non-NULL expert arguments, an expert id outside [0, n_experts)), and those of kie_decode_forced. */
int kie_decode_forced_routed(kie_ctx *ctx, int n, const int32_t *forced, const int32_t *forced_experts,
                             int32_t *out_tokens, float *out_logits, int32_t *out_experts);

/* No counterpart on the pages (they sample on the device and never return logits): an inspection call.
 * Copy the current logits (those the next emitted token is the argmax of) to host float[vocab]. */
int kie_get_logits(kie_ctx *ctx, float *out);

/* No counterpart on the pages: sequence bookkeeping of this library.
 * Number of tokens in the KV cache (the position the next forward writes). */
int kie_position(const kie_ctx *ctx);

/* No counterpart on the pages: sequence bookkeeping of this library.
 * Forget the sequence: position 0, no current logits. The KV cache is not cleared (it is overwritten). */
int kie_reset(kie_ctx *ctx);

/* Device-side wait limit in nanoseconds for grid barriers and ring waits (default 1e9). */
int kie_set_timeout_ns(kie_ctx *ctx, uint64_t ns);

/* Barrier timing of the last launch, from %globaltimer stamps taken by every CTA:
 * barriers = grid barriers the launch passed; mean_wait_ns = mean over CTAs and barriers of the time a CTA
 * spent waiting in a barrier (idle time); mean_latency_ns = mean over barriers of the SHORTEST wait among
 * CTAs (the last CTA to arrive waits only for the barrier's own latency); total_ns = launch duration seen
 * by CTA 0. */
typedef struct {
  int64_t barriers;
  double mean_wait_ns, mean_latency_ns, total_ns;
} kie_barrier_stats;
int kie_get_barrier_stats(kie_ctx *ctx, kie_barrier_stats *out);

/* Raw barrier trace of the last launch (the first 4096 grid barriers): for barrier b in
 * [first, first + count) and CTA i, arrive_ns[(b - first) * n_cta + i] is the %globaltimer value when CTA i
 * arrived and wait_ns[...] how long it waited. Host arrays of count * n_cta entries. Returns the number of
 * barriers copied (>= 0) or a negative error code. */
int kie_get_barrier_trace(kie_ctx *ctx, int first, int count, uint64_t *arrive_ns, uint32_t *wait_ns);

/* Test hook (fault injection on the host side of the contract): if cta >= 0, that CTA skips its arrival
 * at grid barrier number `barrier` of the next launch, so every other CTA's wait runs out and the launch
 * returns KIE_ERR_TIMEOUT after the configured limit. No GPU fault, trap or unbounded wait is involved. */
int kie_debug_skip_arrival(kie_ctx *ctx, int cta, int barrier);

/* No counterpart on the pages: a profiling aid. Runs the decode kernel's split-KV attention step alone (the same
 * device function and grid barrier, one cooperative launch) for layers [0, n_layers) over c cached positions,
 * with the q vector and K/V cache the ctx currently holds, so that a profiler can measure that phase's DRAM bytes
 * and time in isolation. Writes only the attention outputs and split-KV partials of the workspace; the sequence
 * (position, current logits, KV cache) is left as it was. Synchronous. Errors: INVALID (c outside [1, max_seq],
 * n_layers outside [1, n_layers]), CUDA, LAUNCH, TIMEOUT. */
int kie_profile_attention(kie_ctx *ctx, int c, int n_layers);

int kie_n_cta(const kie_ctx *ctx);
const char *kie_last_error(const kie_ctx *ctx); /* ctx may be NULL: last error of a failed create */
void kie_destroy(kie_ctx *ctx);

/* ---- standalone GEMV (the same device code as the monokernel's projections) -------------------------
 * y[M] (fp32) = W[M, K] (fp16) . x[K] (fp16), fp32 accumulation, weights streamed through the same
 * shared-memory ring. W must first be packed into the per-CTA tile layout (kie_gemv_pack), as the
 * decoder's weights are at creation. Requirements: M even, K a multiple of 8, M, K >= 2. */

/* Bytes of the packed matrix (= 2*M*K). */
size_t kie_gemv_packed_bytes(int M, int K);

/* Pack row-major W_dev [M, K] into packed_dev for an n_cta-CTA grid (0 = SM count), on `stream`.
 * Both are device pointers, 16-byte aligned, not overlapping. Asynchronous. */
int kie_gemv_pack(const uint16_t *W_dev, int M, int K, int n_cta, uint16_t *packed_dev, void *stream);

/* y_dev = W . x_dev with W packed for the same n_cta. One launch of n_cta CTAs on `stream`; asynchronous. */
int kie_gemv(const uint16_t *packed_dev, const uint16_t *x_dev, float *y_dev, int M, int K, int n_cta,
             void *stream);

/* ---- decode without device allocation ---------------------------------------------------------------
 * No counterpart on the monokernel pages: this entry point exists for callers of this library that cannot
 * call cudaMalloc once they are running -- for example code whose device memory is owned and capped by a
 * host framework's allocator, or loops that must not hit cudaMalloc/cudaFree because those calls can
 * synchronise the device and stall other streams.
 *
 * kie_decode_noalloc(ctx, n, out_tokens_dev) has the semantics of kie_decode (n greedy tokens, one launch,
 * state carried in ctx), but allocates nothing: the per-launch scratch (activations, split-KV partials and
 * the control block) lives in one static device array of KIE_NOALLOC_SCRATCH_BYTES that every GPU loading
 * the library holds until the process exits. The caller passes the output: out_tokens_dev, n int32 in
 * DEVICE memory. The device the ctx was created on must be the current device (KIE_ERR_INVALID otherwise).
 * The call is synchronous (it waits for the ctx stream) and returns KIE_OK, KIE_ERR_TIMEOUT, or the errors of
 * kie_decode; a model whose scratch exceeds the array is rejected with KIE_ERR_INVALID (the message gives both
 * sizes). It takes the same launch path as kie_decode, so a kie_debug_skip_arrival armed before it applies to
 * it. The first call on a device looks up the array's device address (with that device current), so make that
 * first call before any stream capture. All calls share the one array and it keeps the last call's contents
 * (the control block is cleared by every call): calls that overlap on the GPU, from any ctx on the same
 * device, race with each other and must be serialised by the caller. */
#define KIE_NOALLOC_SCRATCH_BYTES (512u * 1024u)
int kie_decode_noalloc(kie_ctx *ctx, int n, int32_t *out_tokens_dev);

/* ---- sparse-MoE models with FP8 experts ----------------------------------------------------------------
 * The "Extending to frontier MoE models" section of the Kog blog post ("the 2B demo vs frontier scale" in the
 * Creeta write-up) projects the monokernel onto sparse mixture-of-experts models with FP8 weights; the pages
 * give no kernel for it. This library reads it as: the FFN of every layer is n_experts SwiGLU experts of width
 * cfg->ffn_dim; a router (fp16 [n_experts, d_model]) scores the FFN-normalised vector u, the top_k experts are
 * taken (largest logit first, the lowest id among equal logits) and weighted by the softmax of their logits;
 * expert weights are OCP FP8 E4M3 ("fn": no infinities, max 448) codes, one fp32 scale per row, the weight
 * being code value * row scale. out = sum over the routed experts j of w_j * Wd_j (silu(Wg_j u) * (Wu_j u)).
 * Attention, norms, embedding and LM head are those of the dense model. Decode runs the same monokernel with
 * the router folded by linearity into the QKV and WO phases (its logits are inv_rms(h) * (R diag(g) x +
 * R diag(g) Wo o), the two products precomputed in fp32 at creation), the top_k selection right after the WO
 * barrier (ranked on the unnormalised sums, whose order the positive factor inv_rms(h) does not change, so the
 * experts are known before h is staged; the routing weights follow once inv_rms(h) is), and the two expert
 * projections as grid phases: after the selection the producer streams only the routed experts' FP8 tiles, the
 * down projection's once the gate/up tiles have landed.
 *
 * Requirements: 1 <= n_experts <= 256, 1 <= top_k <= min(8, n_experts), d_model and ffn_dim multiples of 16.
 * Prefill of a MoE ctx runs the prompt through the decode kernel one position after another (teacher forcing,
 * LM head at the last position only), in one launch per call. kie_decode_noalloc serves MoE ctxs too. */
typedef struct {
  int n_experts, top_k;
} kie_moe_config;

/* Host MoE weights: arrays of n_layers host pointers. router[l] fp16 bits [n_experts, d_model];
 * gate_q[l], up_q[l] E4M3 codes [n_experts, ffn_dim, d_model]; down_q[l] codes [n_experts, d_model, ffn_dim];
 * gate_s[l], up_s[l] fp32 row scales [n_experts, ffn_dim]; down_s[l] [n_experts, d_model]. The kie_weights
 * passed alongside supply everything else; its w_gate, w_up and w_down are not read (may be NULL).
 * Ownership: read during creation only. */
typedef struct {
  const uint16_t *const *router;
  const uint8_t *const *gate_q, *const *up_q, *const *down_q;
  const float *const *gate_s, *const *up_s, *const *down_s;
} kie_moe_weights;

/* kie_query_buffers for a sparse-MoE model (errors: INVALID for an unsupported cfg or moe, CUDA). */
int kie_query_buffers_moe(const kie_config *cfg, const kie_moe_config *moe, int n_cta, kie_buffer_sizes *out);

/* kie_create / kie_create_with_buffers for a sparse-MoE model: the expert matrices are packed per CTA in
 * 512-code column blocks (kie_packed_offset_fp8), gate and up rows interleaved; the router is stored folded
 * (R diag(g) and R diag(g) Wo, fp32, the second product accumulated in fp64 on the device) and the FFN gains
 * as given (the gain multiplies the staged vector, not the FP8 weights). */
int kie_create_moe(const kie_config *cfg, const kie_moe_config *moe, const kie_weights *w, const kie_moe_weights *mw,
                   void *stream, kie_ctx **out);
int kie_create_moe_with_buffers(const kie_config *cfg, const kie_moe_config *moe, const kie_weights *w,
                                const kie_moe_weights *mw, void *stream, void *weights_dev, size_t weights_bytes,
                                void *kv_dev, size_t kv_bytes, void *workspace_dev, size_t workspace_bytes,
                                kie_ctx **out);

/* ---- a paged K/V cache for a batch of sequences --------------------------------------------------------
 * No counterpart on the pages (they decode one request): operators for a program that serves several sequences
 * next to the batch-1 decoder above. The K/V rows of one layer lie in n_blocks pages of block_size positions;
 * block_table[seq][i] (int32) is the page of positions i * block_size .. of a sequence, and the slot of a position
 * is page * block_size + offset. kie_paged_extend gives sequences the pages of their new tokens and lists the
 * slot of each; kie_paged_append writes the tokens' K/V rows there (rotating q and k); kie_paged_attention attends
 * over the pages; kie_paged_release takes finished sequences' pages back.
 *
 * For all of them: every pointer is a DEVICE pointer of the current device; the call enqueues on `stream` (NULL =
 * the legacy default stream) and returns without synchronising; it allocates nothing, so it may be captured into a
 * graph; the argument struct is read before it returns. Calls that share no output and no workspace may overlap.
 * Errors: KIE_ERR_INVALID (message in kie_paged_last_error, per host thread) before anything is enqueued, or
 * KIE_ERR_CUDA. Index and length arrays live on the device and are not checked by the host: the kernels ignore what
 * is out of range, as said at each call. */
enum { KIE_F16 = 0, KIE_BF16 = 1, KIE_F32 = 2, KIE_E4M3 = 3 };

/* The pages of one layer. k and v: element (page, kv head, position in the page, i) at page * stride[0] +
 * head * stride[1] + position * stride[2] + i, strides in elements, each a multiple of 16 bytes, as are the
 * addresses; they are not negative and below 2^31, stride[2] below 2^26. dtype KIE_F16, KIE_BF16 or KIE_E4M3. E4M3
 * codes (OCP "fn") have one fp32 scale per row, at k_scale / v_scale [page * scale_stride[0] + head * scale_stride[1]
 * + position * scale_stride[2]] (strides from 0 to below 2^31), the value being code * scale, as in the FP8 experts'
 * rows below; else the scales are not read (may be NULL). head_dim 64 or 128; block_size a multiple of 16;
 * n_blocks * block_size < 2^31. */
typedef struct {
  void *k, *v;
  float *k_scale, *v_scale;
  int64_t k_stride[3], v_stride[3], k_scale_stride[3], v_scale_stride[3];
  int n_blocks, n_kv_heads, block_size, head_dim, dtype;
} kie_pages;

/* Pages and slots for new tokens. Request r holds lens[r] positions and brings new_lens[r] tokens; the tokens of
 * all requests are packed in request order into n_rows rows. Requests are taken in order: request r is admitted if
 * its table row has room (lens + new <= max_blocks * block_size), its rows end within n_rows, and the pages that it
 * and all requests before it need do not exceed n_free (a request that needs none is admitted anyway). A request
 * with a negative length is not admitted and counts no rows. Page j of the new ones (numbered over all requests in
 * order) is free_blocks[n_free - 1 - j]: the list is a stack.
 * Written: the new entries of block_table (the others stay), lens_out [n_seqs] (lens + new, or lens if not
 * admitted), n_free_out [1], admitted [n_seqs] (bytes 0 / 1), row_start [n_seqs + 1] (the requests' first rows) and,
 * per row, slots, positions and seqs [n_rows]: -1 for rows of requests not admitted and for rows behind the last.
 * lens_out and n_free_out must not be lens and n_free. */
typedef struct {
  const int32_t *lens, *new_lens, *free_blocks, *n_free;
  int32_t *block_table;
  int64_t table_stride;
  int32_t *lens_out, *n_free_out, *row_start, *slots, *positions, *seqs;
  uint8_t *admitted;
  int n_seqs, max_blocks, block_size, n_rows, free_capacity;
} kie_paged_extend_args;
int kie_paged_extend(const kie_paged_extend_args *a, void *stream);

/* Pages of finished requests (done[r] != 0, bytes) go back on the free list: free_blocks[n_free ...] receives their
 * block_table entries, requests in order, pages in order (those past free_capacity are dropped). lens_out: 0 for the
 * finished, else lens; n_free_out [1]. The table rows stay as they were. lens_out and n_free_out must not be lens
 * and n_free. Entries are moved as they are, here and in extend: one that is no page of the cache stays on the list
 * and is handed out again. No access leaves the pages for it: its rows get the slot -1 or one that the append skips, and
 * the attention leaves its positions out. A page that is released twice is handed out twice, to rows that then overwrite
 * each other.
 * shares (int32 [n_blocks], NULL if no pages are shared) counts the further holders of each page, as kie_paged_fork keeps
 * them: then the call is kie_paged_fork with parents[r] = done[r] ? -1 : r. A page goes back only when its last holder is
 * done, and pages go on the list in the order of their ids; at most KIE_PAGED_MAX_FORK requests. The struct has these two
 * members since pages can be shared: a program that was compiled with an earlier header passes a shorter one, of which the
 * call would read what lies behind it. Compile it anew (a library and its header belong together, here as elsewhere). */
typedef struct {
  const uint8_t *done;
  const int32_t *lens, *n_free, *block_table;
  int64_t table_stride;
  int32_t *free_blocks, *lens_out, *n_free_out;
  int n_seqs, max_blocks, block_size, free_capacity;
  int32_t *shares;
  int n_blocks;
} kie_paged_release_args;
int kie_paged_release(const kie_paged_release_args *a, void *stream);

/* Several continuations of one prompt: every request r continues what request parents[r] held before the call (a step of
 * a beam search; new samples of a prompt), sharing its pages. parents[r] = r or >= n_seqs: request r stays as it is;
 * negative: it ends, as with kie_paged_release. Full pages are shared: shares[page] (int32 [n_blocks], 0 for pages with
 * one holder or none, so that extend needs no part in it) counts the holders beyond the first. A last page that is filled
 * only in part is written by the next append, so one continuation keeps it (the request itself, else the lowest r) and
 * each of the others gets a new page, free_blocks[n_free - 1 - k] for the k-th of them in request order, into which the
 * rows that are there have to be copied: copy_src[r], copy_dst[r], copy_rows[r] (-1, -1, 0 where there is nothing to
 * copy), which kie_paged_copy takes as they are. Then pages without a holder (shares below 0) go back on the list, in
 * the order of their ids and behind the pages that were not taken, with shares 0; those past free_capacity are dropped.
 * If the new pages are more than n_free (taken within [0, free_capacity]), nothing changes: ok [1] (a byte) is 0, lens_out
 * = lens, n_free_out = n_free, nothing to copy. Written: the entries of block_table that hold positions of continued
 * requests (the others stay), shares, free_blocks, lens_out [n_seqs] (the parent's length, 0 where the request ends),
 * n_free_out [1], ok and the three copy arrays [n_seqs]. lens_out and n_free_out must not be lens and n_free. Entries of
 * the table that are no pages are moved like the others and counted nowhere. n_seqs <= KIE_PAGED_MAX_FORK; workspace:
 * n_seqs * max_blocks * 4 bytes, 16-byte aligned, contents arbitrary before and after; calls that may overlap need one each. */
#define KIE_PAGED_MAX_FORK 16384
typedef struct {
  const int32_t *parents, *lens, *n_free;
  int32_t *block_table;
  int64_t table_stride;
  int32_t *shares, *free_blocks, *lens_out, *n_free_out, *copy_src, *copy_dst, *copy_rows;
  uint8_t *ok;
  void *workspace;
  size_t workspace_bytes;
  int n_seqs, max_blocks, block_size, n_blocks, free_capacity;
} kie_paged_fork_args;
int kie_paged_fork(const kie_paged_fork_args *a, void *stream);

/* Pages copied inside a cache, K, V and scales of all layers: for each i, positions 0 .. rows[i] - 1 (rows NULL: all) of
 * page src[i] to page dst[i]. pages describes layer 0; the others follow k_layer_stride .. v_scale_layer_stride elements
 * apart (above 0 and below 2^40, of K and V multiples of 16 bytes; not read for one layer). A pair with a page outside [0,
 * n_blocks), or of a page with itself, is left out. No page may be both a source and a destination, and no two
 * destinations may be the same. n_pairs * n_layers < 2^30. */
typedef struct {
  kie_pages pages;
  int64_t k_layer_stride, v_layer_stride, k_scale_layer_stride, v_scale_layer_stride;
  const int32_t *src, *dst, *rows;
  int n_pairs, n_layers;
} kie_paged_copy_args;
int kie_paged_copy(const kie_paged_copy_args *a, void *stream);

/* A cache's pages moved together at its beginning (so that a smaller one can take its place, or its end be given back).
 * The pages listed in free_blocks[0 .. n_free) are free (entries outside [0, n_blocks) do not count, repeated ones count
 * once), the other n_live are in use, by the table or by others. Pages in use from n_live on move, in the order of their ids,
 * to the free ones below it, in theirs: src, dst [n_blocks / 2] list the moves (-1 behind the last) for kie_paged_copy, and
 * page_map [n_blocks] holds the new id of each page in use, -1 for the free ones, for whoever else knows pages by id. In
 * place: block_table (the entries of the rows' positions), shares [n_blocks] (0 for free pages) and free_blocks, which is
 * n_blocks - 1, ..., n_live from the bottom, so that n_live is given next; n_free_out [1] (free_capacity at most) must not
 * be n_free. The copies have to come before the next append or attention. n_blocks <= KIE_PAGED_MAX_COMPACT. */
#define KIE_PAGED_MAX_COMPACT (1 << 22)
typedef struct {
  const int32_t *lens, *n_free;
  int32_t *block_table;
  int64_t table_stride;
  int32_t *shares, *free_blocks, *n_free_out, *src, *dst, *page_map;
  int n_seqs, max_blocks, block_size, n_blocks, free_capacity;
} kie_paged_compact_args;
int kie_paged_compact(const kie_paged_compact_args *a, void *stream);

/* K/V rows into their slots: row t of k and v ([n_rows] x [n_kv_heads] x [head_dim], strides {row, head} in
 * elements, head_dim contiguous) goes to slot slots[t] of the pages, and q, if given, to q_out (the same type;
 * q_out may be q with the same strides, and else must not overlap it). Strides of 0 are refused in what is written (q_out,
 * pages, scales) where that dimension has more than one entry. All inputs are x_dtype (KIE_F16, KIE_BF16, KIE_F32). With a table
 * rope [n_pos][head_dim / 2] of (cos, sin) fp32 pairs, k and q are rotated first at positions[t] (pairs
 * (i, i + head_dim / 2), in fp32: x_i c - x_j s, x_j c + x_i s); v never. Rows are rounded to the cache's type once;
 * an E4M3 row gets the scale max|x| / 448 (2^-126 where that rounds to 0) and the codes of x / scale. A row whose slot lies
 * outside the pages, or whose position lies outside the table, is padding: nothing is written for it. Slots must
 * not repeat: of two rows with the same slot, each 16 bytes (E4M3: each 8 codes) and each scale may come from either.
 * n_rows times the heads of k, v and q, their sum rounded up to even, must not pass 2^28.
 * k_pairs != 0: k rows hold each pair (i, i + head_dim / 2) in adjacent elements, as the K planes of a ctx's cache
 * do ([n_layers][2][n_kv_heads][max_seq][head_dim], kie_buffer_sizes), so that a prompt that a ctx has prefilled can
 * be copied into pages; the pages always hold plain order. */
typedef struct {
  kie_pages pages;
  const void *k, *v, *q;
  void *q_out;
  int64_t k_stride[2], v_stride[2], q_stride[2], q_out_stride[2];
  const int32_t *slots, *positions;
  const float *rope;
  int n_rows, n_heads, n_pos, x_dtype, k_pairs;
} kie_paged_append_args;
int kie_paged_append(const kie_paged_append_args *a, void *stream);

/* Attention of one new token per sequence: for query head h of sequence b (kv head h / (n_heads / n_kv_heads), up
 * to 8 query heads each), out = sum_j p_j V_j with p = softmax(scale * q . K_j) over the positions j in
 * [max(0, lens[b] - window), lens[b]) (window 0: all), and lse (if not NULL) = ln sum exp(scale * q . K_j). The new
 * token's own row is already in the pages (it is position lens[b] - 1). A sequence of length <= 0 gets zeros and an
 * lse of -inf, as does a head whose every score is -inf; lengths past max_blocks * block_size (at most 2^30) are cut there. Positions on a page outside
 * [0, n_blocks) are left out. Rows behind a sequence's end are never read. q, out: q_dtype, strides {sequence, head} in elements,
 * head_dim contiguous; lse [n_seqs][n_heads]. q_dtype is KIE_F32 (F16 and E4M3 pages), or the pages' own 16-bit
 * type, or either 16-bit type for E4M3 pages. Sums and the softmax are fp32; fp32 queries and the weights p go
 * through the tensor cores as two 16-bit parts (E4M3 value rows whose scale is below 2^-60 with fewer bits).
 * Infinities and NaN where nothing is attended are of no consequence. Attended ones stay with the heads that attend them:
 * an infinity in K counts as IEEE arithmetic has it (a score of -inf has weight 0; an fp32 query element 2^39 times
 * smaller than its head's largest counts as 0), an infinity in V may become NaN in its element of the output, as a NaN
 * does (an infinite E4M3 scale of V: in every element, while lse stays right). Weighted sums are formed of up to 2^15 times the values before the division by the sum of weights, so BF16 values
 * above 2^96 may overflow.
 * n_seqs * max_blocks * block_size * n_kv_heads must not pass 2^45. out may be q, with the same strides, and else must not
 * overlap it; a stride of 0 in out is refused where that dimension has more than one entry.
 * seqs and positions (both or neither; then lens is NULL) take the rows of a step as kie_paged_extend lists them: query
 * row t, of n_seqs rows, is the token at positions[t] of the sequence in row seqs[t] of the block table (n_table rows), and
 * attends to the positions up to its own, [max(0, positions[t] + 1 - window), positions[t] + 1). Sequences without a row,
 * with several (each reads the pages for itself) and rows in any order are fine; a row with seqs[t] outside [0, n_table) or
 * a negative position, as extend lists rows that were not admitted, gets zeros and an lse of -inf.
 * workspace: kie_paged_attention_workspace bytes, 256-byte aligned, contents arbitrary before and after; calls that
 * may overlap need one each. */
typedef struct {
  kie_pages pages;
  const void *q;
  void *out;
  float *lse;
  int64_t q_stride[2], out_stride[2];
  const int32_t *block_table, *lens;
  int64_t table_stride;
  void *workspace;
  size_t workspace_bytes;
  float scale;
  int n_seqs, n_heads, max_blocks, window, q_dtype;
  const int32_t *seqs, *positions;
  int n_table;
} kie_paged_attention_args;
int kie_paged_attention(const kie_paged_attention_args *a, void *stream);

/* kie_paged_attention for sequences that share their beginnings, whose pages are read once for all of them. `a` is as
 * for kie_paged_attention, with window 0. The query rows (with lens or with seqs and positions) come in n_groups groups of
 * neighbours: group g is rows group_start[g] .. group_start[g + 1] - 1 (int32 [n_groups + 1] on the device, taken within
 * [0, n_seqs], a start below an earlier one as that one), and its positions below prefix_lens[g] (any length; what is
 * behind a row's own end is left out for that row) are read through the block table row of the longest of its query rows
 * (the first of those that reach the prefix's end); the positions behind, and those of rows in no group, through each
 * row's own. Rows of one sequence, a part of a prompt, are such a group too: its prefix is what was cached before (the
 * part's own positions are read once for each row: the time grows with the square of the rows, 64 fp16 rows of 20 / 4
 * heads of 128 behind 8,192 positions 35 us, 256 68 us, 1,024 236 us). A prefix is read 64 positions at a time: what its
 * last page holds behind its end may be read and is of no consequence. n_groups <= KIE_PAGED_MAX_GROUPS; n_groups = 0 is
 * kie_paged_attention. The limits and the treatment of infinities are those of kie_paged_attention; a NaN or an infinity
 * in a prefix concerns the rows of its group alone. K and V have to fit a tensor map; INVALID where CUDA refuses to make
 * one of their strides.
 * Inside the call, blocks wait for their own loads and products, microseconds as a rule. A wait that takes longer than two
 * seconds (kie_paged_set_timeout_ns; a GPU that is taken from the process for that long) ends its block's work: what the
 * block had in hand and had still to do is NaN, in out and in lse, for every query head that it concerns. The call itself
 * returned KIE_OK before.
 * a.workspace: kie_paged_prefix_attention_workspace bytes, 256-byte aligned, contents arbitrary before and after; calls
 * that may overlap need one each. */
#define KIE_PAGED_MAX_GROUPS 4096
typedef struct {
  kie_paged_attention_args a;
  const int32_t *group_start, *prefix_lens;
  int n_groups;
} kie_paged_prefix_attention_args;
int kie_paged_prefix_attention(const kie_paged_prefix_attention_args *a, void *stream);

/* How long a wait inside kie_paged_prefix_attention may take, in nanoseconds (2e9 at first): for all later calls of the
 * process; a captured call keeps the limit of its capture. Errors: INVALID (0). */
int kie_paged_set_timeout_ns(uint64_t ns);

/* Test hook (fault injection on the host side of the contract): block `block` of the next kie_paged_prefix_attention call
 * loads nothing from the half-th K or V of 64 positions on that it has to do with (0: nothing at all), so that its waits
 * for them run out; -1: takes that back. No GPU fault, trap or unbounded wait is involved. */
int kie_paged_debug_stop_loads(int block, int half);

/* Bytes of kie_paged_prefix_attention's workspace on the current device (0: bad arguments or no device). */
size_t kie_paged_prefix_attention_workspace(int n_seqs, int n_heads, int n_kv_heads, int head_dim);

/* ---- log probabilities of tokens -------------------------------------------------------------------------
 * What a program reads off the logits besides the argmax: for each of n_rows rows of `vocab` logits (dtype KIE_F16,
 * KIE_BF16 or KIE_F32, row_stride elements apart, >= vocab), with p = softmax(logits): logprob [n_rows] = ln p of
 * tokens[row] (int32; 0 for a token outside [0, vocab), as in padding; tokens and logprob may both be NULL), entropy
 * [n_rows] = -sum p ln p (may be NULL), and the `top` largest logits in descending order, the lowest id first among equal
 * ones: top_ids int32, top_logprobs [n_rows][top] (NULL if top is 0). All results fp32. A logit of -inf is a token that
 * is ruled out: probability 0, ln p = -inf, nothing added to the entropy; a row of only such logits has ln p = -inf
 * everywhere and entropy 0. A NaN or +inf in a row makes its logprob, entropy and top_logprobs NaN; its top_ids count a
 * NaN as larger than +inf. Rows in which fewer than `top` logits are above -inf are read up to `top` times more (4 fp32
 * rows of 32,000 with 20 alternatives 68 us instead of 11, 8,191 bf16 rows 5.7 ms instead of 0.13). 1 <= vocab < 2^30, 0
 * <= top <= min(vocab, KIE_MAX_TOP). Enqueued on `stream` like the paged operators, whose kie_paged_last_error holds its
 * messages; nothing is allocated. */
#define KIE_MAX_TOP 32
typedef struct {
  const void *logits;
  int64_t row_stride;
  const int32_t *tokens;
  float *logprob, *entropy, *top_logprobs;
  int32_t *top_ids;
  int n_rows, vocab, top, dtype;
} kie_token_logprobs_args;
int kie_token_logprobs(const kie_token_logprobs_args *a, void *stream);

/* Bytes of kie_paged_attention's workspace on the current device, for any number of sequences (0: bad arguments or
 * no device). */
size_t kie_paged_attention_workspace(int n_heads, int n_kv_heads, int head_dim);

/* Message of this host thread's last failed kie_paged_* call ("" before the first). */
const char *kie_paged_last_error(void);

/* Host-side layout query (no GPU needed): byte offset of code Q[r][c] inside a packed FP8 matrix [M, K]
 * (column blocks of 512 codes, each CTA's rows in tiles of up to 32 rows; within a full 512-code block the
 * 16-code chunk q of an odd row r is stored at chunk q ^ 4). M even, K a multiple of 16; -1 for bad
 * arguments. */
int64_t kie_packed_offset_fp8(int M, int K, int n_cta, int r, int c);

/* Host-side layout query (no GPU needed): byte offset of W[r][c] inside the prefill's tensor-core copy of an
 * [M, K] fp16 matrix: 128-row x 64-column tiles of 16 KB (rows padded to 128, columns to 64), tile (i, j) at
 * (i * ceil(K / 64) + j) * 16 KB, inside a tile 8 x 8 core matrices of 128 contiguous bytes (the canonical
 * K-major layout the tensor-core instructions read without swizzle). -1 for bad arguments. */
int64_t kie_tc_tile_offset(int M, int K, int r, int c);

/* Host-side layout query (no GPU needed): element offset of W[r][c] inside the packed matrix. */
int64_t kie_packed_offset(int M, int K, int n_cta, int r, int c);

/* Host-side layout query: first and one-past-last row owned by CTA `cta` (pairs of rows are never split). */
int kie_rows_of_cta(int M, int n_cta, int cta, int *r0, int *r1);

#ifdef __cplusplus
}
#endif
#endif /* KIE_H */
