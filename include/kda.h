/*
 * kda.h -- C ABI of the GB300 (sm_103a) Kimi Delta Attention (KDA) serving hot path.
 *
 * KDA is the gated delta rule with channel-wise decay used by Kimi Linear / Kimi K3:
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T ,   o_t = scale * S_t^T q_t
 *
 * Per request and head it keeps a dk x dv fp32 recurrent state S and a short causal-convolution state
 * ("A Preview of Production-Scale Kimi K3 Support on vLLM", section "The Hardest Part: Prefix Caching
 * for KDA": each KDA layer advances a matrix-like recurrent state together with a short convolution
 * state).  One token, for one head, is processed as:
 *   1. causal conv of width W over the raw q | k | v channels (weights [H][2dk+dv][W], tap W-1 on the
 *      current input, tap 0 on the oldest stored one), then SiLU when conv_silu != 0;
 *   2. q^ = q / sqrt(|q|^2 + l2_eps), k^ likewise (v is the conv output as is);
 *   3. alpha = sigmoid(a) per key channel, beta = sigmoid(b) per head (a, b are logits);
 *   4. the update above;  5. o = scale * S^T q^;
 *   6. y = o / sqrt(mean(o^2) + rms_eps) * norm_weight * sigmoid(z)   (gate factor 1 when z is NULL).
 *
 * All entry points are asynchronous on the given stream, allocate nothing, keep no state between
 * calls, and never synchronise the host, so they may be captured in a CUDA graph.  The caller owns
 * every buffer.  All pointers named "device" must be device (or managed) memory of the current device,
 * 16-byte aligned.  bf16 tensors are passed as their uint16 bit patterns.
 *
 * Errors: problems visible on the host return a kda_status before anything is launched.  Problems only
 * visible on the device (an out-of-range slot index, inconsistent sequence or checkpoint tables) OR a bit into *dev_status (a device int32 the caller
 * zeroes and reads after synchronising) and skip the affected work item; kernels never trap.
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define KDA_API __attribute__((visibility("default")))
#else
#define KDA_API
#endif

/* Same type as cudaStream_t.  NULL is the legacy default stream. */
typedef struct CUstream_st *kda_stream_t;

/* Host-side return codes. */
enum kda_status {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = 1,       /* NULL pointer, negative count, misaligned pointer, bad interval */
    KDA_ERR_UNSUPPORTED_SHAPE = 2, /* (dk, dv, conv width, chunk) not compiled in */
    KDA_ERR_WORKSPACE = 3,         /* workspace NULL or smaller than kda_prefill_workspace_bytes() */
    KDA_ERR_CUDA = 4               /* a CUDA launch or attribute call failed */
};

/* Device-side status bits, OR-ed into *dev_status. */
#define KDA_DEV_BAD_SLOT 0x1      /* a slot index outside [0, num_slots) (src may also be -1) */
#define KDA_DEV_BAD_SEQLENS 0x2   /* cu_seqlens not non-decreasing from 0 to total_tokens, or start_pos < 0 */
#define KDA_DEV_BAD_CKPT 0x4      /* ckpt_offsets does not give sequence n exactly its boundary count */
#define KDA_DEV_BAD_PAGE 0x8      /* a page table entry in use outside [0, num_pages) */
#define KDA_DEV_TIMEOUT 0x10      /* a bounded wait on an asynchronous copy gave up */
#define KDA_DEV_NO_PAGES 0x20     /* a page pool operation found too few free pages for an item */

/*
 * The state-slot pool ("The Hardest Part: Prefix Caching for KDA": the physical state block is
 * decoupled from the prefix-match unit; a slot here is one state snapshot).  Layout, slot-major:
 *   S    [num_slots][H][dk][dv]         state_dtype (fp32, or bf16 bit patterns); row i = key channel,
 *                                       column j = value channel
 *   conv [num_slots][H][W-1][2dk+dv]    bf16, the last W-1 RAW (pre-conv) q|k|v inputs, oldest first
 * Both device, owned by the caller.  With a bf16 pool ("moonshotai/Kimi-K3" recipe:
 * --mamba-ssm-cache-dtype bfloat16) every kernel computes in fp32 and rounds the state to bf16 (nearest
 * even) where it is stored; this halves the state bytes of a decode step.
 */
enum kda_state_dtype { KDA_STATE_FP32 = 0, KDA_STATE_BF16 = 1 };

typedef struct kda_pool {
    int32_t H, dk, dv, conv_w;  /* heads, key dim, value dim, conv width W */
    int32_t state_dtype;        /* enum kda_state_dtype */
    int32_t reserved;           /* 0 */
    int64_t num_slots;
    void *S;
    uint16_t *conv;
} kda_pool;

/* Layer constants. */
typedef struct kda_params {
    const float *conv_weight; /* device [H][2dk+dv][W] fp32 */
    const float *norm_weight; /* device [dv] fp32 (shared by all heads) */
    float l2_eps;             /* q/k normalisation: x / sqrt(|x|^2 + l2_eps) */
    float rms_eps;            /* output RMSNorm epsilon */
    float scale;              /* readout scale */
    int32_t conv_silu;        /* 1: SiLU after the conv; 0: none */
} kda_params;

/*
 * One decode token for each of n requests, all heads, in one launch: conv, gates, state update,
 * readout and gated RMSNorm fused ("A Preview of Production-Scale Kimi K3 Support on vLLM", section
 * "KDA prefill and decode"; "vLLM Kimi K3 Support", section "Fused Kernels and Metadata Optimization":
 * one launch, no intermediate tensors, no repeated state traffic).
 *   q, k      device [n][H][dk] bf16        v, z  device [n][H][dv] bf16 (z may be NULL: no gate)
 *   a         device [n][H][dk] bf16 (decay logits)   b  device [n][H] bf16 (beta logits)
 *   y         device [n][H][dv] bf16 output
 *   src_slot  device [n] int32: state read from this slot; -1 = fresh request (zero state and window)
 *   dst_slot  device [n] int32: updated state and window written here (src == dst: in place)
 *   dev_status device int32, OR-ed with KDA_DEV_* bits.
 * Within one call no dst slot may repeat and no slot may be the src of one request and the dst of
 * another ("The Hardest Part: Prefix Caching for KDA": same-step reuse is deferred until the copy is
 * safe).  A request with a bad slot index gets y = 0 and no state write.
 * Supported: (dk, dv) in {(16,16), (32,16), (16,32), (64,64), (128,128)}, W = 4.
 */
KDA_API int kda_decode_step(const kda_pool *pool, const kda_params *prm, int32_t n, const uint16_t *q, const uint16_t *k,
                    const uint16_t *v, const uint16_t *a, const uint16_t *b, const uint16_t *z, uint16_t *y,
                    const int32_t *src_slot, const int32_t *dst_slot, int32_t *dev_status, kda_stream_t stream);

/*
 * The input projections of a KDA layer in one GEMM ("A Preview of Production-Scale Kimi K3 Support on
 * vLLM", section "KDA prefill and decode": the input projections and the causal convolution are fused around
 * the core recurrence).  q, k, v, the decay logits a, the output gate z and the beta logits b come from one
 * packed weight matrix and are written in the layout kda_prefill_chunked reads; the causal convolution is
 * fused into the prefill's chunk kernel, which consumes these raw rows.
 *   x    device [T][hidden] bf16 hidden states (hidden % 8 == 0)
 *   w    device [N][hidden] bf16, N = H*(3*dk + 2*dv) + H: the rows of q (H*dk), k (H*dk), v (H*dv),
 *        a (H*dk), z (H*dv) and b (H), in that order (row = output feature, K-major)
 *   q, k, a  device [T][H][dk] bf16 out    v, z  device [T][H][dv] bf16 out (z may be NULL: not stored)
 *   b    device [T][H] bf16 out
 *   dev_status device int32, OR-ed with KDA_DEV_TIMEOUT if a bounded wait gave up.
 * fp32 accumulation in tensor memory; each output rounded to bf16 (nearest even).  All pointers but b
 * 16-byte aligned.  Asynchronous on `stream`; allocates nothing.
 */
KDA_API int kda_project_inputs(int64_t T, int32_t hidden, int32_t H, int32_t dk, int32_t dv, const uint16_t *x,
                               const uint16_t *w, uint16_t *q, uint16_t *k, uint16_t *v, uint16_t *a, uint16_t *b,
                               uint16_t *z, int32_t *dev_status, kda_stream_t stream);

/* Most tokens per request that one kda_decode_multi call takes. */
#define KDA_DECODE_MULTI_MAX_L 8

/*
 * L consecutive decode tokens for each of n requests in one launch, keeping the state after every position
 * on request: the verification step of speculative decoding ("vLLM Kimi K3 Support", section "Speculative
 * Decoding with DSpark": several tokens accepted per step; "moonshotai/Kimi-K3" recipe:
 * num_speculative_tokens 4, i.e. L = 5 with the bonus position).  The pages do not say how a recurrent state
 * is rolled back after a rejection; here the caller keeps the state at each position it may resume from
 * (per-position retention) and continues from the slot of the last accepted position.
 *   q, k, a   device [n*L][H][dk] bf16   v, z, y  device [n*L][H][dv] bf16   b  device [n*L][H] bf16
 *             (row r*L + j holds token j of request r; z may be NULL)
 *   src_slot  device [n] int32: state before token 0; -1 = fresh request
 *   dst_slots device [n*L] int32: the state and conv window after token j of request r go to slot
 *             dst_slots[r*L + j]; -1 = not kept.  The tokens are processed in order with the state held in
 *             fp32 between them, whatever is kept.
 *   dev_status device int32, OR-ed with KDA_DEV_* bits.
 * Each token's arithmetic is that of kda_decode_step, so L = 1 with dst_slots = dst_slot reproduces it bit
 * for bit.  Aliasing: the non-negative dst_slots of one call are distinct; a request's src may be one of its
 * own dst_slots, never another request's.  A request with a bad slot index gets y = 0 for all L tokens and
 * no state write.  1 <= L <= KDA_DECODE_MULTI_MAX_L; shapes as kda_decode_step.
 */
KDA_API int kda_decode_multi(const kda_pool *pool, const kda_params *prm, int32_t n, int32_t L, const uint16_t *q,
                             const uint16_t *k, const uint16_t *v, const uint16_t *a, const uint16_t *b,
                             const uint16_t *z, uint16_t *y, const int32_t *src_slot, const int32_t *dst_slots,
                             int32_t *dev_status, kda_stream_t stream);

/*
 * Checkpoint boundaries of one sequence: the prefix lengths p with p % interval == 0 and
 * start_pos < p <= start_pos + len ("vLLM Kimi K3 Support", section "Agentic Cache Retention Policies":
 * interval-based retention; "moonshotai/Kimi-K3" recipe: prefix-match unit 128).  Host function; returns
 * the count (0 when interval <= 0 or len <= 0), or -1 for start_pos < 0.
 */
KDA_API int64_t kda_checkpoint_count(int64_t start_pos, int64_t len, int64_t interval);

/* Bytes of device workspace kda_prefill_chunked needs for these sizes (host function, no CUDA call). */
KDA_API size_t kda_prefill_workspace_bytes(const kda_pool *pool, int32_t nseq, int64_t total_tokens, int32_t chunk);

/*
 * Chunked prefill of nseq variable-length sequences with checkpoint emission into the pool ("A Preview
 * of Production-Scale Kimi K3 Support on vLLM", sections "KDA prefill and decode" -- chunked prefill and
 * one-operation initial-state gather -- and "The Hardest Part: Prefix Caching for KDA" -- the state
 * must exist at the exact prefix boundary).
 *   cu_seqlens  device [nseq+1] int32, cu_seqlens[0] = 0, non-decreasing, cu_seqlens[nseq] = total_tokens
 *   start_pos   device [nseq] int64: absolute position of each sequence's first token (tokens already
 *               in its state); chunks are aligned to absolute positions, so a resumed sequence
 *               computes exactly what a full replay computes from the same boundary on
 *   src_slot, dst_slot  as for decode (src -1 = empty prefix)
 *   chunk       tokens per chunk (16 or 64)
 *   ckpt_interval  0 = no checkpoints; else a positive multiple of chunk
 *   ckpt_offsets   device [nseq+1] int32: sequence n's boundaries (kda_checkpoint_count of them,
 *               ascending) own entries ckpt_offsets[n] .. ckpt_offsets[n+1]-1 of ckpt_slots
 *   ckpt_slots     device int32: slot receiving (S, conv window) at that boundary, or -1 to skip.
 *               A boundary equal to the sequence end is emitted too.
 *   q,k,v,a,b,z,y  as for decode with n replaced by total_tokens (token-major)
 *   workspace   device, at least kda_prefill_workspace_bytes() bytes, contents need not be initialised
 * Same aliasing rules as decode, with checkpoint slots counting as dst slots.
 * Supported: (dk, dv) as for decode, W = 4, chunk in {16, 64}.
 * Streams: all work is ordered on `stream`.  At dk = dv = 128, chunk 64, a call with few
 * (sequence, head) chains (nseq*H*4 <= SM count) and at least 512 chunks is launched in segments.
 * The chunk chain of each segment then runs on a library-owned side stream, beside the next segment's
 * intra-chunk kernel.  The side stream forks from `stream` and joins it again before the call returns
 * (events only), so this works under CUDA graph capture too.  Segmented calls on one device are
 * serialised by a host lock.  The results are bit-identical to one launch.
 */
KDA_API int kda_prefill_chunked(const kda_pool *pool, const kda_params *prm, int32_t nseq, int64_t total_tokens,
                        const int32_t *cu_seqlens, const int64_t *start_pos, const int32_t *src_slot,
                        const int32_t *dst_slot, int32_t chunk, int64_t ckpt_interval, const int32_t *ckpt_offsets,
                        const int32_t *ckpt_slots, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                        const uint16_t *a, const uint16_t *b, const uint16_t *z, uint16_t *y, void *workspace,
                        size_t workspace_bytes, int32_t *dev_status, kda_stream_t stream);

/*
 * kda_prefill_chunked without a caller-provided workspace (the pages have no counterpart: this is an
 * interface for callers that cannot allocate device memory -- an engine whose caching allocator owns all
 * free memory, a plug-in handed only tensors, a process with no device allocation after start-up).
 * The workspace is a fixed array of KDA_NOALLOC_SCRATCH_BYTES compiled into the library; every GPU that
 * loads the library holds it until the process exits.  The call allocates nothing.
 *   Arguments: as kda_prefill_chunked, minus workspace and workspace_bytes.
 *   Limit: a problem whose kda_prefill_workspace_bytes() exceeds KDA_NOALLOC_SCRATCH_BYTES returns
 *   KDA_ERR_WORKSPACE without launching (64 MiB holds, e.g., one 512-token sequence at H = 32, dk = dv = 128).
 *   Errors: the argument checks of kda_prefill_chunked come first and make no CUDA call; then the size
 *   check (KDA_ERR_WORKSPACE); then the per-device set-up below (KDA_ERR_CUDA if it fails).
 *   Set-up: the first call on a device (with that device current) looks up the array's device address
 *   (cudaGetSymbolAddress).  Under CUDA's lazy module loading that is also when the driver allocates the
 *   array on that device, so a caller that must allocate nothing later makes this call at start-up,
 *   before it reserves its own memory pool.  The same call does the prefill launchers' one-time set-up
 *   (kernel attributes; the side stream and two events that segmented launches use), so later calls
 *   create nothing.  A call with nseq = 0 does the set-up and nothing else.  Make it before any stream
 *   capture on the device.  The address is cached per device for the life of the process; a device
 *   reset (cudaDeviceReset) invalidates it, and the library must not be used on that device afterwards.
 *   All calls on a device share the one array and it keeps the last call's contents (nothing in it needs
 *   to start at zero): calls whose executions overlap on the GPU -- on different streams, or from
 *   different host threads -- race on it and must be serialised by the caller.
 */
#define KDA_NOALLOC_SCRATCH_BYTES (64u << 20)
KDA_API int kda_prefill_chunked_noalloc(const kda_pool *pool, const kda_params *prm, int32_t nseq,
                                        int64_t total_tokens, const int32_t *cu_seqlens, const int64_t *start_pos,
                                        const int32_t *src_slot, const int32_t *dst_slot, int32_t chunk,
                                        int64_t ckpt_interval, const int32_t *ckpt_offsets,
                                        const int32_t *ckpt_slots, const uint16_t *q, const uint16_t *k,
                                        const uint16_t *v, const uint16_t *a, const uint16_t *b, const uint16_t *z,
                                        uint16_t *y, int32_t *dev_status, kda_stream_t stream);

/*
 * Copy-on-write resume ("The Hardest Part: Prefix Caching for KDA": a cached partial state is copied
 * into a private destination before the request extends it): for each of n pairs, slot dst_slot[i]
 * receives a bit-exact copy of slot src_slot[i] (state and conv window, all heads).  src_slot and
 * dst_slot are device [n] int32; dst slots must be distinct and must not be src slots of the same call.
 */
KDA_API int kda_resume_from_slot(const kda_pool *pool, int32_t n, const int32_t *src_slot, const int32_t *dst_slot,
                         int32_t *dev_status, kda_stream_t stream);

/*
 * Latent attention, the other attention layer of a hybrid model ("A Preview of Production-Scale Kimi K3
 * Support on vLLM", section on the MLA module: a full-attention layer beside the KDA layers).  Per token it
 * keeps one row x_j = [c_j | r_j] for all heads: a latent vector of `rank` values and a rotary key of `rope`
 * values (already rotated).  Keys and values of head h are linear in it, k = [W_K^h c | r] and v = W_V^h c, so
 * attention has two forms:
 *   absorbed  q~ = [W_K^h^T q_nope | q_rope]:  s_j = scale q~.x_j,  o~ = sum_j softmax(s)_j c_j  (then W_V^h o~):
 *             every head reads the same rows, which suits few queries over a long cache (kda_latent_decode);
 *   expanded  keys and values per head, fewer operations per pair: suits prompts (kda_latent_prefill).
 * The projections W are plain matrix products and the caller's.
 *
 * The rows live in pages of page_size tokens: pages [layers][num_pages][page_size][rank + rope], where layers
 * and pages may have any (16-byte aligned, not overlapping) stride.  One page index holds the same tokens in
 * every layer.  Supported: rank in {128, 256, 384, 512}; rope a multiple of 16, 0 to 64; page_size 16, 32 or a
 * multiple of 64 up to 1024.
 * In all of these calls a tensor's strides reach at most 2^44 elements from its first index to its last, and n and
 * max_seqs are at most 2^30 (where no lower limit is given).
 */
enum kda_elem_type { KDA_ELEM_BF16 = 0, KDA_ELEM_FP16 = 1 };

typedef struct kda_latent_cache {
    int32_t rank, rope, page_size, layers;
    int32_t dtype;             /* enum kda_elem_type */
    int32_t reserved;          /* 0 (kda_kv_cache_pages() fills in another value, for the kda_pages_* calls alone) */
    int64_t num_pages;
    int64_t layer_stride;      /* elements from a page's copy in one layer to that in the next */
    int64_t page_stride;       /* elements from one page to the next */
    void *pages;               /* device, 16-byte aligned */
} kda_latent_cache;

/*
 * Which pages hold which sequence: token j of table row s is row j % page_size of page
 * table[s][j / page_size], for j < lens[s].  refcount[p] counts the table rows that page p serves (0 = free);
 * only the kda_pages_* calls use it (it may be NULL for the others).  Entries behind a row's last page are not read.
 * max_pages * page_size is at most 2^31 - 64 tokens.
 */
typedef struct kda_page_table {
    int32_t max_seqs, max_pages;  /* rows, and entries of a row */
    int32_t page_size;
    int32_t reserved;             /* 0 */
    int64_t num_pages;
    int32_t *table;               /* device [max_seqs][max_pages] */
    int32_t *lens;                /* device [max_seqs] */
    int32_t *refcount;            /* device [num_pages] */
} kda_page_table;

/*
 * Writes the cache rows of new tokens of n sequences into one layer.  Sequence b's tokens are rows
 * cu_tokens[b] .. cu_tokens[b+1]-1 of latent and rope and become the LAST tokens of table row rows[b]
 * (rows NULL: row b): lens already counts them, and their pages are in the table (kda_pages_reserve).
 *   rows       device [n] int32 or NULL; -1 = a padding entry, whose tokens are not stored
 *   cu_tokens  device [n+1] int32, non-decreasing, cu_tokens[n] <= num_tokens; tokens behind it are ignored
 *   latent     device [num_tokens][rank], rope device [num_tokens][rope] (NULL when the cache has rope 0), the
 *              cache's type, rows at the given strides (elements, multiples of 8), 16-byte aligned
 * A sequence whose row, lengths or page is bad (KDA_DEV_BAD_SLOT, _SEQLENS, _PAGE) is not stored, as far as it is bad.
 * No two tokens of a call may go to the same place.
 */
KDA_API int kda_latent_append(const kda_latent_cache *cache, int32_t layer, const kda_page_table *pt, int32_t n,
                              const int32_t *rows, const int32_t *cu_tokens, int64_t num_tokens, const void *latent,
                              int64_t latent_stride, const void *rope, int64_t rope_stride, int32_t *dev_status,
                              kda_stream_t stream);

/* Most query tokens per sequence of one kda_latent_decode call, and most heads. */
#define KDA_LATENT_MAX_TOKENS 64
#define KDA_LATENT_MAX_HEADS 128

/* Bytes of device workspace kda_latent_decode needs on the current device for these sizes (0 for unsupported ones);
 * what is enough for some n and max_tokens is enough for smaller ones, too. */
KDA_API size_t kda_latent_decode_workspace_bytes(const kda_latent_cache *cache, int32_t H, int32_t n,
                                                 int32_t max_tokens);

/*
 * Absorbed latent attention of n sequences' newest tokens over one layer of the paged cache: a decode step
 * (one token a sequence) or the verification of drafted tokens (kda_decode_multi's counterpart), whose rows
 * are in the cache already.  Sequence b has nq = cu_tokens[b+1] - cu_tokens[b] query tokens (at most
 * max_tokens), the last nq of the len = lens[rows[b]] tokens of its table row.  Every query sees all tokens
 * before those nq.  Among the nq, query t sees token i when
 *   tree_mask NULL:  i <= t (a chain);
 *   else             bit i of tree_mask[cu_tokens[b] + t] is set (a tree: its ancestors and itself).
 *   rows       device [n] int32 table rows (repeats allowed), or NULL for row b; -1 = a padding entry
 *   cu_tokens  device [n+1] int32, or NULL: max_tokens queries for every sequence (num_tokens = n*max_tokens)
 *   q          device [num_tokens][H][rank+rope], the cache's type, at the given token and head strides
 *              (elements, multiples of 8), 16-byte aligned
 *   tree_mask  device [num_tokens] uint64, or NULL
 *   scale      from 1e-30 to 1e30; scores, scaled by it and by log2 e, have to stay within fp32
 *   out        device [num_tokens][H][rank] contiguous, the cache's type, 16-byte aligned
 *   lse        device [num_tokens][H] fp32: the natural logarithm of the sum of exp(s); or NULL
 * out, lse and the workspace overlap nothing else that the call reads or writes.
 * max_tokens decides how the call is cut: ceil(H max_tokens / 64) CTAs share each part of a sequence, of which those past
 * its own ceil(H nq / 64) idle, so a sequence costs about as much with one query as with max_tokens.  64 sequences of 500 to
 * 8192 tokens with one query each, rank 512: 32 heads 67 us with max_tokens 1, 171 with 8, 1469 with 64; 128 heads 104
 * and 678.  Where few sequences have drafts, one call for these and one for the others is faster.
 * A query that sees nothing (an empty sequence, a padding entry, an empty mask) gets out 0 and lse -inf, and so
 * do the queries of a sequence with a bad row or length (flagged; a bad page's tokens read as zero rows).  Sequences with
 * bad cu_tokens and rows of out behind cu_tokens[n] are left as they were.  Cache rows that a query does not see
 * do not matter to it, whatever they hold (NaN too).  A row with a NaN makes the outputs and lse of the queries that see
 * it NaN, and so does one with an infinity whose score is +infinity or NaN.  Where its score is -infinity it has weight
 * 0, and only the channels that are infinite in it may come out NaN; but where it is one of several drafted tokens (nq
 * above 1, or a tree_mask), all outputs and lse of the queries that see it are NaN.
 * fp32 scores, sums and outputs; weights are rounded to the cache's type for the second product (in fp16 one below
 * 2^-23 of its row's largest by up to 2^-34 of the largest), outputs at the end.  Results do not depend on the other
 * sequences' contents, but a sequence's split over CTAs (and so its last bits) depends on all lengths of the call and
 * on the GPU's number of multiprocessors.  The workspace need not be initialised and keeps nothing between calls; calls
 * that overlap on the GPU need one each.
 * 1 <= H <= KDA_LATENT_MAX_HEADS, max_tokens <= KDA_LATENT_MAX_TOKENS, n <= 65535.  A wait that gives up sets
 * KDA_DEV_TIMEOUT (outputs then are undefined).
 */
KDA_API int kda_latent_decode(const kda_latent_cache *cache, int32_t layer, const kda_page_table *pt, int32_t n,
                              const int32_t *rows, const int32_t *cu_tokens, int64_t num_tokens, int32_t max_tokens,
                              int32_t H, const void *q, int64_t q_token_stride, int64_t q_head_stride,
                              const uint64_t *tree_mask, float scale, void *out, float *lse, void *workspace,
                              size_t workspace_bytes, int32_t *dev_status, kda_stream_t stream);

/* Most queries per sequence of one kda_latent_prefill call. */
#define KDA_LATENT_MAX_QUERIES (1 << 23)

/*
 * Expanded latent attention of nseq sequences' queries over their own keys: s = scale (q_nope . k_nope +
 * q_rope . r), o = softmax(s) v, per head, with one rotary key r for all heads.
 *   cu_q, cu_k  device [nseq+1] int32, non-decreasing from 0 to at most num_q / num_k (num_k at most 2^31 - 256);
 *               max_q bounds the queries of one sequence (H * nseq * ceil(min(max_q, num_q) / 256) at
 *               most 2^26)
 *   causal      1: query i of nq sees keys j <= i + nk - nq (the queries are the last nq tokens of nk, as when
 *               the beginning of the prompt is in the cache already); 0: all nk
 *   q           device [num_q][H][nope+rope]     k_nope  device [num_k][H][nope]
 *   k_rope      device [num_k][rope]             v       device [num_k][H][dv]
 *               all of one type (dtype, enum kda_elem_type), 16-byte aligned, with token and head strides in
 *               elements (multiples of 8), so k_nope and v may be the halves of one [num_k][H][nope+dv] tensor
 *   out         device [num_q][H][dv] contiguous, same type        lse  device [num_q][H] fp32, or NULL
 * A query that sees no key gets out 0 and lse -inf; sequences with bad tables (KDA_DEV_BAD_SEQLENS) and rows
 * behind cu_q[nseq] are left as they were.  Keys and values that a query does not see do not matter to it,
 * whatever they hold.  A seen key with a NaN, or whose score is +infinity, makes a query's outputs and lse NaN (-infinity:
 * weight 0); a seen value that is not finite makes its channel, and in some calls all of the query's outputs and lse,
 * NaN or infinite.  fp32 scores, sums and outputs, roundings as for kda_latent_decode; a query's result depends on its
 * sequence alone, its last bits also on H, nseq and max_q (they decide how the work is cut).  Supported: nope and
 * dv in {64, 128}; rope a multiple of 16, 16 to 64 (a model without rotary keys gives 16 zeros); scale as for
 * kda_latent_decode; max_q up to KDA_LATENT_MAX_QUERIES.
 * A wait that gives up sets KDA_DEV_TIMEOUT (outputs then are undefined).
 */
KDA_API int kda_latent_prefill(int32_t dtype, int32_t H, int32_t nope, int32_t rope, int32_t dv, int32_t nseq,
                               const int32_t *cu_q, const int32_t *cu_k, int64_t num_q, int64_t num_k, int32_t max_q,
                               int32_t causal, const void *q, int64_t q_token_stride, int64_t q_head_stride,
                               const void *k_nope, int64_t k_token_stride, int64_t k_head_stride, const void *k_rope,
                               int64_t rope_token_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                               float scale, void *out, float *lse, int32_t *dev_status, kda_stream_t stream);

/*
 * The page pool's bookkeeping on the device, so that it can run inside a captured step.  Items are taken in
 * order, and new pages are always the lowest free ones of the pool as it was before the call, so that results
 * do not depend on timing.  An item with a bad row index or length, or whose row appears in an earlier item of
 * the call as well, is flagged (KDA_DEV_BAD_SLOT, _SEQLENS) and left out; so is one for which free pages do
 * not suffice (KDA_DEV_NO_PAGES; the demand of items before it counts whether they were served or not).  Row -1
 * (fork: -1 as parent or child) makes a padding item, which does nothing and names no row.
 * Shared pages (refcount > 1) are never written.  cache (all layers) is what page copies apply to; its
 * page_size and num_pages have to be the table's.
 *
 * kda_pages_reserve   row rows[i] grows to new_lens[i] tokens: pages are added behind its last one.  A partly
 *                     filled last page that is shared is replaced by a private copy (copy on write).
 * kda_pages_truncate  row rows[i] keeps its first keep_lens[i] tokens (0: the sequence ends; rejected drafts);
 *                     pages behind them lose a reference, their entries become -1.
 * kda_pages_fork      the empty row children[i] becomes a copy of row parents[i] (a parent may have many
 *                     children): full pages are shared, a partly filled last page is copied into a new one.
 * kda_pages_compact   pages in use move into the lowest places, [0, pages in use): the i-th used page behind them
 *                     (ascending) moves into the i-th free one among them; tables and refcounts follow.
 * kda_pages_copy      contents only, no bookkeeping: page dst[i] of every layer becomes page src[i] (-1 in
 *                     either: skipped; bad indices flagged).  No dst may repeat or be a src.
 *
 * workspace: device, 16-byte aligned, kda_pages_workspace_bytes(pt, n) bytes (n = 0 for compact), not kept
 * between calls.
 */
KDA_API size_t kda_pages_workspace_bytes(const kda_page_table *pt, int32_t n);
KDA_API int kda_pages_reserve(const kda_page_table *pt, const kda_latent_cache *cache, int32_t n, const int32_t *rows,
                              const int32_t *new_lens, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                              kda_stream_t stream);
KDA_API int kda_pages_truncate(const kda_page_table *pt, int32_t n, const int32_t *rows, const int32_t *keep_lens,
                               void *workspace, size_t workspace_bytes, int32_t *dev_status, kda_stream_t stream);
KDA_API int kda_pages_fork(const kda_page_table *pt, const kda_latent_cache *cache, int32_t n, const int32_t *parents,
                           const int32_t *children, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                           kda_stream_t stream);
KDA_API int kda_pages_compact(const kda_page_table *pt, const kda_latent_cache *cache, void *workspace,
                              size_t workspace_bytes, int32_t *dev_status, kda_stream_t stream);
KDA_API int kda_pages_copy(const kda_latent_cache *cache, int32_t n, const int32_t *src, const int32_t *dst,
                           int32_t *dev_status, kda_stream_t stream);

/*
 * Grouped-query attention over the same pool of pages, for a hybrid whose other layers are not latent ones: H query heads
 * share `heads` key-value heads, query head h reading key-value head h / (H / heads).
 *
 *     s_j = scale q . k_j ,   o = sum_j softmax(s)_j v_j
 *
 * A page holds page_size tokens of one layer in one contiguous piece of 16-bit words:
 *   keys    [heads][page_size][head_dim]
 *   values  [heads][page_size][head_dim]
 *   stats   [heads][2][page_size] (only when `stats` is 1): a fp32 sum of attention weights, and an int32 position, of
 *           each token and head.  kda_kv_append sets them (0 and the token's position), kda_kv_decode adds to the sums,
 *           kda_kv_evict decides by them.
 * so heads page_size (2 head_dim + 4 stats) words, whatever the page_size.  Layers and pages may have any stride (16-byte
 * aligned, not overlapping).  Supported: head_dim a multiple of 8, 16 to 256; heads 1 to 128; page_size 16, 32 or a
 * multiple of 64 up to 1024; bf16 and fp16.
 * Tables, row numbers and reference counts are the page pool's (kda_page_table).  The kda_pages_* calls work on these pages
 * through kda_kv_cache_pages(), which describes them as a cache of rows that they only copy.
 */
typedef struct kda_kv_cache {
    int32_t heads, head_dim, page_size, layers;
    int32_t dtype;             /* enum kda_elem_type */
    int32_t stats;             /* 1: pages have sums and positions */
    int64_t num_pages;
    int64_t layer_stride;      /* 16-bit words from a page's copy in one layer to that in the next */
    int64_t page_stride;       /* 16-bit words from one page to the next */
    void *pages;               /* device, 16-byte aligned */
} kda_kv_cache;

/* The cache as the kda_pages_* calls take it (host only, no CUDA call): KDA_OK and *out filled, or why not. */
KDA_API int kda_kv_cache_pages(const kda_kv_cache *cache, kda_latent_cache *out);

/*
 * Rotary positions.  Pair i of dim / 2 turns by the angle a = position * theta_i:
 *     y1 = scale (x1 cos a - x2 sin a),   y2 = scale (x2 cos a + x1 sin a)
 * The pairs are the channels offset + i and offset + dim/2 + i (interleaved 0: halves), or offset + 2i and offset + 2i + 1
 * (interleaved 1); the other channels of a head stay as they are.  turns[i] is theta_i as a fraction of a full turn, times
 * 2^64: position * turns[i] modulo 2^64 is then the exact fraction of a turn at any int32 position, so far positions are
 * as precise as near ones.  All that grows with the position is the error of turns[i] itself: theta_i / 2 pi in 64-bit floating
 * point (two roundings, 2^-52 of it), then half a unit, 2^-65 of a turn (2^-34 of a turn at position 2^31).
 */
typedef struct kda_rope {
    int32_t dim, offset;       /* dim even, 2 to 256 */
    int32_t interleaved;       /* 0 or 1 */
    float scale;               /* not 0; 1 where a model does not say otherwise */
    const uint64_t *turns;     /* device [dim / 2] */
} kda_rope;

/* How theta_i = base^(-2i / dim) is changed for contexts longer than the trained one. */
enum kda_rope_scaling {
    KDA_ROPE_PLAIN = 0,
    KDA_ROPE_LINEAR = 1,       /* theta_i / factor */
    KDA_ROPE_NTK = 2,          /* base * factor^(dim / (dim - 2)) in the place of base */
    KDA_ROPE_PARTS = 3         /* with r = original theta_i / 2 pi (turns within the trained length) and
                                * g = (r - low) / (high - low) clamped to 0..1:  theta_i (g + (1 - g) / factor).  The ramp is
                                * linear in the turns; models whose ramp is linear in the pair's index i give their
                                * frequencies to kda_rope_turns_of() one by one */
};

/* Host only: turns (host [dim / 2]) of a base and a scaling; factor at least 1, 0 < original and 0 <= low < high for
 * KDA_ROPE_PARTS, ignored elsewhere.  kda_rope_turns_of: of any count frequencies in radians a position, for scalings that
 * give them one by one (each finite, not negative, below 2^20). */
KDA_API int kda_rope_turns(int32_t dim, double base, int32_t scaling, double factor, double original, double low,
                           double high, uint64_t *turns);
KDA_API int kda_rope_turns_of(int32_t count, const double *theta, uint64_t *turns);

/*
 * Rotates x [num_tokens][H][D] into out (same shape): the queries or keys of a prompt, the rotary part of latent
 * attention's queries (offset = nope) or rows (H 1).  inverse 1: by -a, the gradient of the rotation (times scale), and
 * with scale 1 what brings rotated keys back.
 *   positions  device [num_tokens] int32, any values
 *   x, out     device, of one type (dtype, enum kda_elem_type), with token and head strides in elements (multiples of 8),
 *              16-byte aligned.  out may be x itself (the same address and strides): then only the rotated channels are
 *              written; else out gets all D channels and may not overlap x.  Rows of out may not overlap one another.
 * The angle's fraction of a turn is taken to 2^-32 and then rounded to fp32, which is off by up to 2^-26 of a turn near half a
 * turn and by less near none; sine, cosine and products are fp32, rounded once to the type.
 * D a multiple of 8 up to 1024, H 1 to 1024, offset + dim <= D.
 */
KDA_API int kda_rope_apply(const kda_rope *rope, int32_t dtype, int64_t num_tokens, int32_t H, int32_t D,
                           const int32_t *positions, int32_t inverse, const void *x, int64_t x_token_stride,
                           int64_t x_head_stride, void *out, int64_t out_token_stride, int64_t out_head_stride,
                           kda_stream_t stream);

/*
 * Writes the keys and values of new tokens of n sequences into one layer, as kda_latent_append does (rows, cu_tokens, lens
 * and what is flagged are as there).  In the same launch keys are rotated on their way (rope not NULL), sums set to 0 and
 * positions stored (a cache with stats), and the tokens' queries rotated (q not NULL, which needs rope) from q into q_out.
 *   k, v       device [num_tokens][heads][head_dim], q [num_tokens][H][head_dim], the cache's type, at the given token and
 *              head strides (elements, multiples of 8), 16-byte aligned: parts of one projection's output, for example
 *   positions  device [num_tokens] int32; NULL only without rope and stats
 *   q_out      device [num_tokens][H][head_dim] contiguous, 16-byte aligned; or q itself (its address, with contiguous
 *              strides).  The queries of all tokens from cu_tokens[0] to before cu_tokens[n] are rotated, those of padding
 *              entries and of sequences with a bad row or page, too; rows before and behind them and those of flagged
 *              cu_tokens are left as they were.
 * rope->offset + rope->dim <= head_dim; H 1 to 1024.  No two tokens of a call may go to the same place.
 */
KDA_API int kda_kv_append(const kda_kv_cache *cache, int32_t layer, const kda_page_table *pt, int32_t n,
                          const int32_t *rows, const int32_t *cu_tokens, int64_t num_tokens, const void *k,
                          int64_t k_token_stride, int64_t k_head_stride, const void *v, int64_t v_token_stride,
                          int64_t v_head_stride, const int32_t *positions, const kda_rope *rope, int32_t H, const void *q,
                          int64_t q_token_stride, int64_t q_head_stride, void *q_out, int32_t *dev_status,
                          kda_stream_t stream);

/* Most query tokens per sequence of one kda_kv_decode call, and most query heads. */
#define KDA_KV_MAX_TOKENS 64
#define KDA_KV_MAX_HEADS 256

/* Bytes of device workspace kda_kv_decode needs on the current device for these sizes (0 for unsupported ones).  max_slots:
 * 0 when weights are not added up, else a bound on the sum of lens over the call's sequences, 1 or more (also where all
 * are empty).  What is enough for some n, max_tokens and max_slots is enough for smaller ones, too. */
KDA_API size_t kda_kv_decode_workspace_bytes(const kda_kv_cache *cache, int32_t H, int32_t n, int32_t max_tokens,
                                             int64_t max_slots);

/*
 * Attention of n sequences' newest tokens over one layer of the paged cache: a decode step (one token a sequence) or the
 * verification of drafted tokens, whose keys and values are in the cache already.  rows, cu_tokens, max_tokens, tree_mask,
 * scale, lse, who sees what, padding entries, empty rows and flags are kda_latent_decode's.
 *   q          device [num_tokens][H][head_dim], the cache's type, at the given token and head strides (elements,
 *              multiples of 8), 16-byte aligned; H a multiple of the cache's heads
 *   out        device [num_tokens][H][head_dim] contiguous, the cache's type, 16-byte aligned
 * out, lse and the workspace overlap nothing else that the call reads or writes.
 *   add_weights  1 (a cache with stats): the sum of each cached token of a sequence with queries becomes weight_decay * sum
 *              + the weights that these give it in this call, summed over the query tokens and over the query heads that
 *              share its key-value head.  weight_decay from 0 to 1; max_slots as the workspace was asked for, 1 or more (a
 *              call with queries and a bound of 0 is refused).  Shared pages (refcount above 1) are never written, so their
 *              tokens' sums stay; refcount may not be NULL then.  No table row may appear twice in such a call.  Sequences
 *              whose slots pass max_slots, added up in order, are flagged (KDA_DEV_BAD_SEQLENS) and leave their sums as
 *              they were, their outputs are as always.  A query whose lse is NaN adds nothing.
 * max_tokens decides for all sequences of a call how many query rows of a key-value head are worked on together: 8, 16, 32 or
 * 64, as few as hold (H / heads) max_tokens rows, or 64.  Up to 32 that costs a sequence with fewer queries little; with 64 it
 * pays for products of rows that it does not have.  64 sequences of 500 to 8192 tokens with one query each, 32 query and 8
 * key-value heads of 128: 190 us with max_tokens 1, 192 with 8, 301 from 9 on.  With 16 queries for one of them: 309 us in one
 * call, 213 in a call for the 63 and one for it; with 5 queries 193 and 206.
 * A query that sees nothing (an empty sequence, a padding entry, an empty mask) gets out 0 and lse -inf, and so do the
 * queries of a sequence with a bad row or length (flagged); a bad page's tokens read as zero keys and values (flagged).
 * Sequences with bad cu_tokens and rows of out behind cu_tokens[n] are left as they were.  Tokens that a query does not see
 * do not matter to it, whatever they hold (NaN too).  A seen key whose score is +infinity or NaN makes the query's outputs
 * and lse NaN (-infinity: weight 0); a seen value that is not finite makes its channel NaN or infinite, and where it is one
 * of several drafted tokens (nq above 1, or a tree_mask) all outputs and lse of the queries that see it NaN.
 * fp32 scores, sums and outputs; weights are rounded to the cache's type for the second product (in fp16 as for
 * kda_latent_decode), outputs at the end.  Results do not depend on the other sequences' contents, but a sequence's split
 * over CTAs (and so its last bits) depends on all lengths of the call and on the GPU's number of multiprocessors.  The
 * workspace need not be initialised and keeps nothing between calls; calls that overlap on the GPU need one each.
 * max_tokens <= KDA_KV_MAX_TOKENS, H <= KDA_KV_MAX_HEADS, n <= 65535.  A wait that gives up sets KDA_DEV_TIMEOUT (outputs
 * then are undefined).
 */
KDA_API int kda_kv_decode(const kda_kv_cache *cache, int32_t layer, const kda_page_table *pt, int32_t n,
                          const int32_t *rows, const int32_t *cu_tokens, int64_t num_tokens, int32_t max_tokens,
                          int32_t H, const void *q, int64_t q_token_stride, int64_t q_head_stride,
                          const uint64_t *tree_mask, float scale, void *out, float *lse, int32_t add_weights,
                          float weight_decay, int64_t max_slots, void *workspace, size_t workspace_bytes,
                          int32_t *dev_status, kda_stream_t stream);

/* Most tokens of a row that kda_kv_evict shortens. */
#define KDA_KV_EVICT_MAX_LEN (1 << 20)

/*
 * Eviction by accumulated attention weight, for n sequences, in all layers: of the len = lens[rows[i]] tokens of its row
 * each layer and key-value head keeps keep[i] of its own, in this order:
 *   1. protected ones: position below `first` (the beginning that most queries look at), position at or above since[i] (the
 *      newest ones), or on a shared page (refcount above 1: those are never written);
 *   2. larger sums (a NaN counts as less than anything);
 *   3. lower slots.
 * The i-th kept token behind the first keep[i] slots (ascending) moves, with its sum and position, to the i-th slot among
 * them whose token is dropped (ascending); what is behind keep[i] slots then is no longer needed: kda_pages_truncate with
 * new_lens ends the call's work.  The order of slots is no longer that of positions, which attention does not mind: keys are
 * rotated when they are stored.  lens, tables and reference counts are read only.
 *   rows      device [n] int32 or NULL (row i); -1 = a padding entry
 *   keep      device [n] int32, not negative; a row of at most keep[i] tokens stays as it is
 *   since     device [n] int32, or NULL (nothing is newest)
 *   max_len   bound on the rows' lens, 0: what the table has room for; KDA_KV_EVICT_MAX_LEN at most.  It decides how much
 *             shared memory a row takes: 64 rows of 2,112 tokens in 4 layers and 8 heads take 39 us with a bound of
 *             2,240 and 77 us with one of 131,072
 *   new_lens  device [n] int32: min(len, keep[i]); 0 for padding entries; len for rows that are flagged and left as they
 *             are: a bad page, more than keep[i] and max_len tokens, a negative keep[i] (0 for a bad row or length)
 * Flags: KDA_DEV_BAD_SLOT, _SEQLENS, _PAGE.  No row may appear twice in a call.  n <= 65535.
 */
KDA_API int kda_kv_evict(const kda_kv_cache *cache, const kda_page_table *pt, int32_t n, const int32_t *rows,
                         const int32_t *keep, int32_t first, const int32_t *since, int32_t max_len, int32_t *new_lens,
                         int32_t *dev_status, kda_stream_t stream);

/*
 * Host-side prefix index and retention policies ("A Preview of Production-Scale Kimi K3 Support on vLLM",
 * section "The Hardest Part: Prefix Caching for KDA": chained fine-grained hashes, copy-on-write of a
 * cached partial state into a private destination, deferred same-step reuse; "vLLM Kimi K3 Support",
 * section "Agentic Cache Retention Policies": interval retention and Marconi-style second-hit retention;
 * "moonshotai/Kimi-K3" recipe: prefix-match unit 128).  Pure host code: it hands out indices of the
 * caller's state pool and fills the ckpt_slots table of kda_prefill_chunked; it allocates no device
 * memory and makes no CUDA call.  Thread-safe (one internal mutex).
 *
 * A plan for a prompt of `len` tokens:
 *   - finds the longest committed cached prefix, a multiple of the match unit shorter than the prompt;
 *   - takes a private slot for the request (copy-on-write destination; LRU-evicting an unpinned cached
 *     state when the pool is full) and pins the cached source until commit;
 *   - lists one entry per match-unit boundary p in (start_pos, len] in ckpt_slots: a slot to keep the
 *     state at p, or -1.  Call kda_prefill_chunked with ckpt_interval = the match unit, these slots,
 *     start_pos, src = private_slot and dst = private_slot, after kda_resume_from_slot(src_slot ->
 *     private_slot) when src_slot >= 0.
 * Entries a plan creates become visible to lookups only at kda_prefix_commit (after the GPU work), so a
 * request planned in the same step never resumes from a state still being written.
 */
enum kda_retention { KDA_RETAIN_INTERVAL = 0, KDA_RETAIN_SECOND_HIT = 1 };

typedef struct kda_prefix_index kda_prefix_index;

typedef struct kda_prefix_plan_t {
    uint64_t plan_id;
    int32_t src_slot;      /* cached state to resume from, or -1 */
    int32_t private_slot;  /* the request's own slot */
    int64_t start_pos;     /* tokens covered by src_slot (0 when src_slot is -1) */
    int32_t num_ckpts;     /* entries written to ckpt_slots */
    int32_t reserved;
} kda_prefix_plan_t;

/* num_slots: pool slots the index manages; match_unit: tokens per hashed block (e.g. 128);
 * interval: 0, or a multiple of match_unit (interval retention keeps multiples of it and the prompt's last
 * boundary; second-hit retention keeps seen interval boundaries and the longest seen boundary).  NULL on
 * invalid arguments. */
KDA_API kda_prefix_index *kda_prefix_index_create(int32_t num_slots, int32_t match_unit, int32_t policy,
                                                  int64_t interval);
KDA_API void kda_prefix_index_destroy(kda_prefix_index *ix);
/* Slots currently unassigned (-1 for a NULL index). */
KDA_API int32_t kda_prefix_index_free_slots(kda_prefix_index *ix);
/* tokens: host [len] int32 token ids.  ckpt_slots: host [ckpt_capacity] int32, receives num_ckpts entries.
 * KDA_ERR_INVALID_ARG for bad arguments or too small a capacity; KDA_ERR_WORKSPACE when no private slot can
 * be found (every slot pinned or pending). */
KDA_API int kda_prefix_plan(kda_prefix_index *ix, const int32_t *tokens, int64_t len, kda_prefix_plan_t *out,
                            int32_t *ckpt_slots, int32_t ckpt_capacity);
/* Publish the plan's entries and unpin its source (call once its GPU work has completed). */
KDA_API int kda_prefix_commit(kda_prefix_index *ix, uint64_t plan_id);
/* Drop an uncommitted plan: its new entries and its private slot return to the free list. */
KDA_API int kda_prefix_abort(kda_prefix_index *ix, uint64_t plan_id);
/* Return a request's private slot (not a cached state) to the free list when the request ends. */
KDA_API int kda_prefix_release_slot(kda_prefix_index *ix, int32_t slot);

/* Static description of a kda_status value. */
KDA_API const char *kda_status_string(int status);

/* What the last failing call of the calling host thread rejected ("decode: q, k, v, a and z must be
 * 16-byte aligned", "prefill launch: <CUDA error text>", ...), or "" when the last call of the thread to
 * kda_decode_step, kda_prefill_chunked(_noalloc), kda_resume_from_slot, kda_check_slots, a kda_latent_*, a kda_kv_*,
 * a kda_rope_* or a kda_pages_* function succeeded.  The
 * string belongs to the library and stays valid until the thread's next such call.  Library-side record
 * only; nothing in the pages defines it. */
KDA_API const char *kda_last_error_string(void);

/*
 * Debug check of one call's slot-aliasing contract, on HOST copies of its slot arrays.  The kernels rely
 * on it but do not check it; it is the host-side form of "same-step reuse is deferred" ("A Preview of
 * Production-Scale Kimi K3 Support on vLLM", section "The Hardest Part: Prefix Caching for KDA").
 *   - every dst_slot[i] in [0, num_slots), every src_slot[i] and ckpt_slots[j] in [-1, num_slots);
 *   - no slot is written twice: the dst slots and the non-negative checkpoint slots are distinct;
 *   - a src slot is written by nobody but its own item (src_slot[i] == dst_slot[i] is in place).
 * Decode: n_ckpt = 0.  Resume: src/dst as passed.  Prefill: its ckpt_slots table.  KDA_OK, or
 * KDA_ERR_INVALID_ARG with kda_last_error_string() naming the first violation.  O((n + n_ckpt) log), no
 * device access.
 */
KDA_API int kda_check_slots(int64_t num_slots, int32_t n, const int32_t *src_slot, const int32_t *dst_slot,
                            int32_t n_ckpt, const int32_t *ckpt_slots);

/* Failure-detection check of the bounded waits every kernel uses (no counterpart in the pages): launches
 * one CTA whose mbarrier wait can never complete; after limit_ns (clamped to [1 ms, 2 s]) of %globaltimer it
 * gives up, ORs KDA_DEV_TIMEOUT into *dev_status (device int32) and returns.  No fault, no trap: the context
 * stays usable.  Asynchronous on `stream`. */
KDA_API int kda_selftest_wait_timeout(int64_t limit_ns, int32_t *dev_status, kda_stream_t stream);

/* Library version, for the loader's sanity check. */
KDA_API int kda_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
