/*
 * spava.h -- C ABI of libspava: B200 (sm_100a) kernels for the per-host
 * approximate attention of APB-V / Spava long-video prefill, with every ZigZag
 * virtual host on one GPU.
 *
 * Method source: "Riepilogo Tecnico: APB-V" (gist.science/it/paper/2601.21444),
 * section "Metodologia: APB-V" -- 1. "Design del Framework" (context split into
 * anchor block, query block and context blocks; ZigZag pairing of virtual hosts
 * h and 2H-1-h; passing blocks of the most essential KV found by query-to-context
 * attention scores; attention over anchor, local context, aggregated passing
 * blocks and query) and 2. "Ottimizzazioni a Livello di Sistema" ("Forward Fuso
 * di Contesto e Query": query partial results merged through log-sum-exp;
 * "Bilanciamento del Carico dell'Attenzione Approssimata").  Also "Spava:
 * Accelerating Long-Video Understanding via Sequence-Parallelism-aware
 * Approximate Attention", abstract.
 *
 * Conventions shared by every entry point
 *   - Tensors are DEVICE pointers unless the name says host, contiguous,
 *     token-major: Q [N, Hq, d], K and V [N, Hkv, d], O [N, Hq, d], all bf16
 *     (passed as void*), and 16-byte aligned.  lse is float32 [Hq, N], natural
 *     log.  scores are float32 [Hkv, C], C = N - a - q, context token t at
 *     column t - a.  idx is int32 [2H-1, Hkv, l]: absolute token positions,
 *     ascending, padded with -1.  Packed passing K/V are bf16 [Hkv, L, d] with
 *     L = a + sum_u min(l, n_u): the anchor rows first, then P_0, P_1, ...
 *   - The caller owns every buffer.  The library allocates no device or host
 *     memory, frees nothing and never synchronises the stream (except
 *     spava_device_status, which says so).
 *   - Calls are asynchronous and ordered on `stream` (a cudaStream_t; NULL is
 *     the legacy default stream).
 *   - Arguments are checked before any launch; on error nothing is launched
 *     and the status says why.  SPAVA_ERR_CUDA means a CUDA runtime call
 *     failed; spava_last_cuda_error() returns its code (per thread).
 *   - Kernels never trap.  A wait inside a kernel that exceeds its bound sets a
 *     flag in the workspace status word and the kernel returns early; read it
 *     with spava_device_status().
 *   - Thread-safe: no mutable global state besides per-thread error codes and
 *     the once-per-process kernel attribute set-up.
 */
#ifndef SPAVA_H_
#define SPAVA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SPAVA_OK = 0,
    SPAVA_ERR_INVALID_ARG = 1, /* a size, offset or pointer is invalid */
    SPAVA_ERR_UNSUPPORTED = 2, /* valid, but outside what the library supports (d, H, ...) */
    SPAVA_ERR_MISALIGNED = 3,  /* a device pointer is not 16-byte aligned */
    SPAVA_ERR_WORKSPACE = 4,   /* workspace missing or smaller than required */
    SPAVA_ERR_CUDA = 5,        /* a CUDA runtime call failed */
    SPAVA_ERR_TIMEOUT = 6      /* a kernel-side bounded wait gave up */
} spava_status;

/* One prefill attention layer.  Sequence split of "Suddivisione del Contesto e
 * Disposizione ZigZag": [anchor a | 2H context chunks | query block q]. */
typedef struct {
    int32_t H;            /* physical hosts = virtual-host pairs; 2H chunks; 1..32 */
    int32_t n_q_heads;    /* Hq */
    int32_t n_kv_heads;   /* Hkv; Hq % Hkv == 0, q-head h uses KV head h / (Hq/Hkv) */
    int32_t head_dim;     /* d: 64 or 128 */
    int64_t n_tokens;     /* N < 2^31 */
    int64_t anchor_len;   /* a >= 0 */
    int64_t query_len;    /* q >= 1 */
    const int64_t *chunk_offsets; /* HOST array [2H+1]: off[0]=a, off[2H]=N-q,
                                     strictly increasing; chunk v = [off[v], off[v+1]) */
    int32_t top_l;        /* l >= 0: passing-block size per KV head per chunk */
    float scale;          /* softmax scale; <= 0 selects 1/sqrt(d) */
    int32_t local_pair_full; /* 1: the later virtual host of a ZigZag pair sees its
                                partner chunk in full and takes no passing block from
                                it; 0: every virtual host takes the passing blocks of
                                all earlier chunks and no full partner chunk */
    /* Selection variants (ablations of the score reading; the pages fix
     * neither): */
    int32_t score_norm;   /* 0 (default): each query row's softmax over the chunk
                             being scored; 1: the row's own attention weights,
                             normalised over every key it attends, [0, t] */
    int32_t score_pool;   /* 0 or 1 (default): rank the scores themselves; odd w
                             in 3..255: rank each key by the sum of the scores of
                             the w keys centred on it inside its chunk (the w-key
                             window mean with zero padding, up to the factor 1/w);
                             spava_score still returns the unpooled scores */
} spava_config;

/* Workspace bytes that any entry point below needs for this config (the
 * largest of them: spava_prefill_attention).  Pass the same buffer to every
 * call; it must be 256-byte aligned.  Its first 256 bytes are the status block:
 * the status word at byte 0 (must start at zero; see spava_device_status) and
 * the work-item counter of the attention kernel's persistent grid at byte 128
 * (zeroed by every spava_attn before its launch).  Calls that share a
 * workspace must be ordered on one stream. */
spava_status spava_workspace_size(const spava_config *cfg, size_t *bytes);

/* L = a + sum_u min(l, n_u): rows of the packed passing K/V per KV head. */
spava_status spava_packed_len(const spava_config *cfg, int64_t *rows);

/* Query-to-context scores ("Blocchi di Passaggio"): for every chunk u < 2H-1,
 * KV head g and key j of chunk u,
 *   scores[g, j-a] = sum_{h in group g} sum_{i in query block}
 *                    softmax_{j' in chunk u}(scale * q_{h,i} . k_{g,j'}) at j'=j.
 * The softmax runs over chunk u only (score_norm 0); no causal mask.  With
 * score_norm 1 each row's weights are instead normalised over every key the
 * row attends, [0, t].  The last chunk has no successor and its columns are
 * left untouched.  Two passes over K: row statistics, then probability column
 * sums.  Reads q, k; writes scores. */
spava_status spava_score(const spava_config *cfg, const void *q, const void *k, float *scores,
                         void *ws, size_t ws_bytes, void *stream);

/* Passing-block selection ("Blocchi di Passaggio": the most essential KV): for
 * every chunk u < 2H-1 and KV head g, the min(l, n_u) largest scores of chunk u
 * (with score_pool w >= 3: the largest sums of the w scores centred on each key
 * inside the chunk, added in ascending order in fp32; ties: the lower token
 * index wins), written as ascending absolute positions into idx[u, g, :], the
 * remaining slots set to -1.  Exact: no approximation in the selection. */
spava_status spava_topk_select(const spava_config *cfg, const float *scores, int32_t *idx,
                               void *stream);

/* Passing-block aggregation ("aggregate in blocchi di passaggio"): pk[g, r] =
 * k[r, g] for r < a (anchor), then for each chunk u the rows k[idx[u,g,s], g],
 * s < min(l, n_u), in that order; pv likewise from v.  On one GPU this gather
 * replaces the cross-host transfer of the passing blocks. */
spava_status spava_pack_passing(const spava_config *cfg, const void *k, const void *v,
                                const int32_t *idx, void *pk, void *pv, void *stream);

/* Approximate attention ("Computazione") with online softmax:
 *   anchor row t < a:        keys [0, t]
 *   context row t, chunk v:  anchor + passing blocks of the earlier chunks
 *                            (local_pair_full=1: those on another physical host)
 *                            + partner chunk 2H-1-v in full (v >= H,
 *                            local_pair_full=1) + own chunk up to t
 *   query row t >= N-q:      keys [0, t], computed as one partial per segment
 *                            (anchor, each chunk, query block) merged by
 *                            log-sum-exp ("Forward Fuso di Contesto e Query").
 * Writes o [N, Hq, d] bf16 and, if lse != NULL, lse [Hq, N] float32. */
spava_status spava_attn(const spava_config *cfg, const void *q, const void *k, const void *v,
                        const void *pk, const void *pv, void *o, float *lse, void *ws,
                        size_t ws_bytes, void *stream);

/* The whole layer, in the order of the fused forward ("Forward Fuso di
 * Contesto e Query"): first the anchor rows and the query rows' per-segment
 * partials, whose per-chunk log-sum-exps are the scoring's normaliser; then
 * scoring, selection and gather of every passing block in one launch; then the
 * context rows and the query-row merge.  Scores, idx and the packed K/V stay in
 * the workspace.  The outputs equal, byte for byte, those of spava_score ->
 * spava_topk_select -> spava_pack_passing -> spava_attn.  If idx_out != NULL
 * the passing-block indices are also written there. */
spava_status spava_prefill_attention(const spava_config *cfg, const void *q, const void *k,
                                     const void *v, void *o, float *lse, int32_t *idx_out,
                                     void *ws, size_t ws_bytes, void *stream);

/* spava_prefill_attention from HOST buffers: copies q_host, k_host, v_host
 * into the caller's device buffers q, k, v, runs the layer, and copies o (and
 * lse if both lse and lse_host are non-NULL) back to o_host / lse_host.
 * Host buffers should be page-locked for the copies to be asynchronous; the
 * call does not wait for them.
 * copy_stream NULL (or equal to stream): everything is ordered on `stream`.
 * Otherwise the copies run on copy_stream, overlapped with the kernels,
 * chunk by chunk in token order: the query block's Q rows and the anchor go up
 * first, then each chunk's Q, K and V rows; once a chunk (and the rows its last
 * 128-row tile reaches into) has arrived, its passing block is scored, selected
 * and gathered and its rows are computed, and its O (and lse) rows go down
 * while later chunks compute; the query block's rows come last.  The kernels
 * of this mode run on three streams the call creates and destroys: scoring at
 * the device's highest stream priority, and the attention launches alternating
 * between two others, each launch waiting only for its rows and the passing
 * blocks before them, so that one launch's CTAs take the SMs its
 * predecessor's last work items leave idle.
 * (With score_norm 1 -- whose statistics need every segment first -- K and the
 * query block's Q rows go up first, then V, and the attention runs in up to 8
 * groups of whole regions as their Q rows arrive.)  The outputs equal
 * spava_prefill_attention's byte for byte.  The copies begin only after
 * all work already enqueued on `stream` (an earlier call may still be reading
 * the device buffers), and `stream` is made to wait for the last copy, so the
 * call's work is complete when `stream` is and back-to-back calls on the same
 * buffers stay ordered.  The call creates and destroys its own CUDA events
 * and streams (no memory).  Neither stream may be capturing a graph.  On an error return, work
 * already enqueued may still run. */
spava_status spava_prefill_attention_host(const spava_config *cfg, const void *q_host,
                                          const void *k_host, const void *v_host, void *o_host,
                                          float *lse_host, void *q, void *k, void *v, void *o,
                                          float *lse, void *ws, size_t ws_bytes, void *stream,
                                          void *copy_stream);

/* Synchronises `stream`, reads the workspace status word (bit 0: a bounded wait
 * in a kernel gave up; bit 1: a spava_cache_* call met a length or a page
 * outside its table or pool), writes it to *flags and clears it.  Returns
 * SPAVA_ERR_TIMEOUT if bit 0 was set, SPAVA_ERR_INVALID_ARG if only bit 1 was,
 * SPAVA_OK otherwise. */
spava_status spava_device_status(void *ws, size_t ws_bytes, void *stream, int32_t *flags);

/* Self-test of the failure path (the pages have no counterpart): launches one
 * thread that waits on a barrier nothing arrives on.  Its bounded wait gives up
 * after about two seconds, sets bit 0 of the workspace status word and the
 * kernel returns, leaving the context usable; spava_device_status() then
 * reports SPAVA_ERR_TIMEOUT and clears the bit.  Needs the first 256 bytes of a
 * workspace (256-byte aligned). */
spava_status spava_selftest_wait_timeout(void *ws, size_t ws_bytes, void *stream);

/* Exact number of (row, key) pairs per query head that spava_attn attends,
 * by row class: pairs[0] anchor rows, pairs[1] context rows, pairs[2] query
 * rows.  Algorithmic FLOPs of spava_attn = 4 * d * Hq * (sum of the three).
 * per_host (may be NULL) receives H entries: the context pairs of each
 * physical host, i.e. of its two virtual hosts p and 2H-1-p (ZigZag balance,
 * "Bilanciamento del Carico dell'Attenzione Approssimata").  Host only. */
spava_status spava_attended_pairs(const spava_config *cfg, int64_t pairs[3], int64_t *per_host);

/* Chunk offsets from a frame list ("Riepilogo Tecnico: APB-V", Metodologia,
 * "Bilanciamento del Carico Visivo": the frames are spread evenly over the
 * virtual hosts).  frame_tokens: HOST array of the n_frames frames' token
 * counts, in order (each >= 1); the 2H chunks take consecutive whole frames,
 * chunk v taking floor(n_frames / 2H) frames plus one more for
 * v < n_frames mod 2H.  Writes chunk_offsets[0..2H] (HOST, int64):
 * off[0] = anchor_len, off[v+1] = off[v] + the tokens of chunk v's frames, so a
 * layer built from them has N = off[2H] + query_len.  SPAVA_ERR_INVALID_ARG if
 * H is outside 1..32, n_frames < 2H (a chunk would be empty), a frame has no
 * token, anchor_len < 0, a pointer is NULL or the sum passes 2^31.  Host only. */
spava_status spava_plan_chunks(int32_t H, const int64_t *frame_tokens, int64_t n_frames,
                               int64_t anchor_len, int64_t *chunk_offsets);

/* ---------------------------------------------------------------------------
 * Multi-GPU ZigZag sequence parallelism ("Riepilogo Tecnico: APB-V",
 * Metodologia, "Suddivisione del Contesto e Disposizione ZigZag": physical host
 * p holds virtual hosts p and 2H-1-p; Ottimizzazioni a Livello di Sistema,
 * "Comunicazione Sovrapposta": the passing blocks travel between hosts while
 * the hosts compute, and "Forward Fuso di Contesto e Query": the query rows'
 * partial results of every host are merged through their log-sum-exp).
 *
 * `world` GPUs, one process each; H % world == 0.  Rank r holds the physical
 * hosts p in [r*m, (r+1)*m), m = H/world -- the chunks v with
 * pair(v) / m == r, pair(v) = v < H ? v : 2H-1-v -- plus the anchor and the
 * query block, which every rank holds.  Its token-major buffers (q, k, v, o:
 * [n_local, heads, d]; lse: [Hq, n_local]) are LOCAL: [anchor | its chunks in
 * increasing v | query block].  A rank computes its chunks' context rows, and
 * (like every rank) the anchor rows and the query rows.
 *
 * One layer on each rank, in this order (all on `stream`, asynchronous):
 *   spava_shard_front        scores, top-l and gather of its chunks' passing
 *                            blocks; writes its pass message
 *   all-gather #1            the caller gathers every rank's pass message,
 *                            rank-major, into pass_all (e.g. NCCL
 *                            all-gather into this GPU's own memory)
 *   spava_shard_local_attn   anchor rows and the query rows' partials over
 *                            the anchor, its chunks and the query block: needs
 *                            nothing from other ranks, so it runs while
 *                            all-gather #1 is in flight; writes its part message
 *   all-gather #2            every rank's part message into part_all
 *   spava_shard_context_attn unpacks pass_all, then the context rows of its
 *                            chunks (runs while all-gather #2 is in flight)
 *   spava_shard_merge        unpacks part_all, merges the query rows
 * The messages have the same size on every rank (spava_shard_sizes).  The
 * outputs equal spava_prefill_attention's rows bit for bit.  score_norm 1 is
 * not offered (SPAVA_ERR_UNSUPPORTED): it needs every chunk's statistics of the
 * query rows before scoring.  The same workspace serves all four calls of a
 * rank; the caller keeps pass_send / part_send unchanged until its gathers
 * have read them.
 * ------------------------------------------------------------------------- */

/* Host only.  local_first (HOST [2H+2], may be NULL): first local row of the
 * anchor (index 0), chunk v (1+v), the query block (2H+1), -1 where the rank
 * does not hold the region; *n_local: rows of its local buffers; slot_chunk
 * (HOST [2H/world], may be NULL): the chunk in each slot of its messages.
 * SPAVA_ERR_INVALID_ARG for rank outside [0, world) or world < 1,
 * SPAVA_ERR_UNSUPPORTED if world does not divide H or score_norm is 1. */
spava_status spava_shard_layout(const spava_config *cfg, int32_t rank, int32_t world,
                                int64_t *local_first, int64_t *n_local, int32_t *slot_chunk);

/* Host only: workspace bytes of a rank (256-byte aligned buffer, first 256
 * bytes the status block as for spava_workspace_size), and the bytes of one
 * rank's pass and part messages (pass_all / part_all hold world of each). */
spava_status spava_shard_sizes(const spava_config *cfg, int32_t world, size_t *ws_bytes,
                               size_t *pass_msg_bytes, size_t *part_msg_bytes);

/* Reads local q, k, v; writes pass_send (device, 16-byte aligned,
 * pass_msg_bytes): per slot the indices and the K and V rows of that chunk's
 * passing block. */
spava_status spava_shard_front(const spava_config *cfg, int32_t rank, int32_t world, const void *q,
                               const void *k, const void *v, void *pass_send, void *ws,
                               size_t ws_bytes, void *stream);

/* Writes the anchor rows of o / lse and part_send (device, part_msg_bytes):
 * the query rows' partials over this rank's chunks. */
spava_status spava_shard_local_attn(const spava_config *cfg, int32_t rank, int32_t world,
                                    const void *q, const void *k, const void *v, void *o, float *lse,
                                    void *part_send, void *ws, size_t ws_bytes, void *stream);

/* Reads pass_all (device, world * pass_msg_bytes, rank-major); writes the
 * context rows of this rank's chunks into o / lse, and, if idx_out != NULL,
 * every chunk's passing-block indices [2H-1, Hkv, l]. */
spava_status spava_shard_context_attn(const spava_config *cfg, int32_t rank, int32_t world,
                                      const void *q, const void *k, const void *v,
                                      const void *pass_all, void *o, float *lse, int32_t *idx_out,
                                      void *ws, size_t ws_bytes, void *stream);

/* Reads part_all (device, world * part_msg_bytes, rank-major); writes the
 * query rows of o / lse. */
spava_status spava_shard_merge(const spava_config *cfg, int32_t rank, int32_t world,
                               const void *part_all, void *o, float *lse, void *ws, size_t ws_bytes,
                               void *stream);

/* spava_score for callers that cannot allocate device memory: same inputs,
 * same scores output, no workspace argument.  (The pages have no counterpart:
 * this is an interface choice of the library, not part of the method.)
 * Who needs it: code that is handed only its input and output buffers, such
 * as a plug-in inside an engine that owns all device memory, or code that must
 * not allocate after start-up (real-time or certified deployments, or a
 * latency-critical path where cudaMalloc would synchronise the device).
 * The scratch for the per-chunk softmax statistics is a fixed 4 MiB array
 * compiled into the library (each GPU that loads the library holds it until
 * the process exits).  Limit: 256 + 4*(2H-1)*Hq*q bytes must fit in 4 MiB
 * (e.g. H=16, Hq=32, q=512 needs 2 MiB); larger layers get
 * SPAVA_ERR_WORKSPACE and nothing is launched.  No allocation of any kind
 * (no cudaMalloc, cudaFree or allocating library routine).
 * Each call looks up the array's device address with the calling thread's
 * current device (cudaGetSymbolAddress; the first lookup on a device loads the
 * library's module there): make the first call on a device before any stream
 * capture.
 * All calls share the one array: calls that overlap on the GPU (other streams,
 * other host threads) race and must be serialised by the caller.  A kernel
 * wait that gives up is recorded in the array's status word, which each call
 * clears at its start; read it with spava_score_noalloc_status. */
spava_status spava_score_noalloc(const spava_config *cfg, const void *q, const void *k,
                                 float *scores, void *stream);

/* Status of the last spava_score_noalloc call on the current device (the
 * pages have no counterpart): synchronises `stream`, reads the status word of
 * the library's fixed scratch array (bit 0: a bounded wait in a kernel gave
 * up, the scores are incomplete), writes it to *flags and clears it.  Returns
 * SPAVA_ERR_TIMEOUT if bit 0 was set, SPAVA_OK otherwise.  Allocates nothing. */
spava_status spava_score_noalloc_status(void *stream, int32_t *flags);

/* ---------------------------------------------------------------------------
 * The answering side: what a model runs around the prefill layer above.  (The
 * pages take post-rotary Q and K and stop at the prefill; these operators make
 * those inputs and answer from what the prefill leaves behind.)
 *
 *   spava_qk_norm_rope  RMS norm of every query and key head and the position
 *                       rotation, in one pass: the Q and K of a layer
 *   spava_cache_write   a layer's K and V rows into a paged cache, as bf16 or
 *                       quantised to e4m3
 *   spava_cache_append  both for new tokens: q normed and rotated, k normed,
 *                       rotated and cached, v cached, in one launch
 *   spava_cache_read    cached rows back as contiguous bf16
 *   spava_cache_attn    attention of one new token per sequence over the cache
 *
 * The conventions at the head of this file hold.  These calls may be captured
 * into CUDA graphs.  The current device must be the one of the buffers and the
 * stream.
 * ------------------------------------------------------------------------- */

/* For a token at position p (one per axis) and a head row x of d elements:
 *   y = x * w / sqrt(mean(x^2) + eps)            (norm 1; norm 0: y = x)
 *   pair j < rope_dim/2: angle = p[axis(j)] * inv_freq[j],
 *     (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)
 * and one rounding to bf16 at the end.  Angles are reduced in 64 bits, so far
 * positions keep their accuracy. */
typedef struct {
    int32_t n_q_heads;   /* Hq: 1..4096 */
    int32_t n_kv_heads;  /* Hkv >= 1, Hq % Hkv == 0 */
    int32_t head_dim;    /* d: 64 or 128 */
    int32_t rope_dim;    /* rotated elements, the first of the head: 0 or a multiple
                            of 16 up to d; the others pass through */
    int32_t interleaved; /* 0: pair j = elements (j, j + rope_dim/2); 1: (2j, 2j+1) */
    int32_t n_axes;      /* position axes: 1..4 */
    int32_t section[4];  /* the first section[0] pairs turn by axis 0's position, the
                            next section[1] by axis 1's, ...; >= 0, the first n_axes
                            sum to rope_dim/2 */
    int32_t norm;        /* 1: RMS norm; 0: none (eps and the weights are not used) */
    float eps;           /* >= 0 */
} spava_rope_config;

/* q [n_rows, Hq, d] and k [n_rows, Hkv, d] bf16, heads contiguous, tokens
 * q_stride and k_stride elements apart (at least Hq*d and Hkv*d, multiples of
 * 8: views of one fused projection are fine).  q_weight, k_weight: bf16 [d]
 * (NULL: ones).  inv_freq: float32 [rope_dim/2] (may be NULL if rope_dim is 0).
 * positions: int32 [n_axes, n_rows] (may be NULL if rope_dim is 0).
 * Writes q_out [n_rows, Hq, d] and k_out [n_rows, Hkv, d] contiguous; either
 * may be its input itself (same address, contiguous stride) and must not
 * overlap an input otherwise.  n_rows 0 is allowed and does nothing. */
spava_status spava_qk_norm_rope(const spava_rope_config *cfg, int64_t n_rows, const void *q,
                                int64_t q_stride, const void *k, int64_t k_stride,
                                const void *q_weight, const void *k_weight, const float *inv_freq,
                                const int32_t *positions, void *q_out, void *k_out, void *stream);

typedef enum {
    SPAVA_CACHE_BF16 = 0,
    SPAVA_CACHE_E4M3 = 1 /* e4m3 values with one int8 exponent per row */
} spava_cache_type;

/* A paged cache of one layer's keys and values.  Position t of a sequence lies
 * in row t % page_size of page table[t / page_size]. */
typedef struct {
    int32_t n_q_heads;  /* Hq (spava_cache_attn) */
    int32_t n_kv_heads; /* Hkv; Hq % Hkv == 0 */
    int32_t head_dim;   /* d: 64 or 128 */
    int32_t page_size;  /* rows per page: 1..65536 */
    int64_t n_pages;    /* >= 1; n_pages * Hkv * page_size < 2^32 - 1 */
    int32_t type;       /* a spava_cache_type */
    float scale;        /* softmax scale; <= 0 selects 1/sqrt(d) */
} spava_cache_config;

/* The caller's pools: k, v [n_pages, Hkv, page_size, d], bf16 or e4m3; for
 * e4m3 also k_exp, v_exp, int8 [n_pages, Hkv, page_size] (else not used).  A
 * row x is held as round_e4m3(x * 2^-e) and e, the smallest e >= -120 with
 * max|x| <= 448 * 2^e over its finite elements (-120 for a row of zeros): a
 * power of two leaves every significand as it is, so the row's only rounding
 * is the one to e4m3.  NaN and infinities are held as NaN. */
typedef struct {
    void *k;
    void *v;
    int8_t *k_exp;
    int8_t *v_exp;
} spava_cache_pools;

/* A batch of sequences, all DEVICE memory (so that a captured graph can be
 * replayed with other contents): table int32 [n_seqs, max_pages] and lens int32
 * [n_seqs], the tokens of each sequence, new ones included.  max_pages >= 1,
 * max_pages * page_size <= 2^31 - 2^16, n_seqs < 2^20; without sequences nothing is done
 * (table, lens and the rows' buffers may be NULL).  Table entries behind the last
 * page of a sequence may hold anything.  Sequences may share pages.  A length below
 * 0 counts as 0; of one beyond the table, what lies behind the table is neither
 * read nor written; a page outside the pool is neither read nor written, its
 * positions count as absent; each of the three sets bit 1 of the workspace status
 * word. */
typedef struct {
    int64_t n_seqs;
    int64_t max_pages;
    const int32_t *table;
    const int32_t *lens;
} spava_cache_batch;

/* Workspace bytes of the spava_cache_* calls for this config, whatever the
 * batch.  256-byte aligned; its first 256 bytes are the status block, whose
 * word must start at zero, the rest may hold anything.  Calls that share a
 * workspace must be ordered (on one stream, or by events). */
spava_status spava_cache_workspace_size(const spava_cache_config *cfg, size_t *bytes);

/* Writes new_rows rows of every sequence, its last ones: row i of sequence b
 * (token b * new_rows + i of k and v) goes to position lens[b] - new_rows + i;
 * rows whose position would be negative, or lies behind the table, are skipped.  k, v: [n_seqs *
 * new_rows, Hkv, d] bf16, tokens k_stride and v_stride elements apart (as in
 * spava_qk_norm_rope).  Two rows that go to one place of the pool leave
 * unspecified contents there.  Nothing else in the pools changes. */
spava_status spava_cache_write(const spava_cache_config *cfg, const spava_cache_pools *pools,
                               const spava_cache_batch *batch, int64_t new_rows, const void *k,
                               int64_t k_stride, const void *v, int64_t v_stride, void *ws,
                               size_t ws_bytes, void *stream);

/* spava_qk_norm_rope and spava_cache_write of its k_out and of v in one launch,
 * byte for byte: q_out [n_seqs * new_rows, Hq, d]; positions int32 [n_axes,
 * n_seqs * new_rows] are those of the rotation.  Head counts and head_dim of
 * both configs must agree. */
spava_status spava_cache_append(const spava_rope_config *rope, const spava_cache_config *cfg,
                                const spava_cache_pools *pools, const spava_cache_batch *batch,
                                int64_t new_rows, const void *q, int64_t q_stride, const void *k,
                                int64_t k_stride, const void *v, int64_t v_stride,
                                const void *q_weight, const void *k_weight, const float *inv_freq,
                                const int32_t *positions, void *q_out, void *ws, size_t ws_bytes,
                                void *stream);

/* Positions [first, first + rows) of every sequence as bf16, k_out and v_out
 * [n_seqs, rows, Hkv, d]: e4m3 rows as value * 2^e (exact in bf16; infinite
 * where e4m3 rounded a value next to bf16's largest up past it); zeros from
 * position lens[b] on.  first >= 0, first + rows < 2^31. */
spava_status spava_cache_read(const spava_cache_config *cfg, const spava_cache_pools *pools,
                              const spava_cache_batch *batch, int64_t first, int64_t rows,
                              void *k_out, void *v_out, void *ws, size_t ws_bytes, void *stream);

/* Attention of one query token per sequence, q [n_seqs, Hq, d] bf16, over the
 * sequence's positions [0, lens[b]):
 *   o[b, h] = sum_t softmax_t(scale * q[b, h] . k[t, h / (Hq/Hkv)]) v[t]
 * o [n_seqs, Hq, d] bf16; lse (may be NULL) float32 [Hq, n_seqs], natural log:
 * with it, partial results over parts of a context can be merged.  A sequence
 * without positions gives o = 0 and lse = -inf.  Scores, sums and outputs are
 * held in 32 bits; the softmax weights enter the product with the values with 16
 * significant bits (22 over an e4m3 cache) and o is rounded once.  Positions past
 * lens[b] are never read, whatever they hold.  Several new tokens of one sequence are
 * several rows of the batch, with the same table row and growing lens.
 * Results do not depend on timing: the same call gives the same bytes.
 * SPAVA_ERR_UNSUPPORTED if the tables hold 2^31 work units or more (a unit is
 * 32 KiB of K and V rows of one KV head and 16, or 8, query heads). */
spava_status spava_cache_attn(const spava_cache_config *cfg, const spava_cache_pools *pools,
                              const spava_cache_batch *batch, const void *q, void *o, float *lse,
                              void *ws, size_t ws_bytes, void *stream);

const char *spava_status_string(spava_status s);

/* The CUDA error code of this thread's last SPAVA_ERR_CUDA (0 if none). */
int32_t spava_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* SPAVA_H_ */
