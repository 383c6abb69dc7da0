// cache_api.cu -- the C ABI's answering side (include/spava.h): argument checks
// and launches of the norm/rotation, paged cache and one-token attention
// kernels.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "../../include/spava.h"
#include "cache_common.cuh"
#include "decode_kernel.cuh"
#include "row_kernels.cuh"
#include "status.cuh"

using namespace spava;

namespace {

spava_status check_heads(int32_t Hq, int32_t Hkv, int32_t d) {
    if (Hq < 1 || Hkv < 1 || d < 1 || Hq % Hkv) return SPAVA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return SPAVA_ERR_UNSUPPORTED;
    if (Hq > 4096) return SPAVA_ERR_UNSUPPORTED;
    return SPAVA_OK;
}

spava_status check_rope(const spava_rope_config *c) {
    if (!c) return SPAVA_ERR_INVALID_ARG;
    SPAVA_TRY(check_heads(c->n_q_heads, c->n_kv_heads, c->head_dim));
    if (c->rope_dim < 0 || c->rope_dim > c->head_dim) return SPAVA_ERR_INVALID_ARG;
    if (c->rope_dim % 2) return SPAVA_ERR_INVALID_ARG;
    if (c->rope_dim % 16) return SPAVA_ERR_UNSUPPORTED;
    if (c->interleaved != 0 && c->interleaved != 1) return SPAVA_ERR_INVALID_ARG;
    if (c->norm != 0 && c->norm != 1) return SPAVA_ERR_INVALID_ARG;
    if (c->norm && !(c->eps >= 0.f && std::isfinite(c->eps))) return SPAVA_ERR_INVALID_ARG;
    if (c->n_axes < 1) return SPAVA_ERR_INVALID_ARG;
    if (c->n_axes > 4) return SPAVA_ERR_UNSUPPORTED;
    int64_t sum = 0;
    for (int a = 0; a < c->n_axes; ++a) {
        if (c->section[a] < 0) return SPAVA_ERR_INVALID_ARG;
        sum += c->section[a];
    }
    return sum == c->rope_dim / 2 ? SPAVA_OK : SPAVA_ERR_INVALID_ARG;
}

spava_status check_cache(const spava_cache_config *c) {
    if (!c) return SPAVA_ERR_INVALID_ARG;
    SPAVA_TRY(check_heads(c->n_q_heads, c->n_kv_heads, c->head_dim));
    if (c->page_size < 1 || c->n_pages < 1) return SPAVA_ERR_INVALID_ARG;
    if (c->type != SPAVA_CACHE_BF16 && c->type != SPAVA_CACHE_E4M3) return SPAVA_ERR_INVALID_ARG;
    if (c->page_size > 65536) return SPAVA_ERR_UNSUPPORTED;
    if (!std::isfinite(c->scale)) return SPAVA_ERR_INVALID_ARG;
    const int64_t per_page = int64_t(c->n_kv_heads) * c->page_size;
    if (c->n_pages > (int64_t(kNoRow) - 1) / per_page) return SPAVA_ERR_UNSUPPORTED;
    return SPAVA_OK;
}

// A token source: heads contiguous, tokens `stride` elements apart.
spava_status check_rows(const void *p, int64_t stride, int heads, int d) {
    SPAVA_TRY(check_ptr(p));
    if (stride < int64_t(heads) * d) return SPAVA_ERR_INVALID_ARG;
    return stride % 8 ? SPAVA_ERR_MISALIGNED : SPAVA_OK;
}

constexpr size_t kCutBytes = sizeof(int4) * kDecMaxCtas;

// Query heads of a KV head in tiles of 8, or two tiles at a time: more than 8 in
// two goes would read the rows twice (262144 tokens, 16 heads on one: 31.5 us, 39.7
// in two goes), while two tiles cost registers that fewer heads do not need.
int head_tile(const spava_cache_config *c) { return c->n_q_heads / c->n_kv_heads > 8 ? 2 : 1; }

// [status block 256 | cut items | partial statistics | partial O]
size_t cache_ws_bytes(const spava_cache_config *c) {
    const size_t heads = 8 * head_tile(c);
    return 256 + kCutBytes + sizeof(float) * 2 * kDecMaxCtas * heads * (3 + c->head_dim);
}

spava_status make_view(const spava_cache_config *c, const spava_cache_pools *p,
                       const spava_cache_batch *b, void *ws, size_t ws_bytes, CacheView *v) {
    SPAVA_TRY(check_cache(c));
    if (!p || !b) return SPAVA_ERR_INVALID_ARG;
    if (b->n_seqs < 0 || b->max_pages < 1) return SPAVA_ERR_INVALID_ARG;
    if (b->n_seqs >= (1LL << 20)) return SPAVA_ERR_UNSUPPORTED;
    if (b->max_pages > ((1LL << 31) - 65536) / c->page_size) return SPAVA_ERR_UNSUPPORTED;
    SPAVA_TRY(check_ptr(p->k));
    SPAVA_TRY(check_ptr(p->v));
    if (c->type == SPAVA_CACHE_E4M3) {
        SPAVA_TRY(check_ptr(p->k_exp));
        SPAVA_TRY(check_ptr(p->v_exp));
    }
    if (b->n_seqs > 0 && (!b->table || !b->lens)) return SPAVA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(b->table) & 3) || (reinterpret_cast<uintptr_t>(b->lens) & 3))
        return SPAVA_ERR_MISALIGNED;
    if (!ws) return SPAVA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(ws) & 255) return SPAVA_ERR_MISALIGNED;
    if (ws_bytes < cache_ws_bytes(c)) return SPAVA_ERR_WORKSPACE;
    v->k = p->k;
    v->v = p->v;
    v->k_exp = p->k_exp;
    v->v_exp = p->v_exp;
    v->table = b->table;
    v->lens = b->lens;
    v->status = static_cast<int *>(ws);
    v->max_pages = b->max_pages;
    v->n_pages = static_cast<uint32_t>(std::min<int64_t>(c->n_pages, INT32_MAX));
    v->n_rows = static_cast<uint32_t>(c->n_pages * c->n_kv_heads * c->page_size);
    v->n_seqs = static_cast<int32_t>(b->n_seqs);
    v->Hkv = c->n_kv_heads;
    v->cap = static_cast<int32_t>(b->max_pages * c->page_size);
    v->page = FastDiv::of(static_cast<uint32_t>(c->page_size));
    return SPAVA_OK;
}

// Tokens of a block (a power of two up to `most`) and blocks that share their
// items, per_pass of which a block works on at a time: enough tokens to fill a
// pass, then more where there are plenty, as a block's tokens share what it makes
// for them; few tokens are spread over the SMs head by head.  (Norm, rotation and
// write of 64 tokens, 48 heads: 3.1 us, 10.5 with eight tokens a block and no
// sharing out.  Norm of 131072 tokens: 350 us, 363 with four tokens a block; of 5000:
// 18.4 us, 20.8 where half as many blocks are plenty.)
void split_tokens(int64_t n_rows, int64_t heads, int most, int per_pass, int32_t *tokens_log2, int64_t *splits) {
    constexpr int kBlocks = 148 * 4;  // enough to fill the SMs
    constexpr int kPlenty = 2 * kBlocks;
    int lg = 0;
    while ((2 << lg) <= most && (((heads << lg) < per_pass && (1LL << lg) < n_rows) ||
                                 ((n_rows >> (lg + 1)) >= kPlenty && (heads << (lg + 1)) <= 8 * per_pass)))
        ++lg;
    const int64_t groups = (n_rows + (1LL << lg) - 1) >> lg, passes = ((heads << lg) + per_pass - 1) / per_pass;
    *tokens_log2 = lg;
    *splits = std::max<int64_t>(1, std::min(passes, kBlocks / groups));
}

template <int CACHE, bool ROPE>
spava_status launch_rows(RowParams &p, int d, cudaStream_t st) {
    const int64_t heads = int64_t(p.Hq) + p.Hk + p.Hv;
    if (p.n_rows == 0) return SPAVA_OK;
    if (p.n_rows >= (1LL << 31) / heads) return SPAVA_ERR_UNSUPPORTED;
    int64_t splits;
    split_tokens(p.n_rows, heads, ROPE ? kRowTokens : kWriteTokens, kRowThreads / (d / 16), &p.tokens_log2, &splits);
    p.splits = FastDiv::of(static_cast<uint32_t>(splits));
    const int64_t groups = (p.n_rows + (1LL << p.tokens_log2) - 1) >> p.tokens_log2;
    return launch(d == 64 ? row_kernel<64, CACHE, ROPE> : row_kernel<128, CACHE, ROPE>,
                  static_cast<unsigned>(groups * splits), kRowThreads, 0, 1, st, p);
}

spava_status set_rope(const spava_rope_config *c, RowParams *p, const void *q_weight,
                      const void *k_weight, const float *inv_freq, const int32_t *positions) {
    if (c->norm) {
        SPAVA_TRY(check_ptr(q_weight, false));
        SPAVA_TRY(check_ptr(k_weight, false));
    }
    if (c->rope_dim > 0) {
        if (!inv_freq || !positions) return SPAVA_ERR_INVALID_ARG;
        if ((reinterpret_cast<uintptr_t>(inv_freq) & 3) || (reinterpret_cast<uintptr_t>(positions) & 3))
            return SPAVA_ERR_MISALIGNED;
    }
    p->q_weight = static_cast<const __nv_bfloat16 *>(q_weight);
    p->k_weight = static_cast<const __nv_bfloat16 *>(k_weight);
    p->inv_freq = inv_freq;
    p->positions = positions;
    p->rope_dim = c->rope_dim;
    p->interleaved = c->interleaved;
    p->norm = c->norm;
    p->eps = c->eps;
    int32_t cut[4], at = 0;
    for (int a = 0; a < 4; ++a) cut[a] = a < c->n_axes ? (at += c->section[a]) : INT32_MAX;
    // the last axis in use ends at rope_dim / 2: no pair lies behind it
    p->cut1 = cut[0];
    p->cut2 = cut[1];
    p->cut3 = cut[2];
    return SPAVA_OK;
}

spava_status check_batch_rows(const spava_cache_batch *b, int64_t new_rows) {
    if (new_rows < 0) return SPAVA_ERR_INVALID_ARG;
    if (new_rows >= (1LL << 31)) return SPAVA_ERR_UNSUPPORTED;
    return SPAVA_OK;
}

template <typename K>
spava_status set_dynamic_smem(K kernel, int bytes, std::atomic<uint64_t> &done, int dev) {
    // once a device: the attribute belongs to the function there
    const uint64_t bit = dev < 64 ? 1ULL << dev : 0;
    if (bit && (done.load(std::memory_order_acquire) & bit)) return SPAVA_OK;
    SPAVA_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    done.fetch_or(bit, std::memory_order_release);
    return SPAVA_OK;
}

// Whether decode_cluster_kernel takes a batch, of `blocks` blocks with tables of at
// most `kib` KiB of K and V rows each.  A block streams 50 KiB a us, all of them
// 6500, and the line's second launch and join cost 2.3 us more: clusters win where
// kib / 50 < 2.3 + blocks * kib / 6500 -- if the sequences are as long as their
// tables; the lengths are not known here, and 256 KiB bound what that can cost.
// By the line / by clusters, device time in us, bf16, 4 KV heads: one sequence (32
// blocks) of 512 tokens 6.8 / 4.9, 2048 (128 KiB) 7.3 / 6.7, 4096 7.4 / 9.4; 4
// sequences (128 blocks) of 4096 13.4 / 11.7; 16 (256 blocks) of 1024 11.5 / 9.4.
bool by_clusters(int64_t blocks, int64_t kib) { return kib <= 256 && kib * (130 - blocks) <= 15000; }

// Whether decode_warp_kernel takes a batch, whose tables hold at most `tiles` tiles
// (8 KiB of K and V rows): always up to two, up to 8 where there are too many items
// for clusters, up to 16 where there are many more.  By the line or clusters / by
// warps, device time in us: one sequence of 32 tokens, 4 KV heads, bf16 4.3 / 3.2
// (of 64, four tiles, 4.4 / 4.4); 100 sequences of 64, 8 KV heads, e4m3 13.8 / 6.1;
// 40 of 500 (320 items, 16 tiles) 17.2 / 23.4, 100 (800 items) 29.5 / 26.3.
bool by_warps(int64_t tiles, int64_t items, int64_t slots) {
    return tiles <= (items <= slots ? 2 : items < 2 * slots ? 8 : 16);
}

template <int D, bool E4M3, int NT>
spava_status launch_decode(DecodeParams &p, int64_t max_units, cudaStream_t st) {
    using S = DecodeShape<D, E4M3, NT>;
    static std::atomic<uint64_t> done{0}, cluster_done{0}, warp_done{0};
    int dev = 0, n_sm = 0;
    SPAVA_CUDA(cudaGetDevice(&dev));
    SPAVA_CUDA(cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev));
    const int64_t items = int64_t(p.cache.n_seqs) * p.cache.Hkv * p.n_hg;
    p.cluster = kDecCluster;
    while (p.cluster > 1 && items * p.cluster > 2 * n_sm) p.cluster /= 2;
    const int64_t blocks = items * p.cluster;
    if (by_warps((p.cache.cap + S::TT - 1) / S::TT, items, 2 * n_sm) && items < (1LL << 31)) {
        SPAVA_TRY(set_dynamic_smem(decode_warp_kernel<D, E4M3, NT>, S::SMEM, warp_done, dev));
        return launch(decode_warp_kernel<D, E4M3, NT>, static_cast<unsigned>((items + kDecWarps - 1) / kDecWarps),
                      kDecThreads, S::SMEM, 1, st, p);
    }
    if (blocks <= 2 * n_sm && by_clusters(blocks, int64_t(p.cache.cap) * 2 * S::ROW / 1024 / p.cluster)) {
        SPAVA_TRY(set_dynamic_smem(decode_cluster_kernel<D, E4M3, NT>, S::SMEM, cluster_done, dev));
        return launch(decode_cluster_kernel<D, E4M3, NT>, static_cast<unsigned>(blocks), kDecThreads,
                      S::SMEM, p.cluster, st, p);
    }
    SPAVA_TRY(set_dynamic_smem(decode_kernel<D, E4M3, NT>, S::SMEM, done, dev));
    // no more blocks than the units of full tables
    const int grid = static_cast<int>(std::min<int64_t>(std::min(2 * n_sm, kDecMaxCtas), max_units));
    p.cuts_by_item = items <= grid;
    SPAVA_TRY(launch(decode_kernel<D, E4M3, NT>, grid, kDecThreads, S::SMEM, 1, st, p));
    const int cuts = static_cast<int>(std::min<int64_t>(items, grid));
    // Items of 16 parts and more are split further (131072 tokens on 4 KV heads,
    // 74 parts: 48.4 us, 59.5 without; 16 sequences on one, 18 parts: 35.1, 41.0;
    // 32 items of 9 parts: 51.1, 48.8 without).
    const bool split = items * 16 <= grid;
    constexpr int kSplitBlocks = 8 * NT * (D / 32), kBlocks = 8 * NT * D / 4 / kDecThreads;  // of an item
    return launch(split ? join_kernel<D, NT, true> : join_kernel<D, NT, false>, cuts * (split ? kSplitBlocks : kBlocks),
                  split ? kJoinThreads : kDecThreads, 0, 1, st, p);
}

}  // namespace

extern "C" {

spava_status spava_qk_norm_rope(const spava_rope_config *cfg, int64_t n_rows, const void *q,
                                int64_t q_stride, const void *k, int64_t k_stride,
                                const void *q_weight, const void *k_weight, const float *inv_freq,
                                const int32_t *positions, void *q_out, void *k_out, void *stream) {
    SPAVA_TRY(check_rope(cfg));
    if (n_rows < 0) return SPAVA_ERR_INVALID_ARG;
    if (n_rows == 0) return SPAVA_OK;
    SPAVA_TRY(check_rows(q, q_stride, cfg->n_q_heads, cfg->head_dim));
    SPAVA_TRY(check_rows(k, k_stride, cfg->n_kv_heads, cfg->head_dim));
    SPAVA_TRY(check_ptr(q_out));
    SPAVA_TRY(check_ptr(k_out));
    RowParams p{};
    SPAVA_TRY(set_rope(cfg, &p, q_weight, k_weight, inv_freq, positions));
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.k_out = static_cast<__nv_bfloat16 *>(k_out);
    p.n_rows = n_rows;
    p.Hq = cfg->n_q_heads;
    p.Hk = cfg->n_kv_heads;
    return launch_rows<0, true>(p, cfg->head_dim, static_cast<cudaStream_t>(stream));
}

spava_status spava_cache_workspace_size(const spava_cache_config *cfg, size_t *bytes) {
    if (!bytes) return SPAVA_ERR_INVALID_ARG;
    SPAVA_TRY(check_cache(cfg));
    *bytes = cache_ws_bytes(cfg);
    return SPAVA_OK;
}

spava_status spava_cache_write(const spava_cache_config *cfg, const spava_cache_pools *pools,
                               const spava_cache_batch *batch, int64_t new_rows, const void *k,
                               int64_t k_stride, const void *v, int64_t v_stride, void *ws,
                               size_t ws_bytes, void *stream) {
    RowParams p{};
    SPAVA_TRY(make_view(cfg, pools, batch, ws, ws_bytes, &p.cache));
    SPAVA_TRY(check_batch_rows(batch, new_rows));
    if (new_rows == 0 || batch->n_seqs == 0) return SPAVA_OK;
    SPAVA_TRY(check_rows(k, k_stride, cfg->n_kv_heads, cfg->head_dim));
    SPAVA_TRY(check_rows(v, v_stride, cfg->n_kv_heads, cfg->head_dim));
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.n_rows = batch->n_seqs * new_rows;
    p.new_rows = FastDiv::of(static_cast<uint32_t>(new_rows));
    p.Hk = p.Hv = cfg->n_kv_heads;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cfg->type == SPAVA_CACHE_E4M3 ? launch_rows<2, false>(p, cfg->head_dim, st)
                                         : launch_rows<1, false>(p, cfg->head_dim, st);
}

spava_status spava_cache_append(const spava_rope_config *rope, const spava_cache_config *cfg,
                                const spava_cache_pools *pools, const spava_cache_batch *batch,
                                int64_t new_rows, const void *q, int64_t q_stride, const void *k,
                                int64_t k_stride, const void *v, int64_t v_stride,
                                const void *q_weight, const void *k_weight, const float *inv_freq,
                                const int32_t *positions, void *q_out, void *ws, size_t ws_bytes,
                                void *stream) {
    SPAVA_TRY(check_rope(rope));
    RowParams p{};
    SPAVA_TRY(make_view(cfg, pools, batch, ws, ws_bytes, &p.cache));
    if (rope->n_q_heads != cfg->n_q_heads || rope->n_kv_heads != cfg->n_kv_heads ||
        rope->head_dim != cfg->head_dim)
        return SPAVA_ERR_INVALID_ARG;
    SPAVA_TRY(check_batch_rows(batch, new_rows));
    if (new_rows == 0 || batch->n_seqs == 0) return SPAVA_OK;
    SPAVA_TRY(check_rows(q, q_stride, cfg->n_q_heads, cfg->head_dim));
    SPAVA_TRY(check_rows(k, k_stride, cfg->n_kv_heads, cfg->head_dim));
    SPAVA_TRY(check_rows(v, v_stride, cfg->n_kv_heads, cfg->head_dim));
    SPAVA_TRY(check_ptr(q_out));
    SPAVA_TRY(set_rope(rope, &p, q_weight, k_weight, inv_freq, positions));
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.n_rows = batch->n_seqs * new_rows;
    p.new_rows = FastDiv::of(static_cast<uint32_t>(new_rows));
    p.Hq = cfg->n_q_heads;
    p.Hk = p.Hv = cfg->n_kv_heads;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cfg->type == SPAVA_CACHE_E4M3 ? launch_rows<2, true>(p, cfg->head_dim, st)
                                         : launch_rows<1, true>(p, cfg->head_dim, st);
}

spava_status spava_cache_read(const spava_cache_config *cfg, const spava_cache_pools *pools,
                              const spava_cache_batch *batch, int64_t first, int64_t rows,
                              void *k_out, void *v_out, void *ws, size_t ws_bytes, void *stream) {
    ReadParams p{};
    SPAVA_TRY(make_view(cfg, pools, batch, ws, ws_bytes, &p.cache));
    if (first < 0 || rows < 0) return SPAVA_ERR_INVALID_ARG;
    if (first >= (1LL << 31) || rows >= (1LL << 31) || first + rows >= (1LL << 31))
        return SPAVA_ERR_UNSUPPORTED;
    if (rows == 0 || batch->n_seqs == 0) return SPAVA_OK;
    SPAVA_TRY(check_ptr(k_out));
    SPAVA_TRY(check_ptr(v_out));
    const int64_t heads = cfg->n_kv_heads;
    if (batch->n_seqs * rows >= (1LL << 31) / heads) return SPAVA_ERR_UNSUPPORTED;
    p.k_out = static_cast<__nv_bfloat16 *>(k_out);
    p.v_out = static_cast<__nv_bfloat16 *>(v_out);
    p.first = static_cast<int32_t>(first);
    p.n_rows = batch->n_seqs * rows;
    p.rows = FastDiv::of(static_cast<uint32_t>(rows));
    p.heads = FastDiv::of(static_cast<uint32_t>(heads));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool e4m3 = cfg->type == SPAVA_CACHE_E4M3;
    int64_t splits;
    split_tokens(p.n_rows, heads, kReadTokens, kRowThreads / (cfg->head_dim / 8), &p.tokens_log2, &splits);
    p.splits = FastDiv::of(static_cast<uint32_t>(splits));
    const unsigned grid = static_cast<unsigned>(((p.n_rows + (1LL << p.tokens_log2) - 1) >> p.tokens_log2) * splits);
    void (*const kernels[4])(ReadParams) = {read_kernel<64, false>, read_kernel<64, true>,
                                            read_kernel<128, false>, read_kernel<128, true>};
    return launch(kernels[(cfg->head_dim == 128 ? 2 : 0) + (e4m3 ? 1 : 0)], grid, kRowThreads, 0, 1, st, p);
}

spava_status spava_cache_attn(const spava_cache_config *cfg, const spava_cache_pools *pools,
                              const spava_cache_batch *batch, const void *q, void *o, float *lse,
                              void *ws, size_t ws_bytes, void *stream) {
    DecodeParams p{};
    SPAVA_TRY(make_view(cfg, pools, batch, ws, ws_bytes, &p.cache));
    if (batch->n_seqs == 0) return SPAVA_OK;
    SPAVA_TRY(check_ptr(q));
    SPAVA_TRY(check_ptr(o));
    if (reinterpret_cast<uintptr_t>(lse) & 3) return SPAVA_ERR_MISALIGNED;
    const int nt = head_tile(cfg);
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.lse = lse;
    p.Hq = cfg->n_q_heads;
    p.G = cfg->n_q_heads / cfg->n_kv_heads;
    p.n_hg = (p.G + 8 * nt - 1) / (8 * nt);
    const double scale = cfg->scale > 0.f ? double(cfg->scale) : 1.0 / std::sqrt(double(cfg->head_dim));
    p.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
    char *at = static_cast<char *>(ws) + 256;
    p.cuts = reinterpret_cast<int4 *>(at);
    p.part_stat = reinterpret_cast<float *>(at + kCutBytes);
    p.part_o = p.part_stat + size_t(2) * kDecMaxCtas * 3 * 8 * nt;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool e4m3 = cfg->type == SPAVA_CACHE_E4M3;
    // the units of a batch of full tables are counted in 32 bits
    const int64_t block = int64_t(kDecWarps) * kDecTileBytes / (2 * cfg->head_dim * (e4m3 ? 1 : 2));
    const int64_t units = ((p.cache.cap + block - 1) / block + kDecItemCost) * cfg->n_kv_heads * p.n_hg;
    if (units >= (1LL << 31) / batch->n_seqs) return SPAVA_ERR_UNSUPPORTED;
    const int64_t all = units * batch->n_seqs;
    if (cfg->head_dim == 64) {
        if (e4m3) return nt == 1 ? launch_decode<64, true, 1>(p, all, st) : launch_decode<64, true, 2>(p, all, st);
        return nt == 1 ? launch_decode<64, false, 1>(p, all, st) : launch_decode<64, false, 2>(p, all, st);
    }
    if (e4m3) return nt == 1 ? launch_decode<128, true, 1>(p, all, st) : launch_decode<128, true, 2>(p, all, st);
    return nt == 1 ? launch_decode<128, false, 1>(p, all, st) : launch_decode<128, false, 2>(p, all, st);
}

}  // extern "C"
