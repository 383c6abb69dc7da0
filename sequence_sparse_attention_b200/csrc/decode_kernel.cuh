// decode_kernel.cuh -- attention of one new token per sequence over the paged
// cache: along a line of equal shares (decode_kernel, whose parts join_kernel
// joins), an item a cluster (decode_cluster_kernel) or an item a warp
// (decode_warp_kernel), as the batch and its tables' room have it.
#pragma once

#include "cache_common.cuh"

namespace spava {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kJoinThreads = 256;  // of a join block that shares its parts out
constexpr int kDecCluster = 8;     // most blocks of decode_cluster_kernel's clusters
constexpr int kDecMaxCtas = 320;   // the workspace's partials are sized for these
// Beginning and ending an item takes a block about as long as two units of its
// tokens, and counts as that: 17 sequences of 100 to 16100 tokens take 55 us, 70
// where only tokens count and some block gets the many short items (e4m3, 8 KV heads).
constexpr int kDecItemCost = 2;
constexpr int kDecStages = 3;
constexpr int kDecTileBytes = 8192;  // K and V bytes of one warp's tile
constexpr int kDecRingBytes = kDecWarps * kDecStages * kDecTileBytes;
constexpr int kDecPageSlots = kDecStages + 1;  // tiles whose table entries are under way

struct DecodeParams {
    CacheView cache;
    const __nv_bfloat16 *q;
    __nv_bfloat16 *o;
    float *lse;
    int32_t Hq, G;        // query heads, per KV head
    int32_t cluster;      // blocks of an item (decode_cluster_kernel): 1, 2, 4 or 8
    int32_t n_hg;         // groups of 8 * NT query heads that share a KV head
    float scale_log2;     // softmax scale * log2 e
    // [min(items, grid)]: an item's first block and number of parts, or of the
    // item that is cut and begins in a block's share where those are fewer; no
    // parts: not cut.  And its sequence and head group.
    int4 *cuts;
    int32_t cuts_by_item;
    float *part_stat;     // [8 * NT][3][2][kDecMaxCtas]: m, lm, l of a block's first and second part
    float *part_o;        // [2 * kDecMaxCtas][8 * NT][D]
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "r"(a)
                 : "memory");
    return r;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
    return r;
}
__device__ __forceinline__ uint32_t lds4(uint32_t a) {
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
    return r;
}
__device__ __forceinline__ void sts4(uint32_t a, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
template <bool HALF>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    if (HALF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t half2_bits(const __half2 &h) { return *reinterpret_cast<const uint32_t *>(&h); }
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) { return half2_bits(__floats2half2_rn(lo, hi)); }
__device__ __forceinline__ uint32_t scale_half2(uint32_t a, float f) {
    return half2_bits(__hmul2(*reinterpret_cast<const __half2 *>(&a), __float2half2_rn(f)));
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_address(const void *mine, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(mine))), "r"(rank));
    return r;
}
__device__ __forceinline__ float cluster_load(uint32_t a) {
    float r;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r) : "r"(a) : "memory");
    return r;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t a) {
    float4 r;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w)
                 : "r"(a)
                 : "memory");
    return r;
}
__device__ __forceinline__ void add_part(float4 &o, const float4 &y, float f) {
    o.x = fmaf(y.x, f, o.x), o.y = fmaf(y.y, f, o.y);
    o.z = fmaf(y.z, f, o.z), o.w = fmaf(y.w, f, o.w);
}

// The state of a softmax over part of a context, in base 2: l = sum 2^(s - lm),
// O = sum 2^(s + e - m) v with e the value's exponent (m = lm where there is
// none).  kDecNone marks a part without a finite score.
constexpr float kDecNone = -3.402823466e38f;
// How far a score may pass its reference before that follows.
constexpr float kDecLag = 8.f;
// e4m3: m lies this far below the largest s + e, as fp16 holds weights of up to
// 2^(kDecLift + kDecLag) and small ones need its range downwards.  What the rounding
// to fp16 leaves of a weight enters by a second product, kDecLow times as large.
constexpr float kDecLift = 7.f, kDecLow = 2048.f;

__device__ __forceinline__ void store_lse(const DecodeParams &p, int b, int head, float lm, float l) {
    if (p.lse)
        p.lse[static_cast<int64_t>(head) * p.cache.n_seqs + b] =
            l == 0.f ? -INFINITY : 0.6931471805599453f * (lm + log2f(l));
}
// The output's element of O's: times 2^(m - lm), over l.  Their product may lie below the normal range
// where neither they nor the output do (values of 2^-117, many tokens), so they are
// applied one after the other.
struct OutputScale {
    float inv, pow;
    __device__ __forceinline__ OutputScale(float m, float lm, float l)
        : inv(l == 0.f ? 0.f : 1.f / l), pow(l == 0.f ? 0.f : exp2f(m - lm)) {}
    __device__ __forceinline__ float operator()(float o) const { return o * inv * pow; }
};
// Four elements of a query head's output, and with the first its lse, from the
// whole context's state.
template <int D>
__device__ __forceinline__ void store_result(const DecodeParams &p, int b, int head, int d, float m, float lm,
                                             float l, const float4 &o) {
    const OutputScale f(m, lm, l);
    *reinterpret_cast<uint2 *>(p.o + (static_cast<int64_t>(b) * p.Hq + head) * D + d) =
        make_uint2(bf_pack(f(o.x), f(o.y)), bf_pack(f(o.z), f(o.w)));
    if (d == 0) store_lse(p, b, head, lm, l);
}

// How decode_body's work is shared out: along the line, an item to a cluster, an
// item to a warp.
enum class DecodeMode { kLine, kCluster, kWarp };

template <int D, bool E4M3, int NT>
struct DecodeShape {
    static constexpr int ROW = D * (E4M3 ? 1 : 2);         // bytes of a cached row
    static constexpr int TT = kDecTileBytes / (2 * ROW);   // tokens of a warp's tile
    static constexpr int SUB = TT / 16;                    // MMA tiles of 16 tokens
    static constexpr int BLOCK = TT * kDecWarps;           // tokens of a work unit
    static constexpr int LPR = ROW / 16;                   // lanes that copy a row
    static constexpr int RPI = 32 / LPR;                   // rows that a copy instruction of the warp takes
    static constexpr int KJ = ROW / 64;                    // 16-byte pieces of a K row per lane
    static constexpr int VB = ROW / 8;                     // bytes of a V row per lane
    static constexpr int KS = D / 16;                      // k steps of a score
    static constexpr int MT = D / 16;                      // 16-row tiles of O^T
    static constexpr int HEADS = 8 * NT;
    // The low products of an e4m3 cache have accumulators of their own where the
    // registers hold them; else the values are made kDecLow times smaller for them,
    // which is exact in fp16 (512 sequences of 2000 tokens, 4 heads a KV head: 327 us,
    // 348 with smaller values; two tiles of heads are at 255 registers without).
    static constexpr bool APART = E4M3 && NT == 1;
    // The 16-byte pieces of a row lie permuted (piece ^ swizzle) so that the
    // eight lanes that read at a time, pieces c of the K rows g, g + 1 or pieces
    // g, g + 1 of the V rows 2c, meet all banks.
    __host__ __device__ static constexpr int k_swizzle(int row) { return ROW >= 128 ? (row & 1) * 4 : 0; }
    __host__ __device__ static constexpr int v_swizzle(int row) {
        return ROW >= 128 ? (row >> 1 & 3) * 2 : row >> 1 & 3;
    }
    // Element of O that a lane of group g holds of tile i, and behind it the next one.
    __host__ __device__ static constexpr int column(int i, int g) {
        return E4M3 ? D / 8 * g + 2 * i : 64 * (i / 4) + 8 * g + 2 * (i % 4);
    }
    static constexpr int OPAD = D + 4;                     // floats of an O row in shared memory
    // The ring is free when a segment ends, and takes the warps' O and statistics.
    static constexpr int MERGE = kDecWarps * HEADS * (OPAD + 3) * 4;
    static constexpr int RING = MERGE > kDecRingBytes ? MERGE : kDecRingBytes;
    // behind it: table entries and, of an e4m3 cache, the words with the rows' exponents
    static constexpr int RW = TT == 64 ? 2 : 1;            // tokens of a tile per lane
    static constexpr int PAGES = kDecPageSlots * RW * 128;         // bytes, a warp
    static constexpr int EXPS = E4M3 ? kDecStages * RW * 2 * 128 : 0;
    static constexpr int SMEM = RING + kDecWarps * (PAGES + EXPS);
};

// What bounds it: every cached row is read once, D bytes or 2 D, and takes
// 4 G D operations, G the query heads of a KV head -- far below what the tensor
// cores do per byte of HBM, so the kernel is a read of the cache with
// arithmetic beside it, and all choices keep that read running:
//
//   - Every warp copies its own tiles with cp.async, row by row, into a ring of
//     its own: no block barrier in the loop, no address constraint but 16
//     bytes, so pages may have any size and end inside a tile.  Each copy
//     instruction takes 512 contiguous bytes where rows follow each other
//     (measured, 268 MB: 42 us; lanes that copy just what they will read
//     themselves, V rows at 512 bytes' stride: 58 us).  The contraction order
//     over d is free, so a lane reads 16 contiguous bytes of a K row for two to
//     four k steps; O's rows are permuted likewise for V.
//   - Transposed products, S^T = K Q^T and O^T = V^T P^T: tokens (or d) take
//     the 16-row side of an MMA and the query heads the 8-column side, so G = 7
//     or 4 wastes little, and the accumulators are 4 NT D / 16 registers.
//   - Softmax against a reference that may lag the maximum by 2^8: then a tile
//     needs one vote and no shuffles, and O is rescaled only when a score
//     passes that.  Sums and O stay in fp32.
//   - bf16: P enters as hi + lo, two bf16 products, 16 significant bits: one
//     bf16 rounding of P would cost as much as the rounding of the output.
//     e4m3: K, V and the scaled q are fp16 (e4m3 is exact in it) and P two fp16
//     products, 22 significant bits down to 2^-25 of the largest weight and steps of
//     2^-42 of it below.  A row's scales come in as exponents: of K into the score,
//     of V into P, whose reference m then covers score + exponent, while the sum
//     l has its own, lm.  (One product, 11 bits: 512 sequences of 2000 tokens 325
//     instead of 328 us.)
//   - The work of the whole batch is a line of units (BLOCK tokens of one
//     sequence and KV head), cut into equal shares, one per block, by every
//     block for itself from the lengths: long and short sequences balance, and
//     a captured launch follows lengths that change.  A block leaves its parts
//     of cut items in the workspace for join_kernel.
//
// Measured: 131072 tokens, 28/4 heads of 128, bf16, 48.0 us with the join, 5.6 TB/s;
// 512 sequences of 2000 tokens, 32/8 heads, e4m3, 328 us.
template <int D, bool E4M3, int NT, DecodeMode MODE>
__device__ __forceinline__ void decode_body(const DecodeParams &p) {
    using S = DecodeShape<D, E4M3, NT>;
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int g = lane / 4, c = lane % 4;
    const CacheView &cv = p.cache;
    const int per_seq = cv.Hkv * p.n_hg;  // items (KV head, head group) of a sequence
    launch_dependents();
    wait_for_primary();

    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) +
                          warp * (kDecStages * kDecTileBytes);
    const uint32_t side = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + S::RING +
                          warp * (S::PAGES + S::EXPS) + lane * 4;

    // ---- the softmax over some of an item's tokens: the tiles t0 + i * STEP, i < n,
    // of every warp; leaves the warps' states in shared memory (a warp with an item
    // of its own stores the result).  Off the line, len is the length as it is in
    // memory, and n what the tiles are rounded up by.
    constexpr bool LINE = MODE == DecodeMode::kLine, CLUSTER = MODE == DecodeMode::kCluster;
    const int STEP = LINE ? S::BLOCK : CLUSTER ? p.cluster * S::BLOCK : S::TT;
    float *sm_o = reinterpret_cast<float *>(smem);          // [warps][HEADS][OPAD]
    float *sm_st = sm_o + kDecWarps * S::HEADS * S::OPAD;   // [3][warps][HEADS]: m, lm, l
    auto segment = [&](int b, int len, int kvh, int head0, int n_heads, int t0, int n) {
        const uint32_t head_rows = static_cast<uint32_t>(kvh) * cv.page.d;

        // ---- the ring
        // Lane i takes care of the tokens i, i + 32 of a tile (i % 16 where a tile
        // has 16): their table entries come by cp.async too, K tiles before the
        // rows that they lead to are asked for, as a load that a register waits for
        // would hold up the warp (24 ragged sequences, e4m3: 95 instead of 106 us,
        // before other steps).
        constexpr int RW = S::RW, K = kDecStages - 1;
        const int32_t *table = cv.table + b * cv.max_pages;
        auto token = [&](int i, int k) {
            return static_cast<int64_t>(t0) + static_cast<int64_t>(i) * STEP +
                   (S::TT == 16 ? lane % 16 : lane + 32 * k);
        };
        auto held_token = [&](int i, int64_t t) { return i < n && t < len; };
        auto row_of = [&](int i, int k, int page) {  // pool row of this lane's k-th token of tile i
            const int64_t t = token(i, k);
            if (!held_token(i, t)) return kNoRow;
            if (static_cast<uint32_t>(page) >= cv.n_pages) {
                atomicOr(cv.status, kStatusBadBatch);
                return kNoRow;
            }
            uint32_t off;
            cv.page.quot(static_cast<uint32_t>(t), off);
            return static_cast<uint32_t>(page) * cv.Hkv * cv.page.d + head_rows + off;
        };
        auto issue = [&](int stage, const uint32_t (&r)[RW]) {
            if (E4M3) {
                // the aligned word with the row's exponent; its end may lie behind the pool's
#pragma unroll
                for (int k = 0; k < RW; ++k) {
                    const uint32_t at = r[k] & ~3u, to = side + S::PAGES + (stage * RW + k) * 256;
                    const uint32_t bytes = r[k] == kNoRow ? 0 : min(4u, cv.n_rows - at);
                    cp_async4(to, cv.k_exp + (bytes ? at : 0), bytes);
                    cp_async4(to + 128, cv.v_exp + (bytes ? at : 0), bytes);
                }
            }
            const uint32_t dst = ring + stage * kDecTileBytes;
            const int piece = lane % S::LPR;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const int at = x * S::RPI + lane / S::LPR;  // row of the tile
                const uint32_t row = __shfl_sync(0xffffffffu, r[x * S::RPI / 32], at % 32);
                const int64_t from = row == kNoRow ? 0 : static_cast<int64_t>(row) * S::ROW + piece * 16;
                const uint32_t bytes = row == kNoRow ? 0 : 16;
                cp_async16(dst + at * S::ROW + (piece ^ S::k_swizzle(at)) * 16,
                           static_cast<const char *>(cv.k) + from, bytes);
                cp_async16(dst + kDecTileBytes / 2 + at * S::ROW + (piece ^ S::v_swizzle(at)) * 16,
                           static_cast<const char *>(cv.v) + from, bytes);
            }
        };
        uint32_t rows[kDecStages][RW];  // of the tiles i, i + 1, ... in flight
        {
            // of the tiles 0 ... 2 K; off the line, where the length is still on its
            // way, asked for as if the table were full
            int page[2 * K + 1][RW];
#pragma unroll
            for (int i = 0; i <= 2 * K; ++i)
#pragma unroll
                for (int k = 0; k < RW; ++k) {
                    const int64_t t = token(i, k);
                    page[i][k] = (!LINE ? t < cv.cap : held_token(i, t))
                                     ? table[cv.page.quot(static_cast<uint32_t>(t))]
                                     : 0;
                }
            if (!LINE) {
                len = fit_len(cv, len);
                n = CLUSTER ? ((len + S::BLOCK - 1) / S::BLOCK + n) / p.cluster : (len + n) / S::TT;
            }
#pragma unroll
            for (int i = 0; i < K; ++i) {
#pragma unroll
                for (int k = 0; k < RW; ++k) rows[i][k] = row_of(i, k, page[i][k]);
                issue(i, rows[i]);
                cp_async_commit();
            }
#pragma unroll
            for (int i = K; i <= 2 * K; ++i)
#pragma unroll
                for (int k = 0; k < RW; ++k) sts4(side + ((i % kDecPageSlots) * RW + k) * 128, page[i][k]);
        }

        // ---- q: the MMA's B operand, and its scale
        uint32_t qf[NT][S::KS][2];
        float q_scale[NT][2];  // of the heads 2c and 2c+1 of this lane's accumulators (e4m3: its root)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int h = t * 8 + g;
            uint32_t w[S::KS][2];
            const __nv_bfloat16 *src = p.q + (static_cast<int64_t>(b) * p.Hq + head0 + h) * D;
#pragma unroll
            for (int j = 0; j < S::KS / 2; ++j) {
                // 16 bytes of q: eight elements, from 8 (c + 4 j) on (bf16), or
                // half of the sixteen from 16 (c + 4 (j / 2)) on (e4m3)
                const int e0 = E4M3 ? 16 * (c + 4 * (j / 2)) + 8 * (j % 2) : 8 * (c + 4 * j);
                const uint4 x = h < n_heads ? *reinterpret_cast<const uint4 *>(src + e0)
                                            : make_uint4(0, 0, 0, 0);
                w[2 * j][0] = x.x, w[2 * j][1] = x.y, w[2 * j + 1][0] = x.z, w[2 * j + 1][1] = x.w;
            }
            if (!E4M3) {
#pragma unroll
                for (int i = 0; i < S::KS; ++i) qf[t][i][0] = w[i][0], qf[t][i][1] = w[i][1];
                q_scale[t][0] = q_scale[t][1] = p.scale_log2;
            } else {
                // q as fp16 times 2^-x, x even and from the row's largest magnitude:
                // what fp16 cannot hold of it is below 2^-24 of that.  The score takes
                // 2^(x/2) before and behind the key's scale: exponents may lie at
                // opposite ends of the range and their sum in the middle.
                float m = 0.f;
#pragma unroll
                for (int i = 0; i < S::KS; ++i)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        m = fmaxf(m, fmaxf(fabsf(bf_lo(w[i][k])), fabsf(bf_hi(w[i][k]))));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const int x = min(max(static_cast<int>(__float_as_uint(m) >> 23) - 127, -126), 127) & ~1;
                const float f = pow2f(-x / 2);
#pragma unroll
                for (int i = 0; i < S::KS; ++i)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        qf[t][i][k] = pack_half2(bf_lo(w[i][k]) * f * f, bf_hi(w[i][k]) * f * f);
                const int xa = __shfl_sync(0xffffffffu, x, 8 * c), xb = __shfl_sync(0xffffffffu, x, 8 * c + 4);
                q_scale[t][0] = sqrtf(p.scale_log2) * pow2f(xa / 2);
                q_scale[t][1] = sqrtf(p.scale_log2) * pow2f(xb / 2);
            }
        }

        float acc[NT][S::MT][4], acc_low[S::MT][4];
        float m_ref[NT][2], l_ref[NT][2], l_sum[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int i = 0; i < S::MT; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[t][i][k] = acc_low[i][k] = 0.f;
#pragma unroll
            for (int k = 0; k < 2; ++k) m_ref[t][k] = l_ref[t][k] = kDecNone, l_sum[t][k] = 0.f;
        }

        int stage = 0, slot = K % kDecPageSlots;  // slot: of tile i + K's table entries
        for (int i = 0; i < n; ++i) {
            // group i + K: the rows of tile i + K, the table entries of tile i + 2 K + 1
#pragma unroll
            for (int k = 0; k < RW; ++k)
                rows[K][k] = row_of(i + K, k, static_cast<int>(lds4(side + (slot * RW + k) * 128)));
            __syncwarp();  // every lane has read what the new copies replace
            if (i + K < n) issue(stage == 0 ? K : stage - 1, rows[K]);
            {
                const int to = slot == 0 ? kDecPageSlots - 1 : slot - 1;  // (i + 2 K + 1) % slots
#pragma unroll
                for (int k = 0; k < RW; ++k) {
                    const int64_t t = token(i + 2 * K + 1, k);
                    if (held_token(i + 2 * K + 1, t))
                        cp_async4(side + (to * RW + k) * 128, table + cv.page.quot(static_cast<uint32_t>(t)), 4);
                }
            }
            cp_async_commit();
            slot = slot == kDecPageSlots - 1 ? 0 : slot + 1;
            cp_async_wait<K>();
            __syncwarp();

            // ---- scores of TT tokens, s[...][x]: token g (x < 2) or g + 8, head 2c + x % 2
            const uint32_t src = ring + stage * kDecTileBytes;
            const uint32_t ksrc = src + g * S::ROW, vsrc0 = src + kDecTileBytes / 2 + 2 * c * S::ROW;
            float s[S::SUB][NT][4];
            float v_exp[S::SUB][2];
            auto exp_of = [&](int which, int k) {  // 0: of K, 128: of V; this lane's k-th token
                const uint32_t w = lds4(side + S::PAGES + (stage * RW + k) * 256 + which);
                return static_cast<int>(static_cast<int8_t>(w >> (8 * (rows[0][k] & 3))));
            };
            uint32_t held[RW];
#pragma unroll
            for (int k = 0; k < RW; ++k) held[k] = __ballot_sync(0xffffffffu, rows[0][k] != kNoRow);
            bool grow = false;
#pragma unroll
            for (int sb = 0; sb < S::SUB; ++sb) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[sb][t][k] = 0.f;
#pragma unroll
                for (int j = 0; j < S::KJ; ++j) {
                    const int piece = ((c + 4 * j) ^ S::k_swizzle(g)) * 16;
                    const uint4 a = lds16(ksrc + sb * 16 * S::ROW + piece);
                    const uint4 e = lds16(ksrc + (sb * 16 + 8) * S::ROW + piece);
                    if (!E4M3) {
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            mma16816<false>(s[sb][t], a.x, e.x, a.y, e.y, qf[t][2 * j][0], qf[t][2 * j][1]);
                            mma16816<false>(s[sb][t], a.z, e.z, a.w, e.w, qf[t][2 * j + 1][0],
                                            qf[t][2 * j + 1][1]);
                        }
                    } else {
                        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, ew[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const uint32_t a0 = f16x2_of_e4m3x2(static_cast<uint16_t>(aw[w]));
                            const uint32_t a2 = f16x2_of_e4m3x2(static_cast<uint16_t>(aw[w] >> 16));
                            const uint32_t a1 = f16x2_of_e4m3x2(static_cast<uint16_t>(ew[w]));
                            const uint32_t a3 = f16x2_of_e4m3x2(static_cast<uint16_t>(ew[w] >> 16));
#pragma unroll
                            for (int t = 0; t < NT; ++t)
                                mma16816<true>(s[sb][t], a0, a1, a2, a3, qf[t][(4 * j + w) % S::KS][0],
                                               qf[t][(4 * j + w) % S::KS][1]);
                        }
                    }
                }
                const int from = S::TT == 16 ? 0 : (sb % 2) * 16;
                constexpr bool two = S::TT == 64;
                float kf[2] = {1.f, 1.f};
                v_exp[sb][0] = v_exp[sb][1] = 0.f;
                if (E4M3) {
                    const int ke = exp_of(0, two ? sb / 2 : 0), ve = exp_of(128, two ? sb / 2 : 0);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        kf[y] = pow2f(max(__shfl_sync(0xffffffffu, ke, from + g + 8 * y), -126));
                        v_exp[sb][y] = static_cast<float>(__shfl_sync(0xffffffffu, ve, from + g + 8 * y));
                    }
                }
                const uint32_t bits = held[two ? sb / 2 : 0] >> from;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float x = s[sb][t][k];
                        x *= q_scale[t][k % 2];
                        if (E4M3) x = x * kf[k / 2] * q_scale[t][k % 2];
                        if (!((bits >> (g + 8 * (k / 2))) & 1)) x = -INFINITY;
                        s[sb][t][k] = x;
                        grow |= x > l_ref[t][k % 2] + kDecLag;
                        if (E4M3) grow |= x + v_exp[sb][k / 2] > m_ref[t][k % 2] + (kDecLift + kDecLag);
                    }
            }
            // ---- a new reference, where a score passed the old one by 2^8
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float lm = l_ref[t][k], m = m_ref[t][k];
#pragma unroll
                        for (int sb = 0; sb < S::SUB; ++sb)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                lm = fmaxf(lm, s[sb][t][2 * y + k]);
                                if (E4M3) m = fmaxf(m, s[sb][t][2 * y + k] + v_exp[sb][y] - kDecLift);
                            }
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) {
                            lm = fmaxf(lm, __shfl_xor_sync(0xffffffffu, lm, o));
                            if (E4M3) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                        }
                        if (!E4M3) m = lm;
                        const float f = exp2_approx(m_ref[t][k] - m);
                        l_sum[t][k] *= exp2_approx(l_ref[t][k] - lm);
                        m_ref[t][k] = m;
                        l_ref[t][k] = lm;
#pragma unroll
                        for (int d = 0; d < S::MT; ++d) {
                            acc[t][d][k] *= f, acc[t][d][2 + k] *= f;
                            if (S::APART) acc_low[d][k] *= f, acc_low[d][2 + k] *= f;
                        }
                    }
            }
            // ---- O^T += V^T P^T
#pragma unroll
            for (int sb = 0; sb < S::SUB; ++sb) {
                uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float w[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float x = s[sb][t][2 * y + k];
                            const float pr = exp2_approx(x - l_ref[t][k]);
                            l_sum[t][k] += pr;
                            w[k] = E4M3 ? exp2_approx(x + v_exp[sb][y] - m_ref[t][k]) : pr;
                        }
                        if (E4M3) {
                            const __half2 h = __floats2half2_rn(w[0], w[1]);
                            const float2 hf = __half22float2(h);
                            hi[t][y] = movmatrix_trans(half2_bits(h));
                            lo[t][y] = movmatrix_trans(pack_half2((w[0] - hf.x) * kDecLow, (w[1] - hf.y) * kDecLow));
                        } else {
                            const uint32_t h = bf_pack(w[0], w[1]);
                            hi[t][y] = movmatrix_trans(h);
                            lo[t][y] = movmatrix_trans(bf_pack(w[0] - bf_lo(h), w[1] - bf_hi(h)));
                        }
                    }
                const uint32_t vsrc = vsrc0 + sb * 16 * S::ROW;  // rows 2c, 2c + 1, 2c + 8, 2c + 9 of it
                if (!E4M3) {
#pragma unroll
                    for (int j = 0; j < S::VB / 16; ++j) {
                        uint4 v[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) v[y] = lds16(vsrc + ((y & 1) + 8 * (y >> 1)) * S::ROW + ((g + 8 * j) ^ S::v_swizzle(2 * c)) * 16);
                        const uint32_t r0[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
                        const uint32_t r1[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
                        const uint32_t r2[4] = {v[2].x, v[2].y, v[2].z, v[2].w};
                        const uint32_t r3[4] = {v[3].x, v[3].y, v[3].z, v[3].w};
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const uint32_t a0 = __byte_perm(r0[w], r1[w], 0x5410);
                            const uint32_t a1 = __byte_perm(r0[w], r1[w], 0x7632);
                            const uint32_t a2 = __byte_perm(r2[w], r3[w], 0x5410);
                            const uint32_t a3 = __byte_perm(r2[w], r3[w], 0x7632);
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                mma16816<false>(acc[t][j * 4 + w], a0, a1, a2, a3, hi[t][0], hi[t][1]);
                                mma16816<false>(acc[t][j * 4 + w], a0, a1, a2, a3, lo[t][0], lo[t][1]);
                            }
                        }
                    }
                } else {
                    constexpr int W = S::VB / 4;  // words of four d's
                    auto low = [](uint32_t a) { return S::APART ? a : scale_half2(a, 1.f / kDecLow); };
                    uint32_t v[4][W];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint32_t at = vsrc + ((y & 1) + 8 * (y >> 1)) * S::ROW;
                        if (S::VB == 8) {
                            const uint2 x = lds8(at + ((g / 2) ^ S::v_swizzle(2 * c)) * 16 + g % 2 * 8);
                            v[y][0] = x.x, v[y][1] = x.y;
                        } else {
                            const uint4 x = lds16(at + (g ^ S::v_swizzle(2 * c)) * 16);
                            v[y][0] = x.x, v[y][1] = x.y, v[y][W - 2] = x.z, v[y][W - 1] = x.w;
                        }
                    }
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const uint32_t x0 = __byte_perm(v[0][w], v[1][w], 0x5140);  // d0, d1
                        const uint32_t x1 = __byte_perm(v[0][w], v[1][w], 0x7362);  // d2, d3
                        const uint32_t y0 = __byte_perm(v[2][w], v[3][w], 0x5140);
                        const uint32_t y1 = __byte_perm(v[2][w], v[3][w], 0x7362);
                        const uint32_t a00 = f16x2_of_e4m3x2(static_cast<uint16_t>(x0));
                        const uint32_t a01 = f16x2_of_e4m3x2(static_cast<uint16_t>(x0 >> 16));
                        const uint32_t a02 = f16x2_of_e4m3x2(static_cast<uint16_t>(y0));
                        const uint32_t a03 = f16x2_of_e4m3x2(static_cast<uint16_t>(y0 >> 16));
                        const uint32_t a10 = f16x2_of_e4m3x2(static_cast<uint16_t>(x1));
                        const uint32_t a11 = f16x2_of_e4m3x2(static_cast<uint16_t>(x1 >> 16));
                        const uint32_t a12 = f16x2_of_e4m3x2(static_cast<uint16_t>(y1));
                        const uint32_t a13 = f16x2_of_e4m3x2(static_cast<uint16_t>(y1 >> 16));
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            mma16816<true>(acc[t][2 * w], a00, a01, a02, a03, hi[t][0], hi[t][1]);
                            mma16816<true>(acc[t][2 * w + 1], a10, a11, a12, a13, hi[t][0], hi[t][1]);
                        }
                        const uint32_t b00 = low(a00), b01 = low(a01), b02 = low(a02), b03 = low(a03);
                        const uint32_t b10 = low(a10), b11 = low(a11), b12 = low(a12), b13 = low(a13);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            float(&to)[S::MT][4] = S::APART ? acc_low : acc[t];
                            mma16816<true>(to[2 * w], b00, b01, b02, b03, lo[t][0], lo[t][1]);
                            mma16816<true>(to[2 * w + 1], b10, b11, b12, b13, lo[t][0], lo[t][1]);
                        }
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kDecStages - 1; ++k)
#pragma unroll
                for (int r = 0; r < RW; ++r) rows[k][r] = rows[k + 1][r];
            stage = stage == kDecStages - 1 ? 0 : stage + 1;
        }
        cp_async_wait<0>();
        if (S::APART)
#pragma unroll
            for (int i = 0; i < S::MT; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[0][i][k] = fmaf(acc_low[i][k], 1.f / kDecLow, acc[0][i][k]);

        if (MODE == DecodeMode::kWarp) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int h = t * 8 + 2 * c + k;
                    float l = l_sum[t][k];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                    if (h >= n_heads) continue;
                    const OutputScale f(m_ref[t][k], l_ref[t][k], l);
                    __nv_bfloat16 *to = p.o + (static_cast<int64_t>(b) * p.Hq + head0 + h) * D;
#pragma unroll
                    for (int i = 0; i < S::MT; ++i)
                        *reinterpret_cast<uint32_t *>(to + S::column(i, g)) =
                            bf_pack(f(acc[t][i][k]), f(acc[t][i][2 + k]));
                    if (g == 0) store_lse(p, b, head0 + h, l_ref[t][k], l);
                }
            return;
        }
        // ---- join the warps of the block
        __syncthreads();
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int h = t * 8 + 2 * c + k;
                float l = l_sum[t][k];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                if (g == 0) {
                    sm_st[warp * S::HEADS + h] = m_ref[t][k];
                    sm_st[(kDecWarps + warp) * S::HEADS + h] = l_ref[t][k];
                    sm_st[(2 * kDecWarps + warp) * S::HEADS + h] = l;
                }
#pragma unroll
                for (int i = 0; i < S::MT; ++i) {
                    *reinterpret_cast<float2 *>(sm_o + (warp * S::HEADS + h) * S::OPAD + S::column(i, g)) =
                        make_float2(acc[t][i][k], acc[t][i][2 + k]);
                }
            }
        __syncthreads();
    };
    // the block's state of one head and 4 floats of d
    auto block_state = [&](int h, int d, float &m, float &lm, float &l, float4 &o) {
        m = lm = kDecNone;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
            m = fmaxf(m, sm_st[w * S::HEADS + h]);
            lm = fmaxf(lm, sm_st[(kDecWarps + w) * S::HEADS + h]);
        }
        l = 0.f;
        o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
            l = fmaf(sm_st[(2 * kDecWarps + w) * S::HEADS + h],
                     exp2_approx(sm_st[(kDecWarps + w) * S::HEADS + h] - lm), l);
            add_part(o, *reinterpret_cast<const float4 *>(sm_o + (w * S::HEADS + h) * S::OPAD + d),
                     exp2_approx(sm_st[w * S::HEADS + h] - m));
        }
    };
    if constexpr (MODE == DecodeMode::kWarp) {
        const int64_t item = static_cast<int64_t>(blockIdx.x) * kDecWarps + warp;
        if (item >= static_cast<int64_t>(cv.n_seqs) * per_seq) return;
        const int b = static_cast<int>(item / per_seq), in_seq = static_cast<int>(item - static_cast<int64_t>(b) * per_seq);
        const int kvh = in_seq / p.n_hg, hg = in_seq - kvh * p.n_hg;
        segment(b, cv.lens[b], kvh, kvh * p.G + hg * S::HEADS, min(S::HEADS, p.G - hg * S::HEADS), 0, S::TT - 1);
    } else if constexpr (LINE) {
        // units of the line that an item takes
        auto item_cost = [](int len) { return len > 0 ? (len + S::BLOCK - 1) / S::BLOCK + kDecItemCost : 0; };
        __shared__ int s_prefix[kDecThreads + 1];
        __shared__ int s_warp[kDecWarps];
        // ---- the line of units.  Up to 32 sequences: every warp for itself, a lane a
        // sequence, without a barrier.  More: groups of `per`, s_prefix[i] the unit
        // where group i begins.
        const bool few = cv.n_seqs <= 32;
        int per = 1, total, lane_len = 1, lane_end = 0;  // lane_end: the unit behind the lane's sequence
        bool empty = true;                               // there may be sequences without positions
        if (few) {
            if (lane < cv.n_seqs) lane_len = cache_len(cv, lane);
            empty = __any_sync(0xffffffffu, lane_len == 0);
            lane_end = lane < cv.n_seqs ? item_cost(lane_len) * per_seq : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, lane_end, o);
                if (lane >= o) lane_end += x;
            }
            total = __shfl_sync(0xffffffffu, lane_end, 31);
        } else {
            per = (cv.n_seqs + kDecThreads - 1) / kDecThreads;
            int scan = 0;
            for (int b = tid * per; b < min((tid + 1) * per, cv.n_seqs); ++b)
                scan += item_cost(cache_len(cv, b));
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, scan, o);
                if (lane >= o) scan += x;
            }
            if (lane == 31) s_warp[warp] = scan;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kDecWarps; ++w)
                if (w < warp) scan += s_warp[w];
            s_prefix[tid + 1] = scan * per_seq;
            if (tid == 0) s_prefix[0] = 0;
            __syncthreads();
            total = s_prefix[kDecThreads];
        }

        // ---- sequences without positions
        if (empty)
            for (int b = blockIdx.x; b < cv.n_seqs; b += gridDim.x) {
                if (cache_len(cv, b) > 0) continue;
                for (int i = tid; i < p.Hq * D / 8; i += kDecThreads)
                    reinterpret_cast<uint4 *>(p.o + static_cast<int64_t>(b) * p.Hq * D)[i] = make_uint4(0, 0, 0, 0);
                if (p.lse)
                    for (int h = tid; h < p.Hq; h += kDecThreads)
                        p.lse[static_cast<int64_t>(h) * cv.n_seqs + b] = -INFINITY;
                if (p.cuts_by_item)
                    for (int i = tid; i < per_seq; i += kDecThreads) p.cuts[b * per_seq + i] = make_int4(0, 0, 0, 0);
            }

        // Shares of `base` units, of one more for the first `more` blocks.
        const int ctas = min(total, static_cast<int>(gridDim.x));  // blocks with a share
        const int cta = blockIdx.x;
        if (tid == 0 && !p.cuts_by_item) p.cuts[cta] = make_int4(0, 0, 0, 0);
        if (cta >= ctas) return;
        const int base = total / ctas, more = total - base * ctas;
        int u = cta * base + min(cta, more);
        const int u_end = u + base + (cta < more ? 1 : 0);
        auto cta_of = [&](int x) {
            const int y = x - more * (base + 1);
            return y < 0 ? x / (base + 1) : more + y / base;
        };

        // ---- the sequence of the first unit
        int b, first, len;  // first: the unit where sequence b begins
        if (few) {
            b = __ffs(__ballot_sync(0xffffffffu, lane_end > u)) - 1;
            len = __shfl_sync(0xffffffffu, lane_len, b);
            first = __shfl_sync(0xffffffffu, lane_end, b) - item_cost(len) * per_seq;
        } else {
            int lo = 0, hi = kDecThreads;  // s_prefix[lo] <= u < s_prefix[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (s_prefix[mid] <= u) lo = mid; else hi = mid;
            }
            b = lo * per;
            first = s_prefix[lo];
            len = cache_len(cv, b);
        }

        while (u < u_end) {
            int cost = item_cost(len);
            while (u >= first + cost * per_seq) {
                first += cost * per_seq;
                len = cache_len(cv, ++b);
                cost = item_cost(len);
            }
            const int item = (u - first) / cost;
            const int item_u0 = first + item * cost, item_u1 = item_u0 + cost;
            const int blocks = cost - kDecItemCost;
            // the item's blocks of tokens that are this share's
            const int lo = max(u - item_u0 - kDecItemCost, 0);
            const int hi = min(u_end, item_u1) - item_u0 - kDecItemCost;
            u = min(u_end, item_u1);
            if (hi <= lo) continue;
            const int kvh = item / p.n_hg, hg = item - kvh * p.n_hg;
            const int head0 = kvh * p.G + hg * S::HEADS;
            const int n_heads = min(S::HEADS, p.G - hg * S::HEADS);
            segment(b, len, kvh, head0, n_heads, lo * S::BLOCK + warp * S::TT, hi - lo);
            const bool whole = lo == 0 && hi == blocks;
            const int part = 2 * cta + (lo == 0 ? 1 : 0);
            for (int x = tid; x < S::HEADS * D / 4; x += kDecThreads) {
                const int h = x / (D / 4), d = x % (D / 4) * 4;
                float m, lm, l;
                float4 o;
                block_state(h, d, m, lm, l, o);
                if (!whole) {
                    if (d == 0) {
                        float *st = p.part_stat + (h * 6 + (lo == 0 ? 1 : 0)) * kDecMaxCtas + cta;
                        st[0] = m, st[2 * kDecMaxCtas] = lm, st[4 * kDecMaxCtas] = l;
                    }
                    reinterpret_cast<float4 *>(p.part_o + (part * S::HEADS + h) * D + d)[0] = o;
                } else if (h < n_heads) {
                    store_result<D>(p, b, head0 + h, d, m, lm, l, o);
                }
            }
            if (lo == 0 && tid == 0 && (p.cuts_by_item || !whole))
                p.cuts[p.cuts_by_item ? b * per_seq + item : cta] =
                    make_int4(cta, whole ? 0 : cta_of(item_u1 - 1) - cta + 1, b, item);
            __syncthreads();  // the ring is free again
        }
    } else {
        const uint32_t item = blockIdx.x / p.cluster, rank = blockIdx.x - item * p.cluster;
        const int b = item / per_seq, in_seq = item - b * per_seq;
        const int kvh = in_seq / p.n_hg, hg = in_seq - kvh * p.n_hg;
        const int head0 = kvh * p.G + hg * S::HEADS;
        const int n_heads = min(S::HEADS, p.G - hg * S::HEADS);
        segment(b, cv.lens[b], kvh, head0, n_heads, rank * S::BLOCK + warp * S::TT,
                p.cluster - 1 - static_cast<int>(rank));
        // the block's state, for the others to read
        float *cl_o = sm_st + 3 * kDecWarps * S::HEADS;  // [HEADS][D]
        float *cl_st = cl_o + S::HEADS * D;              // [3][HEADS]
        for (int x = tid; x < S::HEADS * D / 4; x += kDecThreads) {
            const int h = x / (D / 4), d = x % (D / 4) * 4;
            float m, lm, l;
            float4 o;
            block_state(h, d, m, lm, l, o);
            reinterpret_cast<float4 *>(cl_o)[x] = o;
            if (d == 0) cl_st[h] = m, cl_st[S::HEADS + h] = lm, cl_st[2 * S::HEADS + h] = l;
        }
        cluster_sync();
        const int share = S::HEADS * D / 4 / p.cluster;  // float4s of the result that a block writes
        for (int i = tid; i < share; i += kDecThreads) {
            const int x = rank * share + i, h = x / (D / 4), d = x % (D / 4) * 4;
            if (h >= n_heads) break;
            float ms[kDecCluster], lms[kDecCluster], ls[kDecCluster];
            float4 os[kDecCluster];
#pragma unroll
            for (int r = 0; r < kDecCluster; ++r) {
                ms[r] = lms[r] = kDecNone, ls[r] = 0.f, os[r] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < p.cluster) {
                    const uint32_t st = cluster_address(cl_st + h, r);
                    ms[r] = cluster_load(st);
                    lms[r] = cluster_load(st + 4 * S::HEADS);
                    ls[r] = cluster_load(st + 8 * S::HEADS);
                    os[r] = cluster_load4(cluster_address(cl_o + 4 * x, r));
                }
            }
            float m = kDecNone, lm = kDecNone, l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int r = 0; r < kDecCluster; ++r) m = fmaxf(m, ms[r]), lm = fmaxf(lm, lms[r]);
#pragma unroll
            for (int r = 0; r < kDecCluster; ++r) {
                l = fmaf(ls[r], exp2_approx(lms[r] - lm), l);
                add_part(o, os[r], exp2_approx(ms[r] - m));
            }
            store_result<D>(p, b, head0 + h, d, m, lm, l, o);
        }
        cluster_sync();  // no block leaves while it is read
    }
}

template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kDecThreads) decode_kernel(const __grid_constant__ DecodeParams p) {
    decode_body<D, E4M3, NT, DecodeMode::kLine>(p);
}

// Short contexts: an item is one cluster's, block after block of tokens in turn,
// and the blocks' states are joined through distributed shared memory.  One
// launch, no line, no parts in memory: 2048 tokens, 4/2 heads of 64, 4.3 us, of which
// the length, the pages and the rows, one after the other, are 2.2.
template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kDecThreads)
    decode_cluster_kernel(const __grid_constant__ DecodeParams p) {
    decode_body<D, E4M3, NT, DecodeMode::kCluster>(p);
}

// More items than the SMs hold blocks, and short contexts: an item is one warp's,
// from its first tile to its result, without a barrier or a join: 500 sequences of 64
// tokens, 32/8 heads of 128, e4m3, 22.4 us, 56 along the line.
template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kDecThreads) decode_warp_kernel(const __grid_constant__ DecodeParams p) {
    decode_body<D, E4M3, NT, DecodeMode::kWarp>(p);
}

// The parts of the cut items, weighted by 2^(m_i - max m) and summed in the order
// of the line, so that the same call gives the same bytes.  Part 0 is the second
// one of the item's first block, the others the first ones of the blocks behind.
// It is bound by latency -- a dependent launch and two reads of L2, the second of
// all that the block needs at once: rows and statistics, which each warp works out
// for itself.
// SPLIT: a block is 32 elements of one query head of an item, and its threads
// split the parts: few items, many parts each (128K tokens on 4 KV heads are 74
// parts an item, joined 3 us after the last of them; 256K tokens on one, 296).
// Otherwise a row of O is a warp's (or half a warp's), of many items with a few
// parts each.
template <int D, int NT, bool SPLIT>
__global__ void __launch_bounds__(SPLIT ? kJoinThreads : kDecThreads) join_kernel(const __grid_constant__ DecodeParams p) {
    constexpr int HEADS = 8 * NT, PIECES = SPLIT ? D / 32 : 1;
    constexpr int COLS = D / 4 / PIECES;                         // float4s of a row that a block takes
    constexpr int GROUPS = (SPLIT ? kJoinThreads : kDecThreads) / COLS;
    constexpr int PER = SPLIT ? GROUPS : 1;                      // threads that share a column's parts
    constexpr int AHEAD = SPLIT ? kDecMaxCtas / GROUPS : 8;      // parts of a thread under way
    constexpr int MATES = SPLIT ? 32 : COLS;                     // lanes that work out an item's statistics
    constexpr int OWN = SPLIT ? (kDecMaxCtas + kJoinThreads - 1) / kJoinThreads : 1;
    __shared__ float4 s_o[SPLIT ? kJoinThreads : 1];
    __shared__ float s_st[3][SPLIT ? kDecMaxCtas : 1];           // SPLIT: m, lm, l of the parts
    const int tid = threadIdx.x, col = tid % COLS, group = tid / COLS;
    const int l4 = col + (SPLIT ? blockIdx.x % PIECES * COLS : 0);
    launch_dependents();
    wait_for_primary();
    const int blocks = SPLIT ? PIECES * HEADS : HEADS / GROUPS;  // of an item
    const int4 cut = __ldcg(p.cuts + blockIdx.x / blocks);
    const int c0 = cut.x, parts = cut.y;
    if (parts == 0) return;
    const int kvh = cut.w / p.n_hg, hg = cut.w - kvh * p.n_hg;
    const int head0 = kvh * p.G + hg * HEADS, n_heads = min(HEADS, p.G - hg * HEADS);
    const int first = SPLIT ? group : 0;
    auto slot_of = [&](int i) { return 2 * (c0 + i) + (i == 0 ? 1 : 0); };

    const int h = SPLIT ? blockIdx.x / PIECES % HEADS : blockIdx.x % blocks * GROUPS + group;
    if (h >= n_heads) return;
    // the parts' statistics lie side by side, but part 0's
    const float *stat = p.part_stat + h * 6 * kDecMaxCtas + c0;
    auto stat_at = [&](int i, int which) {
        return __ldcg(stat + (2 * which + (i == 0 ? 1 : 0)) * kDecMaxCtas + i);
    };
    float own[OWN][3];
    if (SPLIT) {
#pragma unroll
        for (int k = 0; k < OWN; ++k)
#pragma unroll
            for (int which = 0; which < 3; ++which)
                own[k][which] = tid + k * kJoinThreads < parts ? stat_at(tid + k * kJoinThreads, which) : 0.f;
    }
    float4 y[AHEAD];
    float w[AHEAD];
    auto load = [&](int at) {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int i = at + k * PER;
            y[k] = make_float4(0.f, 0.f, 0.f, 0.f), w[k] = kDecNone;
            if (i < parts) {
                y[k] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + (slot_of(i) * HEADS + h) * D) + l4);
                if (!SPLIT) w[k] = stat_at(i, 0);
            }
        }
    };
    load(first);
    if (SPLIT) {
#pragma unroll
        for (int k = 0; k < OWN; ++k)
            if (tid + k * kJoinThreads < parts)
#pragma unroll
                for (int which = 0; which < 3; ++which) s_st[which][tid + k * kJoinThreads] = own[k][which];
        __syncthreads();
    }
    // the item's statistics: a lane's parts in turn, then the lanes'
    float m = kDecNone, lm = kDecNone, l = 0.f;
    auto add = [&](float lmi, float li) {
        const float top = fmaxf(lm, lmi);
        l = l * exp2_approx(lm - top) + li * exp2_approx(lmi - top);
        lm = top;
    };
#pragma unroll 2
    for (int i = tid % MATES; i < parts; i += MATES) {
        m = fmaxf(m, SPLIT ? s_st[0][i] : stat_at(i, 0));
        add(SPLIT ? s_st[1][i] : stat_at(i, 1), SPLIT ? s_st[2][i] : stat_at(i, 2));
    }
    const unsigned mates = MATES == 32 ? 0xffffffffu : ((1u << MATES) - 1) << (tid % 32 / MATES * MATES);
#pragma unroll
    for (int o = 1; o < MATES; o <<= 1) {
        const float lmi = __shfl_xor_sync(mates, lm, o), li = __shfl_xor_sync(mates, l, o);
        add(lmi, li);
        m = fmaxf(m, __shfl_xor_sync(mates, m, o));
    }
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int at = first; at < parts; at += AHEAD * PER) {
        if (at != first) load(at);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (SPLIT && at + k * PER < parts) w[k] = s_st[0][at + k * PER];
            add_part(o, y[k], exp2_approx(w[k] - m));
        }
    }
    if (SPLIT) {
        s_o[tid] = o;
        __syncthreads();
        if (group != 0) return;
#pragma unroll 8
        for (int k = 1; k < PER; ++k) add_part(o, s_o[k * COLS + tid], 1.f);
    }
    store_result<D>(p, cut.z, head0 + h, l4 * 4, m, lm, l, o);
}

}  // namespace spava
