// decode_kernel.cuh -- attention of one new token per sequence over the paged
// cache, split over the cache's length and joined in the same launch.
#pragma once

#include "cache_common.cuh"

namespace spava {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kDecMaxCtas = 320;  // the workspace's partials are sized for these
constexpr int kDecStages = 3;
constexpr int kDecTileBytes = 8192;  // K and V bytes of one warp's tile
constexpr int kDecRingBytes = kDecWarps * kDecStages * kDecTileBytes;

struct DecodeParams {
    CacheView cache;
    const __nv_bfloat16 *q;
    __nv_bfloat16 *o;
    float *lse;
    int32_t Hq, G;        // query heads, per KV head
    int32_t n_hg;         // groups of 8 * NT query heads that share a KV head
    float scale_log2;     // softmax scale * log2 e
    int *counters;        // [kDecMaxCtas], zero between calls
    float *part_stat;     // [2 * kDecMaxCtas][3][8 * NT]
    float *part_o;        // [2 * kDecMaxCtas][8 * NT][D]
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes)
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
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// The state of a softmax over part of a context, in base 2: l = sum 2^(s - lm),
// O = sum 2^(s + e - m) v with e the value's exponent (m = lm where there is
// none).  kDecNone marks a part without a finite score.
constexpr float kDecNone = -3.402823466e38f;

template <int D, bool E4M3, int NT>
struct DecodeShape {
    static constexpr int ROW = D * (E4M3 ? 1 : 2);         // bytes of a cached row
    static constexpr int TT = kDecTileBytes / (2 * ROW);   // tokens of a warp's tile
    static constexpr int SUB = TT / 16;                    // MMA tiles of 16 tokens
    static constexpr int BLOCK = TT * kDecWarps;           // tokens of a work unit
    static constexpr int KJ = ROW / 64;                    // 16-byte pieces of a K row per lane
    static constexpr int VB = ROW / 8;                     // bytes of a V row per lane
    static constexpr int KS = D / 16;                      // k steps of a score
    static constexpr int MT = D / 16;                      // 16-row tiles of O^T
    static constexpr int HEADS = 8 * NT;
    static constexpr int OPAD = D + 4;                     // floats of an O row in shared memory
    // The ring is free when a segment is joined, and takes the warps' O and
    // statistics, then the join's weights.
    static constexpr int MERGE = kDecWarps * HEADS * (OPAD + 3) * 4 + HEADS * 2 * 4;
    static constexpr int JOIN = HEADS * (kDecMaxCtas + 3) * 4;
    static constexpr int A = MERGE > kDecRingBytes ? MERGE : kDecRingBytes;
    static constexpr int SMEM = A > JOIN ? A : JOIN;
};

// What bounds it: every cached row is read once, D bytes or 2 D, and takes
// 4 G D operations, G the query heads of a KV head -- far below what the tensor
// cores do per byte of HBM, so the kernel is a read of the cache with
// arithmetic beside it, and all choices keep that read running:
//
//   - Every lane copies with cp.async just the bytes that it will itself feed
//     to the matrix instructions, into a ring of its own, and only ever waits
//     for its own copies: no barrier in the loop, no address constraint but 16
//     bytes, so pages may have any size and end inside a tile.  The
//     contraction order over d is free, so a lane takes 16 contiguous bytes of
//     a K row for two to four k steps; O's rows are permuted likewise for V.
//   - Transposed products, S^T = K Q^T and O^T = V^T P^T: tokens (or d) take
//     the 16-row side of an MMA and the query heads the 8-column side, so G = 7
//     or 4 wastes little, and the accumulators are 4 NT D / 16 registers.
//   - Softmax against a reference that may lag the maximum by 2^8: then a tile
//     needs one vote and no shuffles, and O is rescaled only when a score
//     passes that.  Sums and O stay in fp32.
//   - bf16: P enters as hi + lo, two bf16 products, 16 significant bits: one
//     bf16 rounding of P would cost as much as the rounding of the output.
//     e4m3: K, V, P and the scaled q are fp16 (e4m3 is exact in it, P keeps 11
//     bits).  A row's scales come in as exponents: of K into the score, of V
//     into P, whose reference m then covers score + exponent, while the sum l
//     has its own, lm.
//   - The work of the whole batch is a line of units (BLOCK tokens of one
//     sequence and KV head), cut into equal shares, one per block, by every
//     block for itself from the lengths: long and short sequences balance, and
//     a captured launch follows lengths that change.  A block leaves the parts
//     of a cut sequence in the workspace, and the last of its blocks to arrive
//     joins them, in the order of the line: the result does not depend on who
//     is last.
template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kDecThreads) decode_kernel(const __grid_constant__ DecodeParams p) {
    using S = DecodeShape<D, E4M3, NT>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t s_prefix[kDecThreads + 1];
    __shared__ int64_t s_warp[kDecWarps];
    __shared__ int s_last;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int g = lane / 4, c = lane % 4;
    const CacheView &cv = p.cache;
    const int per_seq = cv.Hkv * p.n_hg;  // items (KV head, head group) of a sequence

    // ---- the line of units: thread t holds the sequences [t * per, (t+1) * per)
    const int per = (cv.n_seqs + kDecThreads - 1) / kDecThreads;
    int64_t mine = 0;
    for (int b = tid * per; b < min((tid + 1) * per, cv.n_seqs); ++b)
        mine += (cache_len(cv, b) + S::BLOCK - 1) / S::BLOCK;
    int64_t scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, scan, o);
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
    const int64_t total = s_prefix[kDecThreads];

    // ---- sequences without positions
    for (int b = blockIdx.x; b < cv.n_seqs; b += gridDim.x) {
        if (cache_len(cv, b) > 0) continue;
        for (int i = tid; i < p.Hq * D / 8; i += kDecThreads)
            reinterpret_cast<uint4 *>(p.o + static_cast<int64_t>(b) * p.Hq * D)[i] = make_uint4(0, 0, 0, 0);
        if (p.lse)
            for (int h = tid; h < p.Hq; h += kDecThreads)
                p.lse[static_cast<int64_t>(h) * cv.n_seqs + b] = -INFINITY;
    }

    const int64_t ctas = total < gridDim.x ? total : gridDim.x;  // blocks with a share
    if (blockIdx.x >= ctas) return;
    int64_t u = blockIdx.x * total / ctas;
    const int64_t u_end = (blockIdx.x + 1) * total / ctas;

    // ---- the sequence of the first unit
    int b;
    int64_t first;  // unit where sequence b begins
    {
        int lo = 0, hi = kDecThreads;  // s_prefix[lo] <= u < s_prefix[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (s_prefix[mid] <= u) lo = mid; else hi = mid;
        }
        b = lo * per;
        first = s_prefix[lo];
    }
    int len = cache_len(cv, b);
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) +
                          warp * (kDecStages * kDecTileBytes);

    while (u < u_end) {
        int64_t blocks = (len + S::BLOCK - 1) / S::BLOCK;
        while (u >= first + blocks * per_seq) {
            first += blocks * per_seq;
            len = cache_len(cv, ++b);
            blocks = (len + S::BLOCK - 1) / S::BLOCK;
        }
        const int item = static_cast<int>((u - first) / blocks);
        const int64_t item_u0 = first + item * blocks, item_u1 = item_u0 + blocks;
        const int kvh = item / p.n_hg, hg = item - kvh * p.n_hg;
        const int64_t seg_end = u_end < item_u1 ? u_end : item_u1;
        const int n = static_cast<int>(seg_end - u);                      // tiles of this warp
        const int t0 = static_cast<int>(u - item_u0) * S::BLOCK + warp * S::TT;  // first token of tile 0
        const int head0 = kvh * p.G + hg * S::HEADS;
        const int n_heads = min(S::HEADS, p.G - hg * S::HEADS);
        const uint32_t head_rows = static_cast<uint32_t>(kvh) * cv.page.d;

        // ---- q: the MMA's B operand, and its scale
        uint32_t qf[NT][S::KS][2];
        float q_scale[NT][2];  // of the heads 2c and 2c+1 of this lane's accumulators
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
                const uint4 x = h < n_heads ? __ldg(reinterpret_cast<const uint4 *>(src + e0))
                                            : make_uint4(0, 0, 0, 0);
                w[2 * j][0] = x.x, w[2 * j][1] = x.y, w[2 * j + 1][0] = x.z, w[2 * j + 1][1] = x.w;
            }
            if (!E4M3) {
#pragma unroll
                for (int i = 0; i < S::KS; ++i) qf[t][i][0] = w[i][0], qf[t][i][1] = w[i][1];
                q_scale[t][0] = q_scale[t][1] = p.scale_log2;
            } else {
                // q as fp16 times 2^x, x from the row's largest magnitude: what
                // fp16 cannot hold of it is below 2^-24 of that.
                float m = 0.f;
#pragma unroll
                for (int i = 0; i < S::KS; ++i)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        m = fmaxf(m, fmaxf(fabsf(bf_lo(w[i][k])), fabsf(bf_hi(w[i][k]))));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const int x = min(max(static_cast<int>(__float_as_uint(m) >> 23) - 127, -100), 127);
                // 2^-127 is no normal number: in two steps
                const float f0 = pow2f(-(x / 2)), f1 = pow2f(-(x - x / 2));
#pragma unroll
                for (int i = 0; i < S::KS; ++i)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        qf[t][i][k] = pack_half2(bf_lo(w[i][k]) * f0 * f1, bf_hi(w[i][k]) * f0 * f1);
                const int xa = __shfl_sync(0xffffffffu, x, 8 * c), xb = __shfl_sync(0xffffffffu, x, 8 * c + 4);
                q_scale[t][0] = p.scale_log2 * pow2f(xa);
                q_scale[t][1] = p.scale_log2 * pow2f(xb);
            }
        }

        float acc[NT][S::MT][4];
        float m_ref[NT][2], l_ref[NT][2], l_sum[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int i = 0; i < S::MT; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[t][i][k] = 0.f;
#pragma unroll
            for (int k = 0; k < 2; ++k) m_ref[t][k] = l_ref[t][k] = kDecNone, l_sum[t][k] = 0.f;
        }

        // ---- the ring
        // Lane i looks up the pool rows of the tokens i, i + 32 of a tile (of
        // i % 16 where a tile has 16).
        constexpr int RW = S::TT == 64 ? 2 : 1;
        auto look_up = [&](int i, uint32_t (&r)[RW]) {
#pragma unroll
            for (int k = 0; k < RW; ++k) {
                const int64_t t = static_cast<int64_t>(t0) + static_cast<int64_t>(i) * S::BLOCK +
                                  (S::TT == 16 ? lane % 16 : lane + 32 * k);
                r[k] = kNoRow;
                if (i < n && t < len) {
                    r[k] = cache_row(cv, b, static_cast<int>(t));
                    if (r[k] != kNoRow) r[k] += head_rows;
                }
            }
        };
        auto issue = [&](int stage, const uint32_t (&r)[RW]) {
            const uint32_t dst = ring + stage * kDecTileBytes;
            const char *kp = static_cast<const char *>(cv.k), *vp = static_cast<const char *>(cv.v);
#pragma unroll
            for (int s = 0; s < S::SUB; ++s) {
                const uint32_t rs = r[S::TT == 64 ? s / 2 : 0];
                const int from = S::TT == 16 ? 0 : (s % 2) * 16;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint32_t row = __shfl_sync(0xffffffffu, rs, from + g + 8 * y);
                    const char *src = kp + (row == kNoRow ? 0 : static_cast<int64_t>(row) * S::ROW) + c * 16;
#pragma unroll
                    for (int j = 0; j < S::KJ; ++j)
                        cp_async16(dst + ((s * 2 + y) * S::KJ + j) * 512 + lane * 16, src + j * 64,
                                   row == kNoRow ? 0 : 16);
                }
                const uint32_t vdst = dst + kDecTileBytes / 2 + s * 16 * S::ROW;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const uint32_t row = __shfl_sync(0xffffffffu, rs, from + 2 * c + (y & 1) + 8 * (y >> 1));
                    const char *src = vp + (row == kNoRow ? 0 : static_cast<int64_t>(row) * S::ROW);
                    if (S::VB == 8) {
                        cp_async8(vdst + y * 256 + lane * 8, src + g * 8, row == kNoRow ? 0 : 8);
                    } else {
#pragma unroll
                        for (int j = 0; j < S::VB / 16; ++j)
                            cp_async16(vdst + (y * (S::VB / 16) + j) * 512 + lane * 16,
                                       src + g * 16 + j * 128, row == kNoRow ? 0 : 16);
                    }
                }
            }
        };
        auto load_exps = [&](const uint32_t (&r)[RW], int (&ke)[RW], int (&ve)[RW]) {
#pragma unroll
            for (int k = 0; k < RW; ++k) {
                ke[k] = ve[k] = 0;
                if (E4M3 && r[k] != kNoRow) {
                    ke[k] = __ldg(cv.k_exp + r[k]);
                    ve[k] = __ldg(cv.v_exp + r[k]);
                }
            }
        };

        uint32_t rows[kDecStages][RW];  // of the tiles i, i + 1, ... in flight
#pragma unroll
        for (int i = 0; i < kDecStages; ++i) look_up(i, rows[i]);
        int ke[RW], ve[RW];
        load_exps(rows[0], ke, ve);
#pragma unroll
        for (int i = 0; i < kDecStages - 1; ++i) {
            issue(i, rows[i]);
            cp_async_commit();
        }

        int stage = 0;
        for (int i = 0; i < n; ++i) {
            {
                const int to = stage == 0 ? kDecStages - 1 : stage - 1;
                if (i + kDecStages - 1 < n) issue(to, rows[kDecStages - 1]);
                cp_async_commit();
            }
            uint32_t ahead[RW];
            look_up(i + kDecStages, ahead);
            int ke_next[RW], ve_next[RW];
            load_exps(rows[1], ke_next, ve_next);
            cp_async_wait<kDecStages - 1>();

            // ---- scores of TT tokens, s[...][x]: token g (x < 2) or g + 8, head 2c + x % 2
            const uint32_t src = ring + stage * kDecTileBytes;
            float s[S::SUB][NT][4];
            float v_exp[S::SUB][2];
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
                    const uint4 a = lds16(src + (sb * 2 * S::KJ + j) * 512 + lane * 16);
                    const uint4 e = lds16(src + ((sb * 2 + 1) * S::KJ + j) * 512 + lane * 16);
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
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        kf[y] = pow2f(max(__shfl_sync(0xffffffffu, ke[two ? sb / 2 : 0], from + g + 8 * y), -126));
                        v_exp[sb][y] = static_cast<float>(
                            __shfl_sync(0xffffffffu, ve[two ? sb / 2 : 0], from + g + 8 * y));
                    }
                }
                const uint32_t bits = held[two ? sb / 2 : 0] >> from;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float x = s[sb][t][k];
                        if (E4M3) x *= kf[k / 2];
                        x *= q_scale[t][k % 2];
                        if (!((bits >> (g + 8 * (k / 2))) & 1)) x = -INFINITY;
                        s[sb][t][k] = x;
                        grow |= x > l_ref[t][k % 2] + 8.f;
                        if (E4M3) grow |= x + v_exp[sb][k / 2] > m_ref[t][k % 2] + 8.f;
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
                                if (E4M3) m = fmaxf(m, s[sb][t][2 * y + k] + v_exp[sb][y]);
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
                        for (int d = 0; d < S::MT; ++d) acc[t][d][k] *= f, acc[t][d][2 + k] *= f;
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
                            hi[t][y] = movmatrix_trans(pack_half2(w[0], w[1]));
                        } else {
                            const uint32_t h = bf_pack(w[0], w[1]);
                            hi[t][y] = movmatrix_trans(h);
                            lo[t][y] = movmatrix_trans(bf_pack(w[0] - bf_lo(h), w[1] - bf_hi(h)));
                        }
                    }
                const uint32_t vsrc = src + kDecTileBytes / 2 + sb * 16 * S::ROW;
                if (!E4M3) {
#pragma unroll
                    for (int j = 0; j < S::VB / 16; ++j) {
                        uint4 v[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) v[y] = lds16(vsrc + (y * (S::VB / 16) + j) * 512 + lane * 16);
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
                    uint32_t v[4][W];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        if (S::VB == 8) {
                            const uint2 x = lds8(vsrc + y * 256 + lane * 8);
                            v[y][0] = x.x, v[y][1] = x.y;
                        } else {
                            const uint4 x = lds16(vsrc + y * 512 + lane * 16);
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
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kDecStages - 1; ++k)
#pragma unroll
                for (int r = 0; r < RW; ++r) rows[k][r] = rows[k + 1][r];
#pragma unroll
            for (int r = 0; r < RW; ++r) {
                rows[kDecStages - 1][r] = ahead[r];
                ke[r] = ke_next[r];
                ve[r] = ve_next[r];
            }
            stage = stage == kDecStages - 1 ? 0 : stage + 1;
        }
        cp_async_wait<0>();

        // ---- join the warps of the block
        float *sm_o = reinterpret_cast<float *>(smem);                    // [warps][HEADS][OPAD]
        float *sm_st = sm_o + kDecWarps * S::HEADS * S::OPAD;             // [3][warps][HEADS]: m, lm, l
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
                    const int d = E4M3 ? D / 8 * g + 2 * i : 64 * (i / 4) + 8 * g + 2 * (i % 4);
                    *reinterpret_cast<float2 *>(sm_o + (warp * S::HEADS + h) * S::OPAD + d) =
                        make_float2(acc[t][i][k], acc[t][i][2 + k]);
                }
            }
        __syncthreads();
        const bool whole = u <= item_u0 && seg_end == item_u1;
        const int slot = 2 * blockIdx.x + (u == item_u0 ? 1 : 0);
        // thread: one head of 4 floats of d at a time
        for (int x = tid; x < S::HEADS * D / 4; x += kDecThreads) {
            const int h = x / (D / 4), d = x % (D / 4) * 4;
            float m = kDecNone, lm = kDecNone;
#pragma unroll
            for (int w = 0; w < kDecWarps; ++w) {
                m = fmaxf(m, sm_st[w * S::HEADS + h]);
                lm = fmaxf(lm, sm_st[(kDecWarps + w) * S::HEADS + h]);
            }
            float l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kDecWarps; ++w) {
                const float f = exp2_approx(sm_st[w * S::HEADS + h] - m);
                l = fmaf(sm_st[(2 * kDecWarps + w) * S::HEADS + h],
                         exp2_approx(sm_st[(kDecWarps + w) * S::HEADS + h] - lm), l);
                const float4 y = *reinterpret_cast<const float4 *>(sm_o + (w * S::HEADS + h) * S::OPAD + d);
                o.x = fmaf(y.x, f, o.x), o.y = fmaf(y.y, f, o.y);
                o.z = fmaf(y.z, f, o.z), o.w = fmaf(y.w, f, o.w);
            }
            if (!whole) {
                if (d == 0) {
                    float *st = p.part_stat + static_cast<int64_t>(slot) * 3 * S::HEADS + h;
                    st[0] = m, st[S::HEADS] = lm, st[2 * S::HEADS] = l;
                }
                reinterpret_cast<float4 *>(p.part_o + (static_cast<int64_t>(slot) * S::HEADS + h) * D + d)[0] = o;
            } else if (h < n_heads) {
                const float f = l == 0.f ? 0.f : exp2f(m - lm) / l;
                *reinterpret_cast<uint2 *>(p.o + (static_cast<int64_t>(b) * p.Hq + head0 + h) * D + d) =
                    make_uint2(bf_pack(o.x * f, o.y * f), bf_pack(o.z * f, o.w * f));
                if (d == 0 && p.lse)
                    p.lse[static_cast<int64_t>(head0 + h) * cv.n_seqs + b] =
                        l == 0.f ? -INFINITY : 0.6931471805599453f * (lm + log2f(l));
            }
        }

        // ---- join the blocks of a cut item: the last to arrive does it
        if (!whole) {
            // block of unit x: the largest i with i * total / ctas <= x
            const int c0 = static_cast<int>(((item_u0 + 1) * ctas - 1) / total);
            const int c1 = static_cast<int>((item_u1 * ctas - 1) / total);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                s_last = atomicAdd(p.counters + c0, 1) == c1 - c0;
                __threadfence();
            }
            __syncthreads();
            if (s_last) {
                const int parts = c1 - c0 + 1;
                float *wt = reinterpret_cast<float *>(smem);      // [HEADS][kDecMaxCtas] weights
                float *res = wt + S::HEADS * kDecMaxCtas;         // [3][HEADS]: m, lm, l
                auto slot_of = [&](int i) { return 2 * (c0 + i) + (i == 0 ? 1 : 0); };
                for (int h = warp; h < S::HEADS; h += kDecWarps) {
                    float m = kDecNone, lm = kDecNone;
                    for (int i = lane; i < parts; i += 32) {
                        const float *st = p.part_stat + static_cast<int64_t>(slot_of(i)) * 3 * S::HEADS + h;
                        m = fmaxf(m, __ldcg(st));
                        lm = fmaxf(lm, __ldcg(st + S::HEADS));
                    }
#pragma unroll
                    for (int o = 16; o; o >>= 1) {
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                        lm = fmaxf(lm, __shfl_xor_sync(0xffffffffu, lm, o));
                    }
                    float l = 0.f;
                    for (int i = lane; i < parts; i += 32) {
                        const float *st = p.part_stat + static_cast<int64_t>(slot_of(i)) * 3 * S::HEADS + h;
                        wt[h * kDecMaxCtas + i] = exp2_approx(__ldcg(st) - m);
                        l = fmaf(__ldcg(st + 2 * S::HEADS), exp2_approx(__ldcg(st + S::HEADS) - lm), l);
                    }
#pragma unroll
                    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                    if (lane == 0) res[h] = m, res[S::HEADS + h] = lm, res[2 * S::HEADS + h] = l;
                }
                __syncthreads();
                for (int x = tid; x < n_heads * D / 4; x += kDecThreads) {
                    const int h = x / (D / 4), d = x % (D / 4) * 4;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int i = 0; i < parts; ++i) {
                        const float f = wt[h * kDecMaxCtas + i];
                        const float4 y = __ldcg(reinterpret_cast<const float4 *>(
                            p.part_o + (static_cast<int64_t>(slot_of(i)) * S::HEADS + h) * D + d));
                        o.x = fmaf(y.x, f, o.x), o.y = fmaf(y.y, f, o.y);
                        o.z = fmaf(y.z, f, o.z), o.w = fmaf(y.w, f, o.w);
                    }
                    const float m = res[h], lm = res[S::HEADS + h], l = res[2 * S::HEADS + h];
                    const float f = l == 0.f ? 0.f : exp2f(m - lm) / l;
                    *reinterpret_cast<uint2 *>(p.o + (static_cast<int64_t>(b) * p.Hq + head0 + h) * D + d) =
                        make_uint2(bf_pack(o.x * f, o.y * f), bf_pack(o.z * f, o.w * f));
                    if (d == 0 && p.lse)
                        p.lse[static_cast<int64_t>(head0 + h) * cv.n_seqs + b] =
                            l == 0.f ? -INFINITY : 0.6931471805599453f * (lm + log2f(l));
                }
                if (tid == 0) p.counters[c0] = 0;
            }
        }
        __syncthreads();  // the ring is free again
        u = seg_end;
    }
}

}  // namespace spava
