// row_kernels.cuh -- the operators that work on one head row at a time: RMS
// norm and rotation of queries and keys, writing keys and values into the paged
// cache (alone or behind the norm and rotation), reading cached rows back.
//
// All three are bound by memory (every row is read once and written once) as
// long as the work beside it stays small; what tokens share -- angles, weights,
// cache places -- is made once a block, in shared memory, and rows are taken heads outside, tokens inside.
#pragma once

#include "cache_common.cuh"
#include "sm100.cuh"

namespace spava {

constexpr int kRowThreads = 256;
constexpr int kRowTokens = 16;    // most tokens of a row_kernel block with tables,
constexpr int kWriteTokens = 32;  // of one without
constexpr int kReadTokens = 16;  // of a read_kernel block

struct RowParams {
    // Sources, in the order of a token's items: Hq query heads, Hk key heads,
    // Hv value heads; a source that a call does not have has no heads.
    const __nv_bfloat16 *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    const __nv_bfloat16 *q_weight, *k_weight;
    const float *inv_freq;
    const int32_t *positions;  // [axes, n_rows]
    __nv_bfloat16 *q_out, *k_out;
    int64_t n_rows;
    int32_t Hq, Hk, Hv;
    int32_t tokens_log2;  // tokens of a block
    FastDiv splits;       // blocks that share a token group's items
    int32_t rope_dim, interleaved, norm;
    int32_t cut1, cut2, cut3;  // first pair of axes 1, 2, 3
    float eps;
    // CACHE != 0
    CacheView cache;
    FastDiv new_rows;
};

// Pool row of KV head 0 of a token row, kNoRow if it has no place.  Places count
// back from the length as it is given: from the table's end, the rows of a sequence
// that has outgrown it would fall on those that it holds.
__device__ __forceinline__ uint32_t row_slot(const RowParams &p, uint32_t row) {
    uint32_t i;
    const uint32_t b = p.new_rows.quot(row, i);
    const int n = p.cache.lens[b], len = fit_len(p.cache, n);
    if (n < 0) return kNoRow;
    const int pos = n - static_cast<int>(p.new_rows.d) + static_cast<int>(i);
    return pos >= 0 && pos < len ? cache_row(p.cache, b, pos) : kNoRow;
}

__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }

// Eight bf16 values as four pairs of fp32, and back.
__device__ __forceinline__ void unpack8(const uint4 &w, float2 (&x)[4]) {
    x[0] = make_float2(bf_lo(w.x), bf_hi(w.x)), x[1] = make_float2(bf_lo(w.y), bf_hi(w.y));
    x[2] = make_float2(bf_lo(w.z), bf_hi(w.z)), x[3] = make_float2(bf_lo(w.w), bf_hi(w.w));
}
__device__ __forceinline__ uint4 pack8(const float2 (&x)[4]) {
    return make_uint4(bf_pack(x[0].x, x[0].y), bf_pack(x[1].x, x[1].y), bf_pack(x[2].x, x[2].y),
                      bf_pack(x[3].x, x[3].y));
}

// Largest magnitude of eight bf16 values, NaN apart, in both halves' maximum.
__device__ __forceinline__ __nv_bfloat162 amax8(const uint4 &w) {
    const uint32_t u[4] = {w.x & 0x7fff7fffu, w.y & 0x7fff7fffu, w.z & 0x7fff7fffu, w.w & 0x7fff7fffu};
    const __nv_bfloat162 *x = reinterpret_cast<const __nv_bfloat162 *>(u);
    return __hmax2(__hmax2(x[0], x[1]), __hmax2(x[2], x[3]));
}
// The same over the finite ones (a row with an infinity).
__device__ __forceinline__ float amax8_finite(const uint4 &w) {
    float2 x[4];
    unpack8(w, x);
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = fabsf(x[i].x), b = fabsf(x[i].y);
        m = fmaxf(m, a < INFINITY ? a : 0.f);  // false for NaN too
        m = fmaxf(m, b < INFINITY ? b : 0.f);
    }
    return m;
}
// Eight bf16 values times 2^-e as e4m3.
template <bool INF>  // infinities, which become NaN, may be among them
__device__ __forceinline__ uint2 e4m3_8(const uint4 &w, float inv) {
    float2 x[4];
    unpack8(w, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 y = fmul2(x[i], make_float2(inv, inv));
        if (INF) {
            x[i].x = fabsf(x[i].x) == INFINITY ? NAN : y.x;
            x[i].y = fabsf(x[i].y) == INFINITY ? NAN : y.y;
        } else {
            x[i] = y;
        }
    }
    return make_uint2(e4m3x2_of(x[0].x, x[0].y) | static_cast<uint32_t>(e4m3x2_of(x[1].x, x[1].y)) << 16,
                      e4m3x2_of(x[2].x, x[2].y) | static_cast<uint32_t>(e4m3x2_of(x[3].x, x[3].y)) << 16);
}

// (a, b) turned by the angles of (cos, sin), two pairs at a time.
__device__ __forceinline__ void turn2(float2 &a, float2 &b, float2 cs, float2 sn) {
    const float2 x = a, y = b;
    a = ffma2(x, cs, fmul2(neg2(y), sn));
    b = ffma2(y, cs, fmul2(x, sn));
}

// One item is one head row of one token; D/16 lanes hold it, each two 16-byte
// chunks, chosen so that both elements of every rotated pair are in one lane:
// chunks (l, l + rope_dim/16) where the halves of the rotated part pair up.
//
// The angle is position * inv_freq radians.  In turns, t = position *
// (inv_freq / 2 pi) is exact to 2^-52 relative in 64 bits, t - rint(t) loses
// nothing, and what is left of it fits 32 bits: an error below 1e-6 radians for
// any 31-bit position, where a 32-bit product is off by up to 2^-24 of the
// angle itself (0.008 radians at position 131072).
//
// Measured, 28/4 heads of 128: 131072 tokens 350 us, 6.1 TB/s read and written (0.93
// of the copy rate); 16384 tokens 49.1 us; e4m3 write of 16384 tokens, 4 KV heads,
// 10.8 us; one token with its write 2.7 us.
//
// ROPE: norm or rotation of queries and keys.  CACHE: 0 none, 1 bf16, 2 e4m3.
template <int D, int CACHE, bool ROPE>
__global__ void __launch_bounds__(kRowThreads, ROPE ? 4 : 7) row_kernel(const __grid_constant__ RowParams p) {
    constexpr int L = D / 16;               // lanes of an item
    constexpr int ITEMS = kRowThreads / L;  // items of a pass
    // What lane l needs is float4 [..][l] of a table: no bank conflicts.
    __shared__ float4 s_w[2][4][L];                          // weights: chunk c0, then c1
    __shared__ float4 s_cs[ROPE ? kRowTokens : 1][4][L];     // cosines (c0's or the pairs' first four), ...
    __shared__ uint32_t s_slot[kWriteTokens];
    launch_dependents();
    wait_for_primary();

    const int tid = threadIdx.x, l = tid % L;
    uint32_t part;
    const uint32_t chunk = p.splits.quot(blockIdx.x, part);
    const int tokens = 1 << p.tokens_log2;
    const uint32_t row0 = chunk << p.tokens_log2;
    const int n_tok = static_cast<int>(min(static_cast<int64_t>(tokens), p.n_rows - row0));
    const int n_items = (p.Hq + p.Hk + p.Hv) << p.tokens_log2, step = p.splits.d * ITEMS;

    const int half = p.rope_dim / 2;
    const int turn = p.rope_dim / 16;  // lanes or chunks of one half of the rotated part
    const bool pairs = ROPE && p.interleaved;
    int c0 = l, c1 = l + L;
    if (ROPE && !pairs && turn < L) {
        c0 = l < turn ? l : 2 * l;
        c1 = l < turn ? l + turn : 2 * l + 1;
    }

    struct Item {
        uint4 w0, w1;
        int head, tok;  // head among all; tok < 0: none
    };
    auto load = [&](int at) {
        Item x;
        x.w0 = x.w1 = make_uint4(0, 0, 0, 0);
        x.head = at >> p.tokens_log2;
        x.tok = at & (tokens - 1);
        if (at >= n_items || x.tok >= n_tok) {
            x.tok = -1;
            return x;
        }
        const uint32_t row = row0 + x.tok;
        const __nv_bfloat16 *src;
        if (x.head < p.Hq)
            src = p.q + row * p.q_stride + x.head * D;
        else if (x.head < p.Hq + p.Hk)
            src = p.k + row * p.k_stride + (x.head - p.Hq) * D;
        else
            src = p.v + row * p.v_stride + (x.head - p.Hq - p.Hk) * D;
        const uint4 *w0 = reinterpret_cast<const uint4 *>(src + c0 * 8), *w1 = reinterpret_cast<const uint4 *>(src + c1 * 8);
        // a plain write leaves L2 to the pool (e4m3, 16K tokens: 11.1 instead of 12.0 us)
        x.w0 = ROPE ? *w0 : __ldcs(w0);
        x.w1 = ROPE ? *w1 : __ldcs(w1);
        return x;
    };
    int at = part * ITEMS + tid / L;
    Item x = load(at);

    // ---- what the block's tokens share
    if (CACHE && tid >= kRowThreads - kWriteTokens) {
        const int t = tid - (kRowThreads - kWriteTokens);
        s_slot[t] = t < n_tok ? row_slot(p, row0 + t) : kNoRow;
    }
    if (ROPE) {
        if (p.norm) {
            for (int i = tid; i < 2 * D; i += kRowThreads) {
                // element e of the head is float e % 8 of a chunk of some lane
                const int kind = i / D, e = i % D, chunk_of = e / 8;
                int lane = chunk_of % L, second = chunk_of / L;
                if (!pairs && turn < L) {
                    if (chunk_of < 2 * turn)
                        lane = chunk_of % turn, second = chunk_of / turn;
                    else
                        lane = chunk_of / 2, second = chunk_of % 2;
                }
                const __nv_bfloat16 *wt = kind == 0 ? p.q_weight : p.k_weight;
                reinterpret_cast<float *>(&s_w[kind][2 * second + e % 8 / 4][lane])[e % 4] =
                    wt ? __bfloat162float(wt[e]) : 1.f;
            }
        }
        for (int i = tid; i < n_tok * (D / 2); i += kRowThreads) {
            const int t = i / (D / 2), j = i % (D / 2);
            if (j >= half) continue;
            const int axis = (j >= p.cut1) + (j >= p.cut2) + (j >= p.cut3);
            const int pos = p.positions[axis * p.n_rows + row0 + t];
            const double a =
                static_cast<double>(pos) * (static_cast<double>(p.inv_freq[j]) * 0.15915494309189533577);
            float sn, cs;
            sincospif(2.f * static_cast<float>(a - rint(a)), &sn, &cs);
            // pair j: float j % 8 of lane j / 8, or float j % 4 of chunk j / 4
            const int lane = pairs ? j / 4 % L : j / 8, which = pairs ? j / 4 / L : j / 4 % 2;
            reinterpret_cast<float *>(&s_cs[t][which][lane])[j % 4] = cs;
            reinterpret_cast<float *>(&s_cs[t][2 + which][lane])[j % 4] = sn;
        }
    }
    __syncthreads();

    // ---- item after item, the next one's load under way
    for (; at < part * ITEMS + (n_items - static_cast<int>(part) * ITEMS + step - 1) / step * step; at += step) {
        const Item next = load(at + step);
        uint4 w0 = x.w0, w1 = x.w1;
        const int kind = x.head < p.Hq ? 0 : x.head < p.Hq + p.Hk ? 1 : 2;
        const int head = x.head - (kind > 0 ? p.Hq : 0) - (kind > 1 ? p.Hk : 0);
        const int tok = max(x.tok, 0);
        if (ROPE) {
            float2 x0[4], x1[4];
            unpack8(w0, x0);
            unpack8(w1, x1);
            if (p.norm) {
                float2 ss = fmul2(x0[0], x0[0]);
#pragma unroll
                for (int i = 1; i < 4; ++i) ss = ffma2(x0[i], x0[i], ss);
#pragma unroll
                for (int i = 0; i < 4; ++i) ss = ffma2(x1[i], x1[i], ss);
                float sum = ss.x + ss.y;
#pragma unroll
                for (int o = 1; o < L; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                const float r = rsqrtf(sum * (1.0f / D) + p.eps);
                const float2 r2 = make_float2(r, r);
                const float4(&wt)[4][L] = s_w[kind == 0 ? 0 : 1];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 g0 = wt[i][l], g1 = wt[2 + i][l];
                    x0[2 * i] = fmul2(fmul2(x0[2 * i], r2), make_float2(g0.x, g0.y));
                    x0[2 * i + 1] = fmul2(fmul2(x0[2 * i + 1], r2), make_float2(g0.z, g0.w));
                    x1[2 * i] = fmul2(fmul2(x1[2 * i], r2), make_float2(g1.x, g1.y));
                    x1[2 * i + 1] = fmul2(fmul2(x1[2 * i + 1], r2), make_float2(g1.z, g1.w));
                }
            }
            if (pairs) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float2(&y)[4] = k ? x1 : x0;
                    if ((k ? c1 : c0) * 8 < p.rope_dim) {
                        const float4 cs = s_cs[tok][k][l], sn = s_cs[tok][2 + k][l];
                        float2 a = make_float2(y[0].x, y[1].x), b = make_float2(y[0].y, y[1].y);
                        turn2(a, b, make_float2(cs.x, cs.y), make_float2(sn.x, sn.y));
                        y[0] = make_float2(a.x, b.x), y[1] = make_float2(a.y, b.y);
                        a = make_float2(y[2].x, y[3].x), b = make_float2(y[2].y, y[3].y);
                        turn2(a, b, make_float2(cs.z, cs.w), make_float2(sn.z, sn.w));
                        y[2] = make_float2(a.x, b.x), y[3] = make_float2(a.y, b.y);
                    }
                }
            } else if (l < turn) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 cs = s_cs[tok][i][l], sn = s_cs[tok][2 + i][l];
                    turn2(x0[2 * i], x1[2 * i], make_float2(cs.x, cs.y), make_float2(sn.x, sn.y));
                    turn2(x0[2 * i + 1], x1[2 * i + 1], make_float2(cs.z, cs.w), make_float2(sn.z, sn.w));
                }
            }
            if (kind < 2) {
                w0 = pack8(x0);
                w1 = pack8(x1);
                __nv_bfloat16 *out = kind == 0 ? p.q_out : p.k_out;
                if (x.tok >= 0 && out) {
                    out += (static_cast<int64_t>(row0 + tok) * (kind == 0 ? p.Hq : p.Hk) + head) * D;
                    *reinterpret_cast<uint4 *>(out + c0 * 8) = w0;
                    *reinterpret_cast<uint4 *>(out + c1 * 8) = w1;
                }
            }
        }
        if (CACHE) {
            uint32_t slot = x.tok >= 0 && kind > 0 ? s_slot[tok] : kNoRow;
            const bool stores = slot != kNoRow;
            slot += head * p.cache.page.d;
            if (CACHE == 1) {
                __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(kind == 1 ? p.cache.k : p.cache.v) +
                                    static_cast<int64_t>(slot) * D;
                if (stores) {
                    *reinterpret_cast<uint4 *>(to + c0 * 8) = w0;
                    *reinterpret_cast<uint4 *>(to + c1 * 8) = w1;
                }
            } else {
                const __nv_bfloat162 m2 = __hmax2(amax8(w0), amax8(w1));
                float m = __bfloat162float(__hmax(m2.x, m2.y));
#pragma unroll
                for (int o = 1; o < L; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                const bool inf = m == INFINITY;
                if (__any_sync(0xffffffffu, inf)) {
                    float f = fmaxf(amax8_finite(w0), amax8_finite(w1));
#pragma unroll
                    for (int o = 1; o < L; o <<= 1) f = fmaxf(f, __shfl_xor_sync(0xffffffffu, f, o));
                    m = f;
                }
                // a row of NaN has no magnitude: __hmax2 gives NaN, fmaxf and the test below 0
                const int e = e4m3_row_exp(m == m ? m : 0.f);
                const float inv = pow2f(-e);
                if (stores) {
                    uint8_t *to = static_cast<uint8_t *>(kind == 1 ? p.cache.k : p.cache.v) +
                                  static_cast<int64_t>(slot) * D;
                    *reinterpret_cast<uint2 *>(to + c0 * 8) = inf ? e4m3_8<true>(w0, inv) : e4m3_8<false>(w0, inv);
                    *reinterpret_cast<uint2 *>(to + c1 * 8) = inf ? e4m3_8<true>(w1, inv) : e4m3_8<false>(w1, inv);
                    if (l == 0) (kind == 1 ? p.cache.k_exp : p.cache.v_exp)[slot] = static_cast<int8_t>(e);
                }
            }
        }
        x = next;
    }
}

struct ReadParams {
    CacheView cache;
    __nv_bfloat16 *k_out, *v_out;
    int64_t n_rows;  // n_seqs * rows
    int32_t first, tokens_log2;
    FastDiv rows, heads, splits;
};

// A block reads up to 16 tokens, whose places it looks up first; an item is one
// KV head of one token, key and value, heads fastest as they are written.  D / 8
// lanes take a row, 16 bytes each on the written side, which a store instruction
// then covers without gaps, and four rows are under way in a thread.  Measured,
// 65536 tokens, 4 KV heads of 128, e4m3: 34.7 us, 5.8 TB/s read and written.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kRowThreads) read_kernel(const __grid_constant__ ReadParams p) {
    constexpr int L = D / 8, ITEMS = kRowThreads / L, AHEAD = 2;
    __shared__ uint32_t s_slot[kReadTokens];
    launch_dependents();
    wait_for_primary();
    const int tid = threadIdx.x, l = tid % L;
    uint32_t part;
    const uint32_t chunk = p.splits.quot(blockIdx.x, part);
    const uint32_t row0 = chunk << p.tokens_log2;
    const int n_tok = static_cast<int>(min(static_cast<int64_t>(1) << p.tokens_log2, p.n_rows - row0));
    if (tid < n_tok) {
        uint32_t i;
        const uint32_t b = p.rows.quot(row0 + tid, i);
        const int pos = p.first + static_cast<int>(i);
        s_slot[tid] = pos < cache_len(p.cache, b) ? cache_row(p.cache, b, pos) : kNoRow;
    }
    __syncthreads();
    const int n_items = n_tok * static_cast<int>(p.heads.d), step = p.splits.d * ITEMS;
    for (int at = part * ITEMS + tid / L; at < n_items; at += AHEAD * step) {
        uint4 x[AHEAD][2];  // keys, values: 8 bytes of e4m3 or 16 of bf16
        int e[AHEAD][2];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            x[k][0] = x[k][1] = make_uint4(0, 0, 0, 0);
            e[k][0] = e[k][1] = 0;
            if (at + k * step < n_items) {
                uint32_t head;
                const uint32_t tok = p.heads.quot(at + k * step, head);
                uint32_t slot = s_slot[tok];
                if (slot != kNoRow) {
                    slot += head * p.cache.page.d;
                    const int64_t from = (static_cast<int64_t>(slot) * L + l) * (E4M3 ? 8 : 16);
                    const char *ks = static_cast<const char *>(p.cache.k) + from;
                    const char *vs = static_cast<const char *>(p.cache.v) + from;
                    if (E4M3) {
                        const uint2 a = __ldcs(reinterpret_cast<const uint2 *>(ks));
                        const uint2 b = __ldcs(reinterpret_cast<const uint2 *>(vs));
                        x[k][0].x = a.x, x[k][0].y = a.y, x[k][1].x = b.x, x[k][1].y = b.y;
                        e[k][0] = p.cache.k_exp[slot];
                        e[k][1] = p.cache.v_exp[slot];
                    } else {
                        x[k][0] = __ldcs(reinterpret_cast<const uint4 *>(ks));
                        x[k][1] = __ldcs(reinterpret_cast<const uint4 *>(vs));
                    }
                }
            }
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (at + k * step < n_items) {
                const int64_t to =
                    (static_cast<int64_t>(row0) * p.heads.d + at + k * step) * L + l;
#pragma unroll
                for (int which = 0; which < 2; ++which) {
                    uint4 w = x[k][which];
                    if (E4M3) {
                        const float f = pow2f(max(e[k][which], -126));
                        const uint32_t u[2] = {w.x, w.y};
                        float2 y[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t h =
                                f16x2_of_e4m3x2(static_cast<uint16_t>(u[j / 2] >> (16 * (j % 2))));
                            y[j] = fmul2(__half22float2(*reinterpret_cast<const __half2 *>(&h)), make_float2(f, f));
                        }
                        w = pack8(y);
                    }
                    reinterpret_cast<uint4 *>(which ? p.v_out : p.k_out)[to] = w;
                }
            }
    }
}

}  // namespace spava
