// row_kernels.cuh -- the operators that work on one head row at a time: RMS
// norm and rotation of queries and keys, writing keys and values into the paged
// cache (alone or behind the norm and rotation), reading cached rows back.
#pragma once

#include "cache_common.cuh"

namespace spava {

constexpr int kRowThreads = 256;

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
    uint32_t n_items;  // n_rows * heads
    int32_t Hq, Hk, Hv;
    int32_t rope_dim, interleaved, norm;
    int32_t cut1, cut2, cut3;  // first pair of axes 1, 2, 3
    float eps;
    FastDiv heads;  // Hq + Hk + Hv
    // CACHE != 0
    CacheView cache;
    FastDiv new_rows;
};

// One token row's place among the sequences.
struct RowPlace {
    int b, pos;
};
__device__ __forceinline__ RowPlace row_place(const RowParams &p, uint32_t row) {
    uint32_t i;
    const uint32_t b = p.new_rows.quot(row, i);
    const int len = cache_len(p.cache, b);
    return {static_cast<int>(b), len - static_cast<int>(p.new_rows.d) + static_cast<int>(i)};
}

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8]) {
    x[0] = bf_lo(w.x), x[1] = bf_hi(w.x), x[2] = bf_lo(w.y), x[3] = bf_hi(w.y);
    x[4] = bf_lo(w.z), x[5] = bf_hi(w.z), x[6] = bf_lo(w.w), x[7] = bf_hi(w.w);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(bf_pack(x[0], x[1]), bf_pack(x[2], x[3]), bf_pack(x[4], x[5]),
                      bf_pack(x[6], x[7]));
}

// Largest finite magnitude of eight bf16 values.
__device__ __forceinline__ float amax8(const uint4 &w) {
    float m = 0.f;
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = fabsf(bf_lo(u[i])), b = fabsf(bf_hi(u[i]));
        m = fmaxf(m, a < INFINITY ? a : 0.f);  // false for NaN too
        m = fmaxf(m, b < INFINITY ? b : 0.f);
    }
    return m;
}
// Eight bf16 values times 2^-e as e4m3; infinities become NaN.
__device__ __forceinline__ uint2 e4m3_8(const uint4 &w, float inv) {
    float x[8];
    unpack8(w, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fabsf(x[i]) == INFINITY ? NAN : x[i] * inv;
    return make_uint2(e4m3x2_of(x[0], x[1]) | static_cast<uint32_t>(e4m3x2_of(x[2], x[3])) << 16,
                      e4m3x2_of(x[4], x[5]) | static_cast<uint32_t>(e4m3x2_of(x[6], x[7])) << 16);
}

// One item is one head row of one token; D/16 lanes hold it, each two 16-byte
// chunks, chosen so that both elements of every rotated pair are in one lane:
// chunks (l, l + rope_dim/16) where the halves of the rotated part pair up.
// A block's items are consecutive, heads fastest, so it touches few tokens;
// their cosines and sines (rope_dim/2 pairs a token) are made once, in shared
// memory, by all its threads while the rows' loads are under way.
//
// The angle is position * inv_freq radians.  In turns, t = position *
// (inv_freq / 2 pi) is exact to 2^-52 relative in 64 bits, t - rint(t) loses
// nothing, and what is left of it fits 32 bits: an error below 1e-6 radians for
// any 31-bit position, where a 32-bit product is off by up to 2^-24 of the
// angle itself (0.008 radians at position 131072).
//
// CACHE: 0 none, 1 bf16, 2 e4m3.
template <int D, int CACHE>
__global__ void __launch_bounds__(kRowThreads) row_kernel(const __grid_constant__ RowParams p) {
    constexpr int L = D / 16;               // lanes of an item
    constexpr int ITEMS = kRowThreads / L;  // items of a block
    // Tokens a block can touch: an item set has at least two heads a token.
    constexpr int TOK = ITEMS / 2 + 1;
    __shared__ __align__(16) float s_cos[TOK * (D / 2)], s_sin[TOK * (D / 2)];

    launch_dependents();
    wait_for_primary();
    const uint32_t item0 = blockIdx.x * static_cast<uint32_t>(ITEMS);
    const uint32_t item = item0 + threadIdx.x / L;
    const int l = threadIdx.x % L;
    const bool live = item < p.n_items;
    uint32_t head;
    const uint32_t row = p.heads.quot(live ? item : item0, head);

    const int half = p.rope_dim / 2;
    const int turn = p.rope_dim / 16;  // lanes or chunks of one half of the rotated part
    int c0 = l, c1 = l + L;
    if (!p.interleaved && turn < L) {
        if (l < turn) {
            c1 = l + turn;
        } else {
            c0 = 2 * l;
            c1 = c0 + 1;
        }
    }
    const __nv_bfloat16 *src;
    int kind;  // 0 query, 1 key, 2 value
    if (head < static_cast<uint32_t>(p.Hq)) {
        kind = 0;
        src = p.q + row * p.q_stride + head * D;
    } else if (head < static_cast<uint32_t>(p.Hq + p.Hk)) {
        kind = 1;
        head -= p.Hq;
        src = p.k + row * p.k_stride + head * D;
    } else {
        kind = 2;
        head -= p.Hq + p.Hk;
        src = p.v + row * p.v_stride + head * D;
    }
    uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
    if (live) {
        w0 = *reinterpret_cast<const uint4 *>(src + c0 * 8);
        w1 = *reinterpret_cast<const uint4 *>(src + c1 * 8);
    }
    uint32_t slot = kNoRow;
    if (CACHE && live && kind > 0) {
        const RowPlace at = row_place(p, row);
        if (at.pos >= 0) slot = cache_row(p.cache, at.b, at.pos);
        if (slot != kNoRow) slot += head * p.cache.page.d;
    }

    const uint32_t tok0 = p.heads.quot(item0);
    if (half > 0) {
        const uint32_t last = min(item0 + ITEMS, p.n_items) - 1;
        const int n = static_cast<int>(p.heads.quot(last) - tok0 + 1) * half;
        for (int i = threadIdx.x; i < n; i += kRowThreads) {
            const int t = i / half, j = i - t * half;
            const int axis = (j >= p.cut1) + (j >= p.cut2) + (j >= p.cut3);
            const int pos = p.positions[axis * p.n_rows + tok0 + t];
            const double a = static_cast<double>(pos) *
                             (static_cast<double>(p.inv_freq[j]) * 0.15915494309189533577);
            const float r = static_cast<float>(a - rint(a));
            float sn, cs;
            sincospif(2.f * r, &sn, &cs);
            s_cos[i] = cs;
            s_sin[i] = sn;
        }
        __syncthreads();
    }

    if (kind < 2 && (p.norm || half > 0)) {
        float x0[8], x1[8];
        unpack8(w0, x0);
        unpack8(w1, x1);
        if (p.norm) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x0[i], x0[i], fmaf(x1[i], x1[i], ss));
#pragma unroll
            for (int o = 1; o < L; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float r = 1.0f / sqrtf(ss * (1.0f / D) + p.eps);
            const __nv_bfloat16 *wt = kind == 0 ? p.q_weight : p.k_weight;
            if (wt) {
                float g0[8], g1[8];
                unpack8(*reinterpret_cast<const uint4 *>(wt + c0 * 8), g0);
                unpack8(*reinterpret_cast<const uint4 *>(wt + c1 * 8), g1);
#pragma unroll
                for (int i = 0; i < 8; ++i) x0[i] = x0[i] * r * g0[i], x1[i] = x1[i] * r * g1[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) x0[i] *= r, x1[i] *= r;
            }
        }
        const int at = static_cast<int>(row - tok0) * half;
        if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                if (c0 * 8 < p.rope_dim) {
                    const int j = at + c0 * 4 + i / 2;
                    const float a = x0[i], b = x0[i + 1], cs = s_cos[j], sn = s_sin[j];
                    x0[i] = a * cs - b * sn;
                    x0[i + 1] = b * cs + a * sn;
                }
                if (c1 * 8 < p.rope_dim) {
                    const int j = at + c1 * 4 + i / 2;
                    const float a = x1[i], b = x1[i + 1], cs = s_cos[j], sn = s_sin[j];
                    x1[i] = a * cs - b * sn;
                    x1[i + 1] = b * cs + a * sn;
                }
            }
        } else if (l < turn) {
            const float4 *pc = reinterpret_cast<const float4 *>(s_cos + at + l * 8);
            const float4 *ps = reinterpret_cast<const float4 *>(s_sin + at + l * 8);
            const float4 ca = pc[0], cb = pc[1], sa = ps[0], sb = ps[1];
            const float cs[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
            const float sn[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = x0[i], b = x1[i];
                x0[i] = a * cs[i] - b * sn[i];
                x1[i] = b * cs[i] + a * sn[i];
            }
        }
        w0 = pack8(x0);
        w1 = pack8(x1);
    }

    if (live && kind < 2) {
        __nv_bfloat16 *out = kind == 0 ? p.q_out : p.k_out;
        if (out) {
            out += (static_cast<int64_t>(row) * (kind == 0 ? p.Hq : p.Hk) + head) * D;
            *reinterpret_cast<uint4 *>(out + c0 * 8) = w0;
            *reinterpret_cast<uint4 *>(out + c1 * 8) = w1;
        }
    }
    if (CACHE == 1 && slot != kNoRow) {
        __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(kind == 1 ? p.cache.k : p.cache.v) +
                            static_cast<int64_t>(slot) * D;
        *reinterpret_cast<uint4 *>(to + c0 * 8) = w0;
        *reinterpret_cast<uint4 *>(to + c1 * 8) = w1;
    }
    if (CACHE == 2) {
        float m = fmaxf(amax8(w0), amax8(w1));
#pragma unroll
        for (int o = 1; o < L; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (slot != kNoRow) {
            const int e = e4m3_row_exp(m);
            const float inv = pow2f(-e);
            uint8_t *to = static_cast<uint8_t *>(kind == 1 ? p.cache.k : p.cache.v) +
                          static_cast<int64_t>(slot) * D;
            *reinterpret_cast<uint2 *>(to + c0 * 8) = e4m3_8(w0, inv);
            *reinterpret_cast<uint2 *>(to + c1 * 8) = e4m3_8(w1, inv);
            if (l == 0) (kind == 1 ? p.cache.k_exp : p.cache.v_exp)[slot] = static_cast<int8_t>(e);
        }
    }
}

struct ReadParams {
    CacheView cache;
    __nv_bfloat16 *k_out, *v_out;
    int32_t first;
    uint32_t n_items;  // n_seqs * rows * Hkv
    FastDiv rows, heads;
};

// One item is one (sequence, position, KV head), key and value; D * size / 16
// lanes of 16 cached bytes each.  Heads run fastest: a token's outputs are
// contiguous.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kRowThreads) read_kernel(const __grid_constant__ ReadParams p) {
    constexpr int L = D * (E4M3 ? 1 : 2) / 16;
    constexpr int ITEMS = kRowThreads / L;
    launch_dependents();
    wait_for_primary();
    const uint32_t item = blockIdx.x * static_cast<uint32_t>(ITEMS) + threadIdx.x / L;
    if (item >= p.n_items) return;
    const int l = threadIdx.x % L;
    uint32_t head, i;
    const uint32_t row = p.heads.quot(item, head);
    const uint32_t b = p.rows.quot(row, i);
    const int pos = p.first + static_cast<int>(i);
    uint32_t slot = kNoRow;
    if (pos < cache_len(p.cache, b)) slot = cache_row(p.cache, b, pos);
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    int ke = 0, ve = 0;
    if (slot != kNoRow) {
        slot += head * p.cache.page.d;
        const int64_t at = static_cast<int64_t>(slot) * (D * (E4M3 ? 1 : 2)) + l * 16;
        k = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const char *>(p.cache.k) + at));
        v = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const char *>(p.cache.v) + at));
        if (E4M3) {
            ke = max(static_cast<int>(p.cache.k_exp[slot]), -126);
            ve = max(static_cast<int>(p.cache.v_exp[slot]), -126);
        }
    }
    const int64_t to = static_cast<int64_t>(item) * D;
    if (!E4M3) {
        reinterpret_cast<uint4 *>(p.k_out + to)[l] = k;
        reinterpret_cast<uint4 *>(p.v_out + to)[l] = v;
    } else {
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const uint4 w = which ? v : k;
            const float f = pow2f(which ? ve : ke);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            uint32_t r[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t h = f16x2_of_e4m3x2(static_cast<uint16_t>(u[j / 2] >> (16 * (j % 2))));
                const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                r[j] = bf_pack(x.x * f, x.y * f);
            }
            uint4 *out = reinterpret_cast<uint4 *>((which ? p.v_out : p.k_out) + to) + 2 * l;
            out[0] = make_uint4(r[0], r[1], r[2], r[3]);
            out[1] = make_uint4(r[4], r[5], r[6], r[7]);
        }
    }
}

}  // namespace spava
