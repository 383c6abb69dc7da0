// cache_common.cuh -- what the kernels around the paged cache share: division
// by a run-time constant, the paged address of a position, e4m3 conversion.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "status.cuh"

namespace spava {

// Quotient by a divisor known at launch, for n < 2^31: floor(n / d) =
// floor(n * m / 2^(32 + s)) with m = ceil(2^(32 + s) / d), s = ceil(log2 d) - 1
// (the rounding of m adds less than n / 2^(32+s) < 1/d to the product).
struct FastDiv {
    uint32_t d, m, s;
    static FastDiv of(uint32_t d) {
        FastDiv f{d, 0, 0};
        if (d > 1) {
            uint32_t l = 0;
            while ((1ULL << l) < d) ++l;
            f.s = l - 1;
            f.m = static_cast<uint32_t>(((1ULL << (32 + f.s)) + d - 1) / d);
        }
        return f;
    }
    __device__ __forceinline__ uint32_t quot(uint32_t n) const {
        return d == 1 ? n : __umulhi(n, m) >> s;
    }
    __device__ __forceinline__ uint32_t quot(uint32_t n, uint32_t &rem) const {
        const uint32_t q = quot(n);
        rem = n - q * d;
        return q;
    }
};

constexpr uint32_t kNoRow = 0xffffffffu;  // no row of the pool (row counts stay below it)

// What the kernels need of a cache and a batch.
struct CacheView {
    void *k, *v;
    int8_t *k_exp, *v_exp;
    const int32_t *table;
    const int32_t *lens;
    int *status;
    int64_t max_pages;
    uint32_t n_pages, n_rows;  // of the pool; n_rows = n_pages * Hkv * page_size
    int32_t n_seqs, Hkv;
    int32_t cap;  // positions of the table: max_pages * page_size
    FastDiv page;
};

// The tokens of sequence b, made to fit the table; out-of-range lengths are
// reported in the status word.
__device__ __forceinline__ int fit_len(const CacheView &c, int n) {
    if (n < 0 || n > c.cap) {
        atomicOr(c.status, kStatusBadBatch);
        return n < 0 ? 0 : c.cap;
    }
    return n;
}
__device__ __forceinline__ int cache_len(const CacheView &c, int b) { return fit_len(c, c.lens[b]); }

// Pool row of (sequence b, position, KV head 0), kNoRow if its page is outside
// the pool.  Head h lies h * page_size rows further.
__device__ __forceinline__ uint32_t cache_row(const CacheView &c, int b, int pos) {
    uint32_t off;
    const uint32_t at = c.page.quot(static_cast<uint32_t>(pos), off);
    const int page = c.table[b * c.max_pages + at];
    if (static_cast<uint32_t>(page) >= c.n_pages) {
        atomicOr(c.status, kStatusBadBatch);
        return kNoRow;
    }
    return static_cast<uint32_t>(page) * c.Hkv * c.page.d + off;
}

// ------------------------------------------------------------------ dependent launches
// Every kernel here is launched as a programmatic dependent of the stream's last
// one: it may come onto the SMs before that has ended, and touches no memory
// before wait_for_primary, which every thread passes and which returns when all
// work before has ended and is visible.  launch_dependents lets the next kernel
// do the same: a decode step is a chain of launches of a few microseconds.  No
// load goes by ld.global.nc: what the kernel before still writes is not
// read-only for this one's whole life.
__device__ __forceinline__ void launch_dependents() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_primary() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename P>
inline spava_status launch(void (*kernel)(P), unsigned grid, unsigned threads, int smem, int cluster,
                           cudaStream_t st, const P &p) {
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cuda_ok(cudaLaunchKernelEx(&cfg, kernel, p));
}

// ------------------------------------------------------------------ e4m3
// Exponent of a row whose largest finite magnitude is amax: the smallest
// e >= -120 with amax <= 448 * 2^e.  448 = 1.75 * 2^8, so with amax = 1.m * 2^x
// e = x - 8, and one more if 1.m > 1.75.
__device__ __forceinline__ int e4m3_row_exp(float amax) {
    const uint32_t u = __float_as_uint(amax);
    return max(static_cast<int>(u >> 23) - 135 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0), -120);
}
__device__ __forceinline__ float pow2f(int e) {  // -126 <= e <= 127
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}
// lo in the low byte; round to nearest even, the values are within +-448.
__device__ __forceinline__ uint16_t e4m3x2_of(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Every e4m3 value is an fp16 value: exact.
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint16_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
    return r;
}

// Halves of a packed bf16 pair as fp32.
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

}  // namespace spava
