// skv_rows.cuh -- what the operators on rows and pages of a paged cache share: the
// e4m3 quantiser, and small host checks.
#pragma once

#include <cuda_fp8.h>

#include <atomic>

#include "skv_paged.h"

namespace skv {

// A head's scale s, brought between 2^-85 and 2^64 together with the values (`by`, a power of two):
// there 1 / s and the remainders below are exact enough at either end of binary32. A value that
// leaves binary32 on the way saturates, or is 0, like its quotient.
struct ScaleOf {
    float by, s, r;
};

__device__ __forceinline__ ScaleOf scale_of(float s) {
    ScaleOf o;
    o.by = s < 0x1p-64f ? 0x1p64f : s > 0x1p64f ? 0x1p-64f : 1.0f;
    o.s = s * o.by;
    o.r = __fdiv_rn(1.0f, o.s);
    return o;
}

// The e4m3 code nearest to x / s. The binary32 quotient alone can land on a tie
// that the real quotient only comes near, so it is rounded to odd first: the
// remainder x - q s is exact in an fma for any q within a step of the quotient, and
// where it is not 0 the quotient is cut towards 0 and its last bit set, which keeps it
// off every border of the much coarser code grid. q: one product with the
// reciprocal of s and one correction by the remainder.
__device__ __forceinline__ uint32_t e4m3_of(float value, const ScaleOf &c) {
    const float x = value * c.by;
    float q = x * c.r;
    if (fabsf(q) >= 1.0e-30f && fabsf(q) < 1.0e30f) {
        q = fmaf(fmaf(-q, c.s, x), c.r, q);
        const float rem = fmaf(-q, c.s, x);
        uint32_t b = __float_as_uint(q);
        // the remainder's sign against the quotient's (s > 0): q is too large in magnitude
        if ((__float_as_uint(rem) ^ b) >> 31) --b;
        if (rem != 0.0f) q = __uint_as_float(b | 1u);
    }
    return (uint32_t)__nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float bf16_float(uint32_t bits) { return __uint_as_float(bits << 16); }

// Two binary32 numbers that one instruction works on; each is rounded as by itself.
__device__ __forceinline__ uint64_t bits2(float2 a) { return (uint64_t)__float_as_uint(a.y) << 32 | __float_as_uint(a.x); }
__device__ __forceinline__ float2 floats2(uint64_t b) { return make_float2(__uint_as_float((uint32_t)b), __uint_as_float((uint32_t)(b >> 32))); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return floats2(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return floats2(r);
}

// Four codes, the same as e4m3_of's. The product with the reciprocal is within 2^-22 of the real quotient, so where a
// little more and a little less than it have one code, that is the code; only a value next to a border (one
// in some 60,000) takes the long way.
__device__ __forceinline__ uint32_t e4m3x4_of(const float2 &a, const float2 &b, const ScaleOf &c) {
    const float2 r = make_float2(c.r, c.r), up = make_float2(1.0f + 0x1p-21f, 1.0f + 0x1p-21f), down = make_float2(1.0f - 0x1p-21f, 1.0f - 0x1p-21f);
    const bool plain = c.by == 1.0f;
    const float2 x = mul2(plain ? a : make_float2(a.x * c.by, a.y * c.by), r), y = mul2(plain ? b : make_float2(b.x * c.by, b.y * c.by), r);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 u = mul2(x, i ? up : down), v = mul2(y, i ? up : down);
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(u.y), "f"(u.x));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v.y), "f"(v.x));
        w[i] = (uint32_t)hi << 16 | lo;
    }
    if (w[0] == w[1]) return w[0];
    return e4m3_of(a.x, c) | (e4m3_of(a.y, c) << 8) | (e4m3_of(b.x, c) << 16) | (e4m3_of(b.y, c) << 24);
}

inline bool device_sms(uint32_t *sms) {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return false;
    *sms = (uint32_t)n;
    return true;
}

// Clusters of more than eight CTAs and as much shared memory as there is, once per kernel and device.
inline bool allow_cluster(const void *kernel, std::atomic<uint64_t> &ready) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (bit && (ready.load(std::memory_order_relaxed) & bit)) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) != cudaSuccess)
        return false;
    ready.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

inline bool aligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

}  // namespace skv
