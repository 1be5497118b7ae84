// kv8_device.cuh -- device helpers that the kernels of the paged 8-bit cache share.
#pragma once

#include <cuda_fp16.h>

#include "internal.h"

namespace hra {

// 2^x, flushing to zero
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// two E4M3 codes (the low 16 bits) <-> two f16; four codes -> two pairs of f16
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((unsigned short)w));
    return d;
}
__device__ __forceinline__ uint32_t f16x2_e4m3x2(uint32_t v) {
    unsigned short d;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(d) : "r"(v));
    return d;
}
__device__ __forceinline__ void e4m3x4_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
// a scale's floor(log2), and the scale over 2^that
__device__ __forceinline__ float exponent_of(float s) { return (float)((int)((__float_as_uint(s) >> 23) & 255u) - 127); }
__device__ __forceinline__ float mantissa_of(float s) {
    return __uint_as_float((__float_as_uint(s) & 0x807FFFFFu) | 0x3F800000u);
}

// Exclusive scan of one value a thread over a CTA of 1024 threads; total gets the sum.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T& total) {
    __shared__ T warp_sum_s[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    T incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) warp_sum_s[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        T t = warp_sum_s[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T u = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += u;
        }
        warp_sum_s[lane] = t;
    }
    __syncthreads();
    const T before = warp ? warp_sum_s[warp - 1] : 0;
    total = warp_sum_s[31];
    __syncthreads();
    return before + incl - v;
}

}  // namespace hra
