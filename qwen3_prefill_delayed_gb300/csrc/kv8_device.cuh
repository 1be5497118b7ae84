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
// a scale (0 or a power of two from 2^-126 on; -1 where a kernel marks an absent block) as exponent and factor: the factor is 0
// for a scale of 0, which so gives a weight of 0, and else 1
__device__ __forceinline__ float exponent_of(float s) { return (float)((int)((__float_as_uint(s) >> 23) & 255u) - 127); }
__device__ __forceinline__ float mantissa_of(float s) {
    return s == 0.f ? 0.f : __uint_as_float((__float_as_uint(s) & 0x807FFFFFu) | 0x3F800000u);
}

// A V with a NaN at a position that some rows of a tile see and others do not: the tile's product carries it, by a weight of 0,
// to the rows that do not.  Nothing on the way looks for that; an output that is a NaN is looked at here, by the thread that
// wrote it: dims dim .. dim + n - 1 (n <= 32) of a row that sees positions [0, end) while its tile's last row sees
// [0, keys).  Those with a NaN behind `end` are done again, from the definition.
[[maybe_unused]] static __device__ __noinline__ void kv8_row_again(const Kv8View& c, const bf16* q, int row, int head, int end,
                                                                   int keys, int dim, int n, float scale_log2, bf16* out) {
    uint32_t dims = 0u;
    for (int pos = max(0, end); pos < keys; ++pos) {
        const int page = kv8_page_of(c, row, pos);
        if (page < 0) continue;
        const uint8_t* v = c.codes + kv8_code_at(c, page, 1, head, pos & (c.page_size - 1)) + dim;
        for (int i = 0; i < n; ++i) dims |= (v[i] & 0x7Fu) == 0x7Fu ? 1u << i : 0u;
    }
    if (dims == 0u) return;
    auto value = [](uint8_t code) {
        const uint32_t h = e4m3x2_f16x2(code);
        return __half2float(*reinterpret_cast<const __half*>(&h));
    };
    float m = -INFINITY, l = 0.f, acc[32];
    for (int i = 0; i < n; ++i) acc[i] = 0.f;
    for (int pos = 0; pos < end; ++pos) {
        const int page = kv8_page_of(c, row, pos), slot = pos & (c.page_size - 1);
        if (page < 0) continue;
        const uint8_t* k = c.codes + kv8_code_at(c, page, 0, head, slot);
        const uint8_t* v = c.codes + kv8_code_at(c, page, 1, head, slot) + dim;
        float s = 0.f;
        for (int d = 0; d < c.head_dim; ++d) s += __bfloat162float(q[d]) * value(k[d]);
        s *= c.scales[kv8_scale_at(c, page, 0, head, slot)] * scale_log2;
        // what the row sees is a NaN itself: its outputs are, and stay
        for (int i = 0; i < n; ++i) dims &= (v[i] & 0x7Fu) == 0x7Fu ? ~(1u << i) : ~0u;
        if (s != s || dims == 0u) return;
        const float mn = fmaxf(m, s), r = mn == -INFINITY ? 0.f : mn;
        const float before = exp2f(m - r), w = exp2f(s - r), vs = c.scales[kv8_scale_at(c, page, 1, head, slot)];
        m = mn;
        l = l * before + w;
        for (int i = 0; i < n; ++i) acc[i] = acc[i] * before + w * (value(v[i]) * vs);
    }
    for (int i = 0; i < n; ++i)
        if (dims >> i & 1u) out[i] = __float2bfloat16_rn(l == 0.f ? 0.f : acc[i] / l);
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
