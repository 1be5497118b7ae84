// kv8_append.cu -- K/V rows into the pages of the 8-bit cache.
//
// For each block of 16 positions, head, and K or V that the new rows touch:
//   a = max |x| over the block's new rows, s = the smallest power of two with a <= 448 s;
//   a block that already held tokens below the first new row takes s = max(stored s, s), and when s
//   has grown its earlier codes become e4m3(value * s_old / s);
//   code = e4m3(x / s) (round to nearest even; |x / s| <= 448, so nothing saturates but infinities).
// E4M3 is a floating-point format, so a power-of-two scale loses no precision against max|x| / 448: the
// division, the dequantisation and the re-scaling of earlier codes are exact in fp32, the last one
// except where a code falls under 2^-6 (E4M3's subnormals).
//
// One warp per (block, head, K|V): it reads the block's rows with 16-byte loads, all in flight
// before the first use, reduces the maximum, and writes the block's codes as 2 KB (head_dim 128) of
// contiguous memory.  No two warps share a block, so there are no atomics.
//
// Bound by memory: prompts of 11,400 rows x 8 heads x 128 (70 MB read and written) take 12.7 us in a captured graph over the
// pools of 36 layers, 5.5 TB/s (on one layer again and again, out of the L2, 9.8), and one frame of 8 rows 2.1 us, a launch's
// latency.  The maximum is taken on the bf16 bits
// and the rows are requested before the page is looked up: in fp32, after it, 100 registers hold 20 warps an SM
// instead of 32 (16.5 us; 7 CTAs of 4 warps 13.5, 6 13.9).  One warp for a block's K and V together took
// 16.5 us and 3.5 for the frame (its two chains of loads, maximum and stores follow one another).
#include <cuda_fp8.h>

#include "internal.h"

namespace hra {

namespace {

__device__ __forceinline__ uint2 to_e4m3x8(const float (&f)[8], float inv) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = make_float2(f[2 * i] * inv, f[2 * i + 1] * inv);
        w[i >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(p, __NV_SATFINITE, __NV_E4M3) << (16 * (i & 1));
    }
    return make_uint2(w[0], w[1]);
}

template <int HD>
__global__ void __launch_bounds__(128, 8) kv8_append_kernel(const Kv8AppendArgs a) {
    pdl_launch();
    pdl_wait();
    constexpr int LPR = HD / 8;                 // lanes that hold one row
    constexpr int RPL = 32 / LPR;               // rows of one pass
    constexpr int PASSES = kKv8Block / RPL;
    const Kv8View& c = a.view;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    const int unit = blockIdx.x * (blockDim.x >> 5) + warp;   // (block of the row, which, head)
    const int head = unit % c.n_kv;
    const int which = (unit / c.n_kv) & 1;
    const int blk = unit / (2 * c.n_kv);
    int row0, n;
    const int first = a.start[b];
    kv8_rows(a.cu, b, a.total_rows, row0, n);
    if (n == 0) return;
    const long long room = (long long)c.max_pages << c.page_shift;
    if (unit == 0 && lane == 0 && (first < 0 || first + (long long)n > room || n > a.max_new))
        raise_error(c.err, HRA_DEVERR_POS_RANGE);
    n = min(n, a.max_new);
    const bool keeps_len = unit == 0 && a.lens != nullptr;   // this warp writes the row's length
    // the error bit says so; the products below stay inside 32 bits
    if (first < 0 || first >= room) {   // nothing is written: the row holds no more than it did
        if (keeps_len && lane == 0 && first < 0) a.lens[b] = min(a.lens[b], max(0, first + n));
        return;
    }
    const int pos0 = (first / kKv8Block + blk) * kKv8Block;   // the block's first position
    if (pos0 < 0 || pos0 - first >= n) return;
    const int page = kv8_page_of(c, b, pos0);
    if (keeps_len) {   // nor does one none of whose new tokens has a page
        const int end = (int)min(room, (long long)first + n);
        bool any = page >= 0;
        for (int i = (first >> c.page_shift) + 1 + lane; !any && i <= (end - 1) >> c.page_shift; i += 32)
            any = kv8_page_of(c, b, i << c.page_shift) >= 0;
        any = __any_sync(0xffffffffu, any);
        if (lane == 0) a.lens[b] = any ? end : min(a.lens[b], end);
    }
    const int lo = max(0, first - pos0);                 // new rows are slots [lo, hi) of the block
    const int hi = min(kKv8Block, first - pos0 + n);
    const bf16* src = (which ? a.v : a.k) + (long long)head * HD;
    const int r = lane / LPR, e8 = (lane % LPR) * 8;

    uint4 raw[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int i = p * RPL + r;
        raw[p] = make_uint4(0u, 0u, 0u, 0u);
        if (i >= lo && i < hi)
            raw[p] = *reinterpret_cast<const uint4*>(src + (long long)(row0 + (pos0 + i - first)) * a.row_stride + e8);
    }
    if (page < 0) {   // (the rows are on their way, whether or not they have one)
        if (lane == 0 && (pos0 >> c.page_shift) < c.max_pages) raise_error(c.err, HRA_DEVERR_PAGE_RANGE);
        return;
    }
    const int slot0 = pos0 & (c.page_size - 1);
    float* scale = c.scales + kv8_scale_at(c, page, which, head, slot0);
    uint8_t* dst = c.codes + kv8_code_at(c, page, which, head, slot0);
    const float before = lo > 0 ? *scale : 0.f;
    // bf16 bits without their sign order like the values; a NaN is ignored, and stays one as a code
    uint32_t top = 0u;
#pragma unroll
    for (int p = 0; p < PASSES; ++p)
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(raw[p].x & 0x7FFF7FFFu, raw[p].y & 0x7FFF7FFFu),
                                     __vmaxu2(raw[p].z & 0x7FFF7FFFu, raw[p].w & 0x7FFF7FFFu)));
    top = max(top & 0xFFFFu, top >> 16);
    if (__any_sync(0xffffffffu, top > 0x7F80u)) {
        float m = 0.f;
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            float f[8];
            unpack8(raw[p], f);
#pragma unroll
            for (int q = 0; q < 8; ++q) m = fmaxf(m, fabsf(f[q]));
        }
        top = __float_as_uint(m) >> 16;
    }
    top = min(__reduce_max_sync(0xffffffffu, top), 0x7F7Fu);   // infinities count as the largest bf16 and saturate
    const float m = __uint_as_float(top << 16);
    const float s = fmaxf(before, __uint_as_float(kv8_scale_bits(__float_as_uint(m))));
    const float inv = 1.0f / s;
    if (lo > 0 && s > before) {   // the block's earlier codes follow its scale
        const float ratio = before * inv;
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int i = p * RPL + r;
            if (i < lo) {
                uint2* at = reinterpret_cast<uint2*>(dst + i * HD + e8);
                const uint2 w = *at;
                float f[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const uint32_t byte = ((q < 4 ? w.x : w.y) >> (8 * (q & 3))) & 0xFFu;
                    f[q] = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
                }
                *at = to_e4m3x8(f, ratio);
            }
        }
    }
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int i = p * RPL + r;
        if (i >= lo && i < hi) {
            float f[8];
            unpack8(raw[p], f);
            *reinterpret_cast<uint2*>(dst + i * HD + e8) = to_e4m3x8(f, inv);
        }
    }
    __syncwarp();   // every lane has read `before`
    if (lane == 0 && s != before) *scale = s;
}

__global__ void kv8_lens_kernel(const int32_t* __restrict__ row_pos, const int32_t* __restrict__ last_row, int batch,
                                int32_t* kv_len, int32_t* one_each) {
    pdl_launch();
    pdl_wait();
    for (int b = threadIdx.x; b <= batch; b += blockDim.x) {
        if (b < batch) kv_len[b] = row_pos[last_row[b]] + 1;
        one_each[b] = b;
    }
}

}  // namespace

cudaError_t launch_kv8_lens(const int32_t* row_pos, const int32_t* last_row, int batch, int32_t* kv_len,
                            int32_t* one_each, cudaStream_t st) {
    HRA_LAUNCH(kv8_lens_kernel, dim3(1), dim3(256), 0, st, row_pos, last_row, batch, kv_len, one_each);
    return cudaGetLastError();
}

cudaError_t launch_kv8_append(const Kv8AppendArgs& a, cudaStream_t st) {
    const int units = kv8_max_blocks(a.max_new) * 2 * a.view.n_kv;
    const dim3 grid((unsigned)((units + 3) / 4), (unsigned)a.batch);
    if (a.view.head_dim == 128)
        HRA_LAUNCH(kv8_append_kernel<128>, grid, dim3(128), 0, st, a);
    else
        HRA_LAUNCH(kv8_append_kernel<64>, grid, dim3(128), 0, st, a);
    return cudaGetLastError();
}

}  // namespace hra
