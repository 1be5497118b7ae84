// kv8_attention.cu -- causal grouped-query attention over the paged 8-bit cache.
//
// Row i of the n new tokens of a sequence with L cached positions sits at position L - n + i and q head
// h attends positions 0 .. L - n + i of kv head h / G, G = n_q / n_kv:
//   s_j = scale * sum_d q_d Kc_jd ks_j,   o = sum_j 2^(s_j - m) Vc_j vs_j / sum_j 2^(s_j - m)
// with Kc, Vc the E4M3 codes' values and ks, vs their blocks' scales.  A row that sees no position
// gets 0.
//
// The scales never touch the codes: ks is uniform over a block of 16 keys and multiplies the block's
// scores, vs multiplies the block's probabilities.  So the codes go to the tensor cores as f16, which
// holds every E4M3 value exactly.
//   q       scaled by a power of two per row so that its largest element lies in [2^14, 2^15): bf16
//           values down to 2^-31 of the row's largest are exact in f16.
//   p       the weights 2^(s_j - m) vs_j as f16 relative to their own running maximum M, times
//           2^15: an 11-bit rounding (2^-11 relative) of weights down to 2^-29 of the largest, well below
//           the output's bf16 rounding of 2^-8.  The sum 2^(s_j - m) is kept in fp32 from the unrounded
//           values, with its own maximum m: a block whose V is zero or tiny still counts in it.
//
// A warp takes 16 keys (one block) at a time straight from global memory into fragments: the order of
// the dims inside a dot product and of the dims among the output rows is free, so it is chosen such
// that every lane's share of a block is a few whole 16-byte pieces that only this lane reads.
//   S = Q K^T   (m16n8k16): rows are up to 16 (position, head) pairs, lane (g, t) = (lane / 4, lane % 4)
//               holds 16-byte pieces 16 t and 64 + 16 t of keys g and g + 8;
//   O^T = V^T P^T: lane (g, t) holds dims 16 g .. 16 g + 15 of keys 2t, 2t + 1, 2t + 8, 2t + 9, and the
//               P^T fragment is the lane's own S accumulators.
// Each lane copies its pieces with cp.async into a private queue in shared memory: no barrier and
// no bank conflict stands between the copies and the arithmetic.
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>

#include "internal.h"

namespace hra {

namespace {

constexpr int kWarps = 4;
constexpr int kStages = 3;      // blocks of 16 keys in flight per warp
constexpr int kShortRows = 16;  // (position, head) rows of a kv head that fit this kernel's tile
constexpr int kSerialKeys = 2048;   // keys that a short sequence may walk alone among prompts
constexpr float kPScale = 15.f; // log2 of the largest p

__device__ __forceinline__ void cp_async_ca(uint32_t dst, const void* src, int bytes) {
    if (bytes == 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// two E4M3 codes (low 16 bits of w) -> two f16
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((unsigned short)w));
    return d;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float ex2(float x) { return exp2f(x); }

// Bytes of one lane's share of a block of 16 keys, and where its parts lie in a stage.
template <int HD>
struct Piece {
    static constexpr int KP = HD / 64;            // 16-byte pieces of each of the lane's two keys
    static constexpr int VB = HD / 8;             // bytes of each of the lane's four value rows
    static constexpr int OFF_V = 2 * KP * 512;    // [piece][lane][16]
    static constexpr int OFF_S = OFF_V + 4 * VB * 32;
    static constexpr int STAGE = OFF_S + 32 * 8;  // the block's two scales, one copy a lane
};

// One CTA = one (sequence, tile of query positions, kv head); its four warps take every fourth block
// of 16 keys and join their (m, l, M, O) through shared memory.  NG x 8 rows a tile.
template <int HD, int NG>
__global__ void __launch_bounds__(kWarps * 32, 3) kv8_attn_kernel(const Kv8AttnArgs a, int G, int QT, int max_rows) {
    pdl_launch();
    pdl_wait();
    using Pc = Piece<HD>;
    constexpr int KS = HD / 16;       // k steps of S
    constexpr int DT = HD / 16;       // 16-dim tiles of O^T
    constexpr int ROWS = 8 * NG;
    extern __shared__ __align__(16) uint8_t sm[];
    const Kv8View& c = a.view;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int tile = blockIdx.x, head = blockIdx.y, b = blockIdx.z;
    int row0, n;
    kv8_rows(a.cu, b, a.total_rows, row0, n);
    if (tile * QT >= n || n * G > max_rows) return;
    const long long room = (long long)c.max_pages << c.page_shift;
    int kv_len = a.kv_len[b];
    if (kv_len < 0 || kv_len > room) {
        if (threadIdx.x == 0) raise_error(c.err, HRA_DEVERR_POS_RANGE);
        kv_len = kv_len < 0 ? 0 : (int)room;
    }
    if (n > a.max_new && threadIdx.x == 0) raise_error(c.err, HRA_DEVERR_POS_RANGE);
    const int q_lo = tile * QT, q_n = min(QT, n - q_lo);
    const int keys = max(0, kv_len - n + q_lo + q_n);   // positions below the tile's last row's
    const int n_blk = (keys + kKv8Block - 1) / kKv8Block;

    // ---- q fragments: f16, each row scaled by a power of two
    uint32_t qa[KS][2 * NG];
    float q_unscale[NG];
    int limit[NG];             // keys below this one count for the row
#pragma unroll
    for (int x = 0; x < NG; ++x) {
        const int r = g + 8 * x, qi = r / G, hq = r - qi * G;
        const bool ok = qi < q_n;
        limit[x] = ok ? min(keys, kv_len - n + q_lo + qi + 1) : 0;
        const bf16* src = a.q + (long long)(row0 + q_lo + (ok ? qi : 0)) * a.row_stride + (long long)(head * G + hq) * HD;
        float f[HD / 64][16];
        float mx = 0.f;
#pragma unroll
        for (int h = 0; h < HD / 64; ++h) {
            uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
            if (ok) {
                u0 = *reinterpret_cast<const uint4*>(src + h * 64 + t4 * 16);
                u1 = *reinterpret_cast<const uint4*>(src + h * 64 + t4 * 16 + 8);
            }
            float lo[8], hi[8];
            unpack8(u0, lo);
            unpack8(u1, hi);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[h][e] = lo[e];
                f[h][8 + e] = hi[e];
                mx = fmaxf(mx, fmaxf(fabsf(lo[e]), fabsf(hi[e])));
            }
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // 2^(14 - floor(log2 mx)), its exponent kept inside fp32's normal range
        const int ex = min(254, max(14, (int)(__float_as_uint(mx) >> 23)));
        const float mul = __uint_as_float((uint32_t)(268 - ex) << 23);
        q_unscale[x] = __uint_as_float((uint32_t)max(1, ex - 14) << 23) * a.scale_log2;
#pragma unroll
        for (int h = 0; h < HD / 64; ++h)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                qa[h * 4 + q][x] = pack_h2(f[h][4 * q] * mul, f[h][4 * q + 1] * mul);
                qa[h * 4 + q][NG + x] = pack_h2(f[h][4 * q + 2] * mul, f[h][4 * q + 3] * mul);
            }
    }

    float o[NG][DT][4];
#pragma unroll
    for (int x = 0; x < NG; ++x)
#pragma unroll
        for (int d = 0; d < DT; ++d) o[x][d][0] = o[x][d][1] = o[x][d][2] = o[x][d][3] = 0.f;
    float m[NG], l[NG], M[NG];
#pragma unroll
    for (int x = 0; x < NG; ++x) {
        m[x] = M[x] = -INFINITY;
        l[x] = 0.f;
    }

    const uint32_t queue = smem_u32(sm) + warp * kStages * Pc::STAGE;
    // this lane's pieces of block `blk` into stage st; keys at or past `keys`, and blocks whose page is
    // not in the pool, are zero-filled and masked below
    bool bad_page = false;
    auto request = [&](int blk, int st) {
        const int pos0 = blk * kKv8Block;
        const int page = kv8_page_of(c, b, pos0);
        bad_page |= page < 0;
        const int slot0 = pos0 & (c.page_size - 1);
        const int pg = page < 0 ? 0 : page;
        const int left = page < 0 ? 0 : keys - pos0;          // keys of this block that count
        const uint8_t* kb = c.codes + kv8_code_at(c, pg, 0, head, slot0);
        const uint8_t* vb = c.codes + kv8_code_at(c, pg, 1, head, slot0);
        const uint32_t base = queue + st * Pc::STAGE;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int h = 0; h < Pc::KP; ++h)
                cp_async16(base + ((i * Pc::KP + h) * 32 + lane) * 16, kb + (g + 8 * i) * HD + h * 64 + t4 * 16,
                           g + 8 * i < left ? 16u : 0u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int key = 2 * t4 + (i & 1) + 8 * (i >> 1);
            const uint32_t dst = base + Pc::OFF_V + (i * 32 + lane) * Pc::VB;
            if (HD == 128) {
                cp_async16(dst, vb + key * HD + g * 16, key < left ? 16u : 0u);
            } else {
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(vb + key * HD + g * 8),
                             "r"(key < left ? 8 : 0)
                             : "memory");
            }
        }
        const uint32_t sc = base + Pc::OFF_S + lane * 8;
        cp_async_ca(sc, c.scales + kv8_scale_at(c, pg, 0, head, slot0), 4);
        cp_async_ca(sc + 4, c.scales + kv8_scale_at(c, pg, 1, head, slot0), 4);
    };

    // ---- the warp's blocks: warp, warp + 4, ...
    int ahead = warp;
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
        if (ahead < n_blk) request(ahead, s);
        cp_async_commit();
        ahead += kWarps;
    }
    int st = 0, st_in = kStages - 1;
    for (int blk = warp; blk < n_blk; blk += kWarps) {
        if (ahead < n_blk) request(ahead, st_in);
        cp_async_commit();
        ahead += kWarps;
        st_in = st_in + 1 == kStages ? 0 : st_in + 1;
        cp_async_wait<kStages - 1>();
        const uint8_t* sp = sm + warp * kStages * Pc::STAGE + st * Pc::STAGE;
        st = st + 1 == kStages ? 0 : st + 1;
        const float2 sc = *reinterpret_cast<const float2*>(sp + Pc::OFF_S + lane * 8);

        float s[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
            for (int h = 0; h < Pc::KP; ++h) {
                const uint4 w = *reinterpret_cast<const uint4*>(sp + ((i * Pc::KP + h) * 32 + lane) * 16);
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t b0 = e4m3x2_f16x2(ww[q] & 0xFFFFu), b1 = e4m3x2_f16x2(ww[q] >> 16);
                    if (NG == 1)
                        mma_f16(s[i], qa[h * 4 + q][0], 0u, qa[h * 4 + q][1], 0u, b0, b1);
                    else
                        mma_f16(s[i], qa[h * 4 + q][0], qa[h * 4 + q][NG - 1], qa[h * 4 + q][NG], qa[h * 4 + q][2 * NG - 1],
                                b0, b1);
                }
            }
        }
        // a page outside the pool: its keys are absent
        const bool there = kv8_page_of(c, b, blk * kKv8Block) >= 0;
        const uint32_t vbits = __float_as_uint(sc.y);
        const float ev = (float)((int)((vbits >> 23) & 255u) - 127);
        const float vm = __uint_as_float((vbits & 0x807FFFFFu) | 0x3F800000u);
        uint32_t pb[NG][2];
        float al[NG];
        bool moved = false;
#pragma unroll
        for (int x = 0; x < NG; ++x) {
            const float coef = q_unscale[x] * sc.x;
            float z[4];
            float mx = -INFINITY;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = blk * kKv8Block + (e >> 1) * 8 + 2 * t4 + (e & 1);
                z[e] = there && key < limit[x] ? s[e >> 1][2 * x + (e & 1)] * coef : -INFINITY;
                mx = fmaxf(mx, z[e]);
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float mn = fmaxf(m[x], mx), Mn = fmaxf(M[x], mx + ev);
            const float mr = mn == -INFINITY ? 0.f : mn, Mr = Mn == -INFINITY ? 0.f : Mn;
            l[x] *= ex2(m[x] - mr);
            al[x] = ex2(M[x] - Mr);
            moved |= al[x] != 1.f;
            m[x] = mn;
            M[x] = Mn;
            const float off = ev + kPScale - Mr;
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                l[x] += ex2(z[e] - mr);
                w[e] = ex2(z[e] + off) * vm;
            }
            pb[x][0] = pack_h2(w[0], w[1]);
            pb[x][1] = pack_h2(w[2], w[3]);
        }
        if (__any_sync(0xffffffffu, moved)) {   // O's columns are rows 2 t, 2 t + 1 (+ 8 x)
#pragma unroll
            for (int x = 0; x < NG; ++x) {
                const float a0 = __shfl_sync(0xffffffffu, al[x], 8 * t4), a1 = __shfl_sync(0xffffffffu, al[x], 8 * t4 + 4);
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    o[x][d][0] *= a0;
                    o[x][d][1] *= a1;
                    o[x][d][2] *= a0;
                    o[x][d][3] *= a1;
                }
            }
        }
        // O^T += V^T P^T: words of keys 2t and 2t + 1 interleave into pairs of one dim
        uint32_t vw[4][HD / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint8_t* at = sp + Pc::OFF_V + (i * 32 + lane) * Pc::VB;
            if (HD == 128) {
                const uint4 w = *reinterpret_cast<const uint4*>(at);
                vw[i][0] = w.x;
                vw[i][1] = w.y;
                vw[i][HD / 32 - 2] = w.z;
                vw[i][HD / 32 - 1] = w.w;
            } else {
                const uint2 w = *reinterpret_cast<const uint2*>(at);
                vw[i][0] = w.x;
                vw[i][1] = w.y;
            }
        }
#pragma unroll
        for (int j = 0; j < HD / 32; ++j) {
            const uint32_t p0 = __byte_perm(vw[0][j], vw[1][j], 0x5140), p1 = __byte_perm(vw[0][j], vw[1][j], 0x7362);
            const uint32_t p2 = __byte_perm(vw[2][j], vw[3][j], 0x5140), p3 = __byte_perm(vw[2][j], vw[3][j], 0x7362);
            const uint32_t a0 = e4m3x2_f16x2(p0 & 0xFFFFu), a1 = e4m3x2_f16x2(p0 >> 16);
            const uint32_t a2 = e4m3x2_f16x2(p2 & 0xFFFFu), a3 = e4m3x2_f16x2(p2 >> 16);
            const uint32_t c0 = e4m3x2_f16x2(p1 & 0xFFFFu), c1 = e4m3x2_f16x2(p1 >> 16);
            const uint32_t c2 = e4m3x2_f16x2(p3 & 0xFFFFu), c3 = e4m3x2_f16x2(p3 >> 16);
#pragma unroll
            for (int x = 0; x < NG; ++x) {
                mma_f16(o[x][2 * j], a0, a1, a2, a3, pb[x][0], pb[x][1]);
                mma_f16(o[x][2 * j + 1], c0, c1, c2, c3, pb[x][0], pb[x][1]);
            }
        }
    }
    cp_async_wait<0>();
    if (bad_page) raise_error(c.err, HRA_DEVERR_PAGE_RANGE);
    __syncthreads();   // the queues are free: the warps' results go over them

    // ---- join the four warps: [warp][row][HD] sums and [warp][row] (m, l, M)
    float* s_o = reinterpret_cast<float*>(sm);
    float* s_m = s_o + kWarps * ROWS * HD;
#pragma unroll
    for (int x = 0; x < NG; ++x) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        if (t4 == 0) {
            float* at = s_m + (warp * ROWS + g + 8 * x) * 3;
            at[0] = m[x];
            at[1] = l[x];
            at[2] = M[x];
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            // rows 2 t, 2 t + 1 (+ 8 x); dims g * (HD / 8) + 2 d, + 1
            float* at = s_o + (warp * ROWS + 2 * t4 + 8 * x) * HD + g * (HD / 8) + 2 * d;
            *reinterpret_cast<float2*>(at) = make_float2(o[x][d][0], o[x][d][2]);
            *reinterpret_cast<float2*>(at + HD) = make_float2(o[x][d][1], o[x][d][3]);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < q_n * G * (HD / 2); i += kWarps * 32) {
        const int r = i / (HD / 2), d = (i - r * (HD / 2)) * 2;
        const int qi = r / G, hq = r - qi * G;
        float mm = -INFINITY, MM = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            mm = fmaxf(mm, s_m[(w * ROWS + r) * 3]);
            MM = fmaxf(MM, s_m[(w * ROWS + r) * 3 + 2]);
        }
        const float mr = mm == -INFINITY ? 0.f : mm, Mr = MM == -INFINITY ? 0.f : MM;
        float L = 0.f, x0 = 0.f, x1 = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float* at = s_m + (w * ROWS + r) * 3;
            L += at[1] * ex2(at[0] - mr);
            const float f = ex2(at[2] - Mr);
            const float2 ov = *reinterpret_cast<const float2*>(s_o + (w * ROWS + r) * HD + d);
            x0 += ov.x * f;
            x1 += ov.y * f;
        }
        // L is 0 for a row that saw no key, and NaN when a score was
        const float f = L == 0.f ? 0.f : ex2(Mr - mr) / L;
        x0 = x0 * 0x1p-15f * f;
        x1 = x1 * 0x1p-15f * f;
        bf16* dst = a.out + ((long long)(row0 + q_lo + qi) * a.nq + head * G + hq) * HD + d;
        *reinterpret_cast<uint32_t*>(dst) = pack_bf2(x0, x1);
    }
}

template <int HD, int NG>
cudaError_t launch_ng(const Kv8AttnArgs& a, int G, int QT, int tiles, int max_rows, cudaStream_t st) {
    constexpr int queue = kWarps * kStages * Piece<HD>::STAGE;
    constexpr int join = kWarps * 8 * NG * (HD + 3) * 4;
    constexpr int smem = queue > join ? queue : join;
    static bool configured[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(kv8_attn_kernel<HD, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    const dim3 grid((unsigned)tiles, (unsigned)a.view.n_kv, (unsigned)a.batch);
    HRA_LAUNCH((kv8_attn_kernel<HD, NG>), grid, dim3(kWarps * 32), smem, st, a, G, QT, max_rows);
    return cudaGetLastError();
}

}  // namespace

size_t kv8_attention_scratch_bytes(const Kv8View& c, int batch, int total_rows, int nq, int max_new, int max_len) {
    const int G = nq / c.n_kv;
    if ((long long)G * max_new <= kShortRows) return 0;
    return kv8_prompt_scratch_bytes(batch, total_rows, G);
}

cudaError_t launch_kv8_attention(const Kv8AttnArgs& a, cudaStream_t st) {
    const int G = a.nq / a.view.n_kv;
    const bool prompts = (long long)G * a.max_new > kShortRows && kv8_prompt_supported(a.view);
    const int long_keys = a.max_len > kSerialKeys;
    // short sequences go with the prompts unless they may hold many keys
    const int short_rows = prompts && !long_keys ? 0 : kShortRows;
    if (prompts) {
        cudaError_t e = launch_kv8_prompt(a, short_rows, st);
        if (e != cudaSuccess || short_rows == 0 || (long long)a.batch * a.max_new == a.total_rows) return e;
    }
    // one n = 8 column group while the rows of a tile fit it, else two
    const int rows = prompts ? kShortRows : 1 << 30;
    const int ng = (long long)G * a.max_new <= 8 ? 1 : 2;
    const int QT = 8 * ng / G;
    const int tiles = prompts ? 1 : (a.max_new + QT - 1) / QT;
    if (a.view.head_dim == 128)
        return ng == 1 ? launch_ng<128, 1>(a, G, QT, tiles, rows, st) : launch_ng<128, 2>(a, G, QT, tiles, rows, st);
    return ng == 1 ? launch_ng<64, 1>(a, G, QT, tiles, rows, st) : launch_ng<64, 2>(a, G, QT, tiles, rows, st);
}

}  // namespace hra
