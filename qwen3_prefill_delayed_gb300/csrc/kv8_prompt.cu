// kv8_prompt.cu -- prompt and chunk attention over the paged 8-bit cache on the tensor cores.
//
// The formulas and the treatment of the scales are those of kv8_attention.cu.  Here an item is one
// kv head and QT = 128 / G query positions of a sequence (128 rows (position, head), row r = (r / G, r % G))
// over all their keys, in tiles of 64 keys:
//   S = Q K^T    kind::f8f6f4 on the codes as they lie in the pages.  Q enters as the sum of two E4M3
//                matrices under a power of two s per row: hi = e4m3(q / s), lo = e4m3(q / s - hi).  A bf16 value
//                has 8 significant bits and each E4M3 value 4, so hi + lo is q / s exactly where lo's last bit is
//                2^-9 or more, from q / s = 2^-2 on.  The row's largest has q / s in (224, 448]: elements below 2^-2 / 224 =
//                2^-9.8 of it are off by at most half a subnormal step, 2^-10 / 224 = 2^-17.8 of it.  Two MMAs
//                at twice the f16 rate cost what one f16 MMA would, and no K is converted.
//   O += P V     kind::f16: P, the probabilities times their blocks' V scales in f16 relative to a lazy
//                running maximum M (it moves when it is exceeded by 2^4; 2^11 is the unit, so weights stay
//                below 2^15), from tensor memory over the columns of S; V converted to f16 (exact).
// Measured on GB300 (one thread issuing, SM clocks an instruction): 128 x N x 32 bytes takes 64 for N = 128 and
// 53-63 for any smaller N.  128-key tiles would use the tensor cores a quarter better, but tensor memory then has room
// for one S only; with 64 keys S(g + 1) is computed while the softmax works on S(g) (8 long prompts: 277 us with one S of
// 128 keys, 238 with two of 64).
//
// 320 threads, two CTAs an SM (256 tensor memory columns and 101 KB each), so that one CTA's softmax runs
// under the other's MMAs:
//   warp 0     TMA of K (one 16-key box a lane, page by page) into four stages, and the blocks' scales;
//   warp 1     tensor memory, and one thread that issues the MMAs;
//   warps 2-5  softmax, one row a thread, S read twice from tensor memory (maximum, then weights), O rescaled
//              when M moves, and the output;
//   warps 6-9  V: codes from global memory in registers, two tiles ahead, to f16 in shared memory (keys that
//              do not count as zeros, so stale slots never reach a product); and the items' Q.
// What bounds it: the chain S -> softmax -> PV of a tile, about 2800 clocks with two CTAs at work, in which the tensor
// pipe is 35% busy and 53% of the issue slots are taken.  No part carries it alone (chunks after many positions, then 338 us,
// with work left out: the exponentials and packing 0, half of S's MMAs 8%, V's conversion 9%, all but one of PV's MMAs
// 4%, the maxima 2%): the MMAs and the shared memory of two CTAs queue behind one another.  Two groups of softmax warps
// that take the tiles in turn (448 threads at 72 registers) took 410 us against 353, a third V buffer 349 against 338.
// The items come from a list built on the device (kv8_schedule_kernel).  Many items: most key tiles first, and CTA c
// takes entries in snake order.  Few long ones (prompt chunks after many cached positions): the tiles of all items
// form a line of which every CTA takes an equal share; parts of an item go to scratch as fp32 sums with their
// (m, l, M) and a second kernel joins them in order.  2 rows of 500-1021 tokens after 9-16 thousand: 376 items on 304
// CTAs took two turns of the longest, 405 us; equal shares 371.

#include <algorithm>
#include <math.h>

#include "kv8_device.cuh"

namespace hra {

namespace {

constexpr int kThreads = 320;
constexpr int TROWS = 128;
constexpr int TK = 64;             // keys a tile
constexpr int NB = TK / kKv8Block; // blocks a tile
constexpr float kUnit = 11.f;      // log2 of the weight of the reference maximum
// Keys from which items count as long (see prompt_shares).  8 kv heads of 128, 4 q heads each, in a graph, equal shares / whole
// items: 1 row of 128 tokens after 2000 positions 36 / 42 us, after 16000 64 / 245; 2 rows of 500 and 1021 after 8000 210 / 224,
// after 16000 362 / 424, but after 4000 137 / 125; 4 of 512 after 8000 295 / 312; from 8 of 1024 on equal after 4000 (617 / 618),
// shares slower below (306 / 256 after 1000).  2 of 600 are as many items as CTAs, and whole ones better at any length.
constexpr int kSharesFrom = 2048;
constexpr float kSlack = 4.f;      // how far a maximum may pass the reference before it moves

struct PromptRec {   // 32 bytes: one (query tile, sequence) pair
    int b, row0, n, q_lo, kv_len, keys;
    long long before;   // equal shares: tiles of the items of the pairs before
};
__host__ __device__ __forceinline__ int key_tiles(int keys) {   // an item without keys has one empty tile: its rows get 0
    return keys > 0 ? (keys + TK - 1) / TK : 1;
}
// Parts of split items, as for single tokens: CTA c has slots 2 c (the item that its share begins in) and 2 c + 1 (the
// one it ends in); a slot is [TROWS][HD] sums, then m, l and M of the rows.
struct PromptDesc {   // the item whose first part is slot 2 c + 1, and the last CTA that has a part of it
    int row0, n, q_lo, head, last;   // row0 < 0: none
    int b, kv_len, keys;             // as in the pair's record
};
template <int HD>
struct PromptSlot {
    static constexpr int FLOATS = TROWS * (HD + 3);
};
constexpr int kRecWords = 8;

constexpr int NK = 4;              // K stages
constexpr int NSC = 8;             // tiles whose scales are held
constexpr int NQS = 4;             // items whose q scales are held

template <int HD>
struct Cfg {
    static constexpr int QB = TROWS * HD;               // bytes of Q hi (and of lo)
    static constexpr int KB = TK * HD;                  // one K stage
    static constexpr int VB = TK * HD * 2;              // one of two stages of V as f16
    static constexpr int OFF_K = 2 * QB;
    static constexpr int OFF_V = OFF_K + NK * KB;
    static constexpr int OFF_BAR = OFF_V + 2 * VB;
    static constexpr int OFF_SC = OFF_BAR + 320;             // [NSC][3][NB]: K scale, V scale's exponent and factor
    static constexpr int OFF_QS = OFF_SC + NSC * 3 * NB * 4; // [NQS][TROWS] q scales
    static constexpr int OFF_TH = OFF_QS + NQS * TROWS * 4;  // [NSC] whether a tile's blocks are all there
    static constexpr int SMEM = OFF_TH + NSC * 4;
    static constexpr int ALLOC = SMEM + 1024;           // the base is aligned up to 1024 bytes
    // tile g: K stage g % NK, S / P / V buffer g & 1, scales g % NSC; item it: q scales it % NQS
    static constexpr int B_QF = 0, B_QE = 1, B_KF = 2, B_KE = B_KF + NK, B_SF = B_KE + NK, B_PF = B_SF + 2, B_VF = B_PF + 2,
                         B_PV = B_VF + 2, B_OF = B_PV + 2, B_IDLE = B_OF + 1, B_SC = B_IDLE + 1, B_QS = B_SC + NSC,
                         NBARS = B_QS + NQS;
    static_assert(NBARS * 8 + 16 <= 320, "barrier area");
    static_assert(ALLOC <= 115712, "two CTAs an SM");
};

struct PromptArgs {
    Kv8View view;
    const bf16* q;
    long long row_stride;
    bf16* out;
    const int32_t* list;    // [0] = pairs, [2..3] all items' tiles, records from word 8 on
    PromptDesc* desc;       // equal shares (null: snake order)
    float* parts;
    float scale_log2;
    int nq, G, QT;
    int v8;                 // out 32-byte aligned
};

// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long d;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tmov.b64 c, {%5, %6};\n\t"
        "fma.rn.f32x2 %0, a, b, c;\n\t}"
        : "=l"(d)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return make_float2(__uint_as_float((uint32_t)d), __uint_as_float((uint32_t)(d >> 32)));
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long d;
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tadd.rn.f32x2 %0, a, b;\n\t}"
        : "=l"(d)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return make_float2(__uint_as_float((uint32_t)d), __uint_as_float((uint32_t)(d >> 32)));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long d;
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\tmul.rn.f32x2 %0, a, b;\n\t}"
        : "=l"(d)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return make_float2(__uint_as_float((uint32_t)d), __uint_as_float((uint32_t)(d >> 32)));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// D[tmem] (+)= A[tmem, f16 pairs] * B[smem]
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
}
// 32 lanes x 16 columns, no wait
__device__ __forceinline__ void tmem_st16_async(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
// the maxima of columns 0 .. 15 and 16 .. 31 of each lane's row (the columns themselves are dropped)
__device__ __forceinline__ void tmem_max32(uint32_t taddr, float& top0, float& top1) {
    float v[16], w[16];
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, %32, [%34];\n\t"
        "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 "
        "{%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, %33, [%35];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
          "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]),
          "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(w[0]), "=f"(w[1]), "=f"(w[2]), "=f"(w[3]), "=f"(w[4]), "=f"(w[5]),
          "=f"(w[6]), "=f"(w[7]), "=f"(w[8]), "=f"(w[9]), "=f"(w[10]), "=f"(w[11]),
          "=f"(w[12]), "=f"(w[13]), "=f"(w[14]), "=f"(w[15]),
          "=f"(top0), "=f"(top1)
        : "r"(taddr), "r"(taddr + 16));
}
// Dims dim .. dim + n - 1 of row `row` of an item's tile, written to out, hold a NaN: see kv8_row_again.
__device__ __noinline__ void look_again(const PromptArgs& p, const PromptRec& r, int head, int row, int dim, int n, bf16* out) {
    const int qi = row / p.G, hq = row - qi * p.G;
    const bf16* q = p.q + (long long)(r.row0 + r.q_lo + qi) * p.row_stride + (long long)(head * p.G + hq) * p.view.head_dim;
    kv8_row_again(p.view, q, r.b, head, r.kv_len - r.n + r.q_lo + qi + 1, r.keys, dim, n, p.scale_log2, out);
}
__device__ __forceinline__ int snake(int k) {
    return k * (int)gridDim.x + ((k & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
}

// One row's tile of S, 32 columns at a time: unrolled as straight code, the weights and masks make the softmax warps wait
// for instructions (a tile of it took 4600 clocks instead of 2400).  Where not every key of the tile counts, the keys below
// `limit` of blocks that are there (scale >= 0) do.
// mx: the maximum of s; Mx: the maximum of s + log2 of the block's V scale.  The loads themselves take the maximum of a
// block's 16 scores (chunks after many positions: 353 us by max instructions, 339 so; holding the scores for the weights
// meanwhile spills, 494).
__device__ __forceinline__ void max_pass_whole(uint32_t lS, const float* ks, float q_unscale, float& mx, float& Mx) {
#pragma unroll
    for (int ch = 0; ch < TK / 32; ++ch) {
        float top0, top1;
        const float2 k2 = *reinterpret_cast<const float2*>(ks + 2 * ch), e2 = *reinterpret_cast<const float2*>(ks + NB + 2 * ch);
        tmem_max32(lS + 32 * ch, top0, top1);
        const float z0 = top0 * (q_unscale * k2.x), z1 = top1 * (q_unscale * k2.y);
        mx = max3(mx, z0, z1);
        Mx = max3(Mx, z0 + e2.x, z1 + e2.y);
    }
}
__device__ __forceinline__ void max_pass_masked(uint32_t lS, const float* ks, float q_unscale, int limit, float& mx,
                                                float& Mx) {
#pragma unroll 1
    for (int ch = 0; ch < TK / 32; ++ch) {
        float a[32];
        tmem_ld32(lS + 32 * ch, a);
        const float2 k2 = *reinterpret_cast<const float2*>(ks + 2 * ch), e2 = *reinterpret_cast<const float2*>(ks + NB + 2 * ch);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float k = h ? k2.y : k2.x, ev = h ? e2.y : e2.x;
            const int n = k >= 0.f ? limit - 32 * ch - 16 * h : 0;
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (e >= n) a[16 * h + e] = -INFINITY;
            float top[2] = {fmaxf(a[16 * h], a[16 * h + 1]), fmaxf(a[16 * h + 2], a[16 * h + 3])};
#pragma unroll
            for (int e = 4; e < 16; e += 2) top[(e >> 1) & 1] = max3(top[(e >> 1) & 1], a[16 * h + e], a[16 * h + e + 1]);
            const float bm = fmaxf(top[0], top[1]);
            const float z = bm == -INFINITY ? bm : bm * (q_unscale * k);
            mx = fmaxf(mx, z);
            Mx = fmaxf(Mx, z + ev);
        }
    }
}
// The weights: l's terms 2^(s - mr) are returned summed; times the block's V scale and 2^(mr - Mr + 11)
// (`up` its exponent) they go as f16 to columns 16 ch, which this row has read.
template <bool MASK>
__device__ __forceinline__ float weight_pass(uint32_t lS, const float* ks, float q_unscale, int limit, float mr,
                                             float up) {
    float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    const float2 neg = make_float2(-mr, -mr);
#pragma unroll 1
    for (int ch = 0; ch < TK / 32; ++ch) {
        float a[32];
        tmem_ld32(lS + 32 * ch, a);
        const float2 k2 = *reinterpret_cast<const float2*>(ks + 2 * ch), e2 = *reinterpret_cast<const float2*>(ks + NB + 2 * ch),
                     m2 = *reinterpret_cast<const float2*>(ks + 2 * NB + 2 * ch);
        uint32_t w[16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float k = h ? k2.y : k2.x, ev = h ? e2.y : e2.x;
            const float coef = q_unscale * k;
            const float f = ex2(fminf(up + ev, 126.f)) * (h ? m2.y : m2.x);
            const int n = MASK ? (k >= 0.f ? limit - 32 * ch - 16 * h : 0) : 16;
            const float2 coef2 = make_float2(coef, coef), f2 = make_float2(f, f);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                const float2 z = fma2(make_float2(a[16 * h + e], a[16 * h + e + 1]), coef2, neg);
                float2 x = make_float2(ex2(z.x), ex2(z.y));
                if (MASK) {
                    if (e >= n) x.x = 0.f;
                    if (e + 1 >= n) x.y = 0.f;
                }
                ls[(e >> 1) & 1] = add2(ls[(e >> 1) & 1], x);
                const float2 y = mul2(x, f2);
                w[8 * h + e / 2] = pack_h2(y.x, y.y);
            }
        }
        tmem_st16_async(lS + 16 * ch, w);
    }
    return (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
}

// One CTA.  The non-empty (query tile, sequence) pairs: by a counting sort, most key tiles first, or, for equal shares,
// in the order of the sequences with the tiles before each (the shares' borders decide where sums are split, so the
// order must not depend on which thread comes first).  A thread a sequence counts its tiles, then a thread a pair
// finds its sequence in their running sum: the time follows the tiles there are, not batch times the longest.
constexpr int kBins = 1024;
__global__ void __launch_bounds__(1024) kv8_schedule_kernel(const Kv8AttnArgs a, int G, int QT, int short_rows, int shares,
                                                            int most, int32_t* __restrict__ list) {
    pdl_launch();
    pdl_wait();
    __shared__ int hist[kBins];
    __shared__ int at_s[1025], row0_s[1024], n_s[1024], len_s[1024];
    __shared__ int total;
    const int tid = threadIdx.x;
    for (int i = tid; i < kBins; i += blockDim.x) hist[i] = 0;
    const long long room = (long long)a.view.max_pages << a.view.page_shift;
    // Sequences b0 .. b0 + 1023, after `count` pairs: their pairs, and at_s = the pairs before each.  Rows beyond
    // max_new are left out: the first n of a sequence with n fewer positions are what they are.
    auto chunk = [&](int b0, int count, bool report) {
        const int b = b0 + tid;
        int row0 = 0, n = 0, len = 0;
        if (b < a.batch) {
            kv8_rows(a.cu, b, a.total_rows, row0, n);
            if (n > 0) {
                const int held = a.kv_len[b];
                len = held < 0 ? 0 : (int)min(room, (long long)held);
                const int over = max(0, n - a.max_new);
                if (report && n > short_rows / G && (len != held || over)) raise_error(a.view.err, HRA_DEVERR_POS_RANGE);
                if (n <= short_rows / G) n = 0;
                else n -= over;
                len -= over;
            }
        }
        long long all;
        const long long at = block_scan((long long)((n + QT - 1) / QT), all);
        const int left = most - count;   // enough for rows that no two sequences share
        if (report && tid == 0 && all > left) raise_error(a.view.err, HRA_DEVERR_POS_RANGE);
        at_s[tid] = (int)min((long long)left, at);
        row0_s[tid] = row0;
        n_s[tid] = n;
        len_s[tid] = len;
        if (tid == 0) at_s[1024] = (int)min((long long)left, all);
        __syncthreads();
        return at_s[1024];
    };
    auto pair = [&](int p, int b0, PromptRec& r) {   // pair p of the chunk
        int lo = 0, hi = min(1024, a.batch - b0);     // the last sequence with at_s <= p that has a tile
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (at_s[mid] <= p) lo = mid;
            else hi = mid;
        }
        r.b = b0 + lo;
        r.row0 = row0_s[lo];
        r.n = n_s[lo];
        r.q_lo = (p - at_s[lo]) * QT;
        r.kv_len = len_s[lo];
        r.keys = max(0, r.kv_len - r.n + min(r.n, r.q_lo + QT));
        return kBins - 1 - min(kBins - 1, (r.keys + TK - 1) / TK);
    };
    auto put = [&](int i, const PromptRec& r, long long before) {
        int4* to = reinterpret_cast<int4*>(list + kRecWords * (1 + (long long)i));
        to[0] = make_int4(r.b, r.row0, r.n, r.q_lo);
        to[1] = make_int4(r.kv_len, r.keys, (int)(before & 0xFFFFFFFFll), (int)(before >> 32));
    };
    PromptRec r;
    int count = 0;
    if (shares) {
        long long before = 0;
        for (int b0 = 0; b0 < a.batch; b0 += 1024) {
            const int here = chunk(b0, count, true);
            for (int p0 = 0; p0 < here; p0 += 1024) {
                const bool in = p0 + tid < here;
                if (in) pair(p0 + tid, b0, r);
                long long units;
                const long long at = block_scan((long long)(in ? key_tiles(r.keys) : 0), units);
                if (in) put(count + p0 + tid, r, before + a.view.n_kv * at);
                before += a.view.n_kv * units;
            }
            count += here;
        }
        if (tid == 0) {
            list[0] = count;
            *reinterpret_cast<long long*>(list + 2) = before;
        }
        return;
    }
    for (int b0 = 0; b0 < a.batch; b0 += 1024) {
        const int here = chunk(b0, count, true);
        for (int p = tid; p < here; p += 1024) atomicAdd(&hist[pair(p, b0, r)], 1);
        count += here;
        __syncthreads();
    }
    if (tid < 32) {
        constexpr int per = kBins / 32;
        int s = 0;
        for (int i = 0; i < per; ++i) s += hist[tid * per + i];
        int incl = s;
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (tid >= o) incl += v;
        }
        int run = incl - s;
        for (int i = 0; i < per; ++i) {
            const int h = hist[tid * per + i];
            hist[tid * per + i] = run;
            run += h;
        }
        if (tid == 31) total = incl;
    }
    __syncthreads();
    count = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 1024) {
        const int here = a.batch <= 1024 ? at_s[1024] : chunk(b0, count, false);
        for (int p = tid; p < here; p += 1024) {
            const int bin = pair(p, b0, r);
            put(atomicAdd(&hist[bin], 1), r, 0);
        }
        count += here;
        __syncthreads();
    }
    if (tid == 0) list[0] = total;
}

// The outputs of the items that this CTA did alone once more, a thread 32 dims of a row.  first: equal shares' first item, its
// first tile, the tiles of the share.
template <int HD>
__device__ __noinline__ void outputs_again(const PromptArgs& p, const int* first) {
    const bool shares = p.desc != nullptr;
    const int n_items = p.list[0] * p.view.n_kv;
    int left = shares ? first[2] : 0;
    for (int k = 0;; ++k) {
        const int i = shares ? first[0] + k : snake(k);
        if (i >= n_items || (shares && left == 0)) return;
        const int32_t* rec = p.list + kRecWords * (1 + (long long)(i / p.view.n_kv));
        const PromptRec r{rec[0], rec[1], rec[2], rec[3], rec[4], rec[5], 0};
        const int head = i % p.view.n_kv;
        if (shares) {   // not the parts: they are looked at where they are joined
            const int from = k == 0 ? first[1] : 0, all = key_tiles(r.keys), n = min(left, all - from);
            left -= n;
            if (n < all) continue;
        }
        for (int x = threadIdx.x; x < TROWS * (HD / 32); x += kThreads) {
            const int row = x / (HD / 32), dim = x % (HD / 32) * 32, qi = row / p.G;
            if (qi >= p.QT || r.q_lo + qi >= r.n) continue;
            bf16* dst = p.out + ((long long)(r.row0 + r.q_lo + qi) * p.nq + head * p.G + row - qi * p.G) * HD + dim;
            bool nan = false;
            for (int e = 0; e < 32; ++e) nan |= __hisnan(dst[e]);
            if (nan) look_again(p, r, head, row, dim, 32, dst);
        }
    }
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 2) kv8_prompt_kernel(const __grid_constant__ CUtensorMap tmK,
                                                                 const __grid_constant__ PromptArgs p) {
    using C = Cfg<HD>;
    pdl_launch();
    pdl_wait();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint32_t* slots = reinterpret_cast<uint32_t*>(bars + C::NBARS);   // tmem, abort, K tiles requested
    volatile int* abort_flag = reinterpret_cast<volatile int*>(slots + 1);
    volatile int* issued = reinterpret_cast<volatile int*>(slots + 2);
    float* sc = reinterpret_cast<float*>(smem + C::OFF_SC);
    float* qs = reinterpret_cast<float*>(smem + C::OFF_QS);
    __shared__ int nan_out_s;    // a row of an item that this CTA did alone has a NaN
    volatile int* nan_out = &nan_out_s;   // (looked at behind the items: a call inside them costs 6-12 %, 2 % so)
    __shared__ int first_s[3];   // equal shares: the first item, its first tile, the tiles of the share
    volatile int* there = reinterpret_cast<volatile int*>(smem + C::OFF_TH);
    auto bar = [&](int i) { return smem_u32(bars + i); };
    const Kv8View& c = p.view;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_items = p.list[0] * c.n_kv;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NBARS; ++i) {
            const bool four = i == C::B_QF || (i >= C::B_PF && i < C::B_PV) || i == C::B_OF || i >= C::B_QS;
            mbar_init(bar(i), four ? 4 : 1);
        }
        *abort_flag = 0;
        *issued = 0;
        *nan_out = 0;
        if (p.desc != nullptr) {
            const long long all = *reinterpret_cast<const long long*>(p.list + 2);
            const long long share = (all + gridDim.x - 1) / gridDim.x, u = blockIdx.x * share;
            p.desc[blockIdx.x].row0 = -1;
            first_s[0] = first_s[1] = 0;
            first_s[2] = (int)max(0LL, min(share, all - u));
            if (u < all) {
                int lo = 0, hi = p.list[0];   // the last pair with before <= u
                auto before = [&](int i) {
                    return *reinterpret_cast<const long long*>(p.list + kRecWords * (1 + (long long)i) + 6);
                };
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (before(mid) <= u) lo = mid;
                    else hi = mid;
                }
                const int n = key_tiles(p.list[kRecWords * (1 + (long long)lo) + 5]);
                const long long at = u - before(lo);
                first_s[0] = lo * c.n_kv + (int)(at / n);
                first_s[1] = (int)(at % n);
            }
        }
        mbar_fence_init();
        tma_prefetch_map(&tmK);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(slots), 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tS = slots[0], tO = tS + 2 * TK;   // two S buffers, then O
    // Items k = 0, 1, ... of this CTA; the next one's record is on its way while one is worked on.  Every role calls
    // item(0), item(1), ... until there is none.
    const bool shares = p.desc != nullptr;
    int left = shares ? first_s[2] : 0;   // tiles of the share
    int4 next_x = make_int4(0, 0, 0, 0), next_y = next_x;
    auto index = [&](int k) { return shares ? first_s[0] + k : snake(k); };
    auto fetch = [&](int k) {
        const int i = index(k);
        if (i < n_items) {
            const int4* at = reinterpret_cast<const int4*>(p.list + kRecWords * (1 + (long long)(i / c.n_kv)));
            next_x = at[0];
            next_y = at[1];
        }
    };
    int t_first = 0, t_all = 0;                         // this item's tiles [t_first, t_first + count) of t_all
    auto item = [&](int k, PromptRec& r, int& head) {   // its count, 0 when there is none
        const int i = index(k);
        if (i >= n_items || (shares && left == 0)) return 0;
        head = i % c.n_kv;
        r.b = next_x.x;
        r.row0 = next_x.y;
        r.n = next_x.z;
        r.q_lo = next_x.w;
        r.kv_len = next_y.x;
        r.keys = next_y.y;
        fetch(k + 1);
        t_all = key_tiles(r.keys);
        if (!shares) return t_all;
        t_first = k == 0 ? first_s[1] : 0;
        const int n = min(left, t_all - t_first);
        left -= n;
        return n;
    };
    fetch(0);
    PromptRec r;
    int head;
    bool ok = true;

    if (warp == 0) {
        // ---- K tiles and scales: lanes 0-3 block `lane` of K, lanes 4-7 block lane - 4 of V (its scale only)
        const int blk = lane & (NB - 1), which = (lane / NB) & 1;
        int g = 0;
        for (int k = 0; ok; ++k) {
            const int n_kt = item(k, r, head);
            if (n_kt == 0) break;
            auto page_of = [&](int t) {
                const int pos = (t_first + t) * TK + blk * kKv8Block;
                return lane < 2 * NB && pos < r.keys ? kv8_page_of(c, r.b, pos) : -1;
            };
            auto scale_of = [&](int t, int page) {   // -1: the block's keys are absent
                const int pos = (t_first + t) * TK + blk * kKv8Block;
                return page < 0 ? -1.f : c.scales[kv8_scale_at(c, page, which, head, pos & (c.page_size - 1))];
            };
            int page = page_of(0), page1 = n_kt > 1 ? page_of(1) : -1;
            float s = scale_of(0, page);
            for (int t = 0; t < n_kt && ok; ++t, ++g) {
                // a tile ahead: its scale; two ahead: its page
                const float s1 = t + 1 < n_kt ? scale_of(t + 1, page1) : 0.f;
                const int page2 = t + 2 < n_kt ? page_of(t + 2) : -1;
                const int st = g % NK;
                if (g >= NK) ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_KE + st), (uint32_t)(g / NK - 1) & 1u, abort_flag));
                if (!ok) break;
                const bool want = lane < NB && page >= 0;
                const int pos = (t_first + t) * TK + blk * kKv8Block;
                if (lane < NB && pos < r.keys && page < 0) raise_error(c.err, HRA_DEVERR_PAGE_RANGE);
                if (lane < NB) {
                    sc[(g % NSC) * 3 * NB + blk] = s;
                } else if (lane < 2 * NB) {
                    sc[((g % NSC) * 3 + 1) * NB + blk] = exponent_of(s);
                    sc[((g % NSC) * 3 + 2) * NB + blk] = mantissa_of(s);
                }
                const int boxes = __popc(__ballot_sync(0xffffffffu, want));
                if (lane == 0) there[g % NSC] = boxes == NB;
                __syncwarp();   // the scales are written
                if (lane == 0) {
                    *issued = g + 1;
                    mbar_arrive(bar(C::B_SC + g % NSC));
                    if (boxes) mbar_expect_tx(bar(C::B_KF + st), (uint32_t)(boxes * kKv8Block * HD));
                    else mbar_arrive(bar(C::B_KF + st));
                }
                __syncwarp();
                if (want) {
                    const long long row = kv8_code_at(c, page, 0, head, pos & (c.page_size - 1)) / HD;
                    tma_load_2d(smem_u32(smem + C::OFF_K + st * C::KB + blk * kKv8Block * HD), &tmK, bar(C::B_KF + st), 0,
                                (int)row);
                }
                page = page1;
                page1 = page2;
                s = s1;
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc_s = idesc_e4m3_f32(TROWS, TK);
            // A and B f16 (type code 0), D fp32, B transposed (MN-major), N = HD
            constexpr uint32_t idesc_o = (1u << 4) | (1u << 16) | ((uint32_t)(HD >> 3) << 17) | ((uint32_t)(TROWS >> 4) << 24);
            const uint32_t sQ = smem_u32(smem), sK = smem_u32(smem + C::OFF_K);
            const uint64_t q_desc = HD == 128 ? sdesc_sw128(sQ) : sdesc_sw64(sQ);
            const uint64_t k_desc = HD == 128 ? sdesc_sw128(sK) : sdesc_sw64(sK);
            const uint64_t v_desc = sdesc_sw128_mn(smem_u32(smem + C::OFF_V), TK * 128, 1024);
            int g = 0, it = 0;
            for (int k = 0; ok; ++k) {
                const int n_kt = item(k, r, head);
                if (n_kt == 0) break;
                // S(x) into buffer x & 1, over P(x - 2): its PV is done
                auto issue_s = [&](int x) {
                    const int st = x % NK;
                    if (!mbar_wait(bar(C::B_KF + st), (uint32_t)(x / NK) & 1u, abort_flag) ||
                        (x >= 2 && !mbar_wait(bar(C::B_PV + (x & 1)), (uint32_t)((x >> 1) - 1) & 1u, abort_flag)))
                        return false;
                    tc_fence_after();
                    const uint64_t kd = k_desc + (uint64_t)(st * (C::KB >> 4));
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int kk = 0; kk < HD / 32; ++kk)
                            tc_mma_f8(tS + (x & 1) * TK, q_desc + (uint64_t)(part * (C::QB >> 4) + 2 * kk), kd + 2ull * kk, idesc_s,
                                      part + kk > 0 ? 1u : 0u);
                    tc_commit(bar(C::B_SF + (x & 1)));
                    tc_commit(bar(C::B_KE + st));
                    return true;
                };
                ok = mbar_wait(bar(C::B_QF), (uint32_t)it & 1u, abort_flag) && issue_s(g);
                if (n_kt == 1) tc_commit(bar(C::B_QE));
                for (int t = 0; t < n_kt && ok; ++t, ++g) {
                    if (t + 1 < n_kt) {
                        ok = issue_s(g + 1);
                        if (!ok) break;
                        if (t + 2 == n_kt) tc_commit(bar(C::B_QE));
                    }
                    const uint32_t ph = (uint32_t)(g >> 1) & 1u;
                    ok = mbar_wait(bar(C::B_PF + (g & 1)), ph, abort_flag) && mbar_wait(bar(C::B_VF + (g & 1)), ph, abort_flag) &&
                         (t > 0 || it == 0 || mbar_wait(bar(C::B_OF), (uint32_t)(it - 1) & 1u, abort_flag));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t tP = tS + (g & 1) * TK;
#pragma unroll
                    for (int ks = 0; ks < TK / 16; ++ks)
                        tc_mma_f16_ts(tO, tP + 8 * ks, v_desc + (uint64_t)((g & 1) * (C::VB >> 4) + ks * (16 * 128 >> 4)), idesc_o,
                                      (t > 0 || ks > 0) ? 1u : 0u);
                    tc_commit(bar(C::B_PV + (g & 1)));
                }
                ++it;
            }
            tc_commit(bar(C::B_IDLE));   // completes once every MMA of this thread has
        }
    } else if (warp < 6) {
        // ---- softmax: one row a thread
        const int quad = warp & 3;
        const int row = quad * 32 + lane;
        const int qi = row / p.G, hq = row - qi * p.G;
        const uint32_t lS0 = tS + ((uint32_t)(quad * 32) << 16), lO = tO + ((uint32_t)(quad * 32) << 16);
        int g = 0, it = 0;
        for (int k = 0; ok; ++k) {
            const int n_kt = item(k, r, head);
            if (n_kt == 0) break;
            const bool row_ok = qi < p.QT && r.q_lo + qi < r.n;
            const int limit = row_ok ? r.kv_len - r.n + r.q_lo + qi + 1 : 0;      // keys below it count
            const int clear = r.kv_len - r.n + r.q_lo + 1;                        // ... for every row of the tile
            ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_QS + it % NQS), (uint32_t)(it / NQS) & 1u, abort_flag));
            if (!ok) break;
            const float q_unscale = qs[(it % NQS) * TROWS + row] * p.scale_log2;
            float m = -INFINITY, M = -INFINITY, l = 0.f;
            for (int t = 0; t < n_kt && ok; ++t, ++g) {
                ok = __all_sync(0xffffffffu,
                                mbar_wait(bar(C::B_SC + g % NSC), (uint32_t)(g / NSC) & 1u, abort_flag) &&
                                    mbar_wait(bar(C::B_SF + (g & 1)), (uint32_t)(g >> 1) & 1u, abort_flag));
                if (!ok) break;
                tc_fence_after();
                const uint32_t lS = lS0 + (g & 1) * TK;
                const float* ks = sc + (g % NSC) * 3 * NB;   // then the V exponents and factors
                const int j0 = (t_first + t) * TK;
                const bool whole = j0 + TK <= clear && there[g % NSC] != 0;   // every key counts for every row
                float mx = -INFINITY, Mx = -INFINITY;
                if (whole)
                    max_pass_whole(lS, ks, q_unscale, mx, Mx);
                else
                    max_pass_masked(lS, ks, q_unscale, limit - j0, mx, Mx);
                const float mn = fmaxf(m, mx);
                const float mr = mn == -INFINITY ? 0.f : mn;
                l *= ex2(m - mr);
                m = mn;
                const float Mn = Mx > M + kSlack ? Mx : M;
                const float Mr = Mn == -INFINITY ? 0.f : Mn;
                const float alpha = ex2(M - Mr);   // exactly 1 while the reference stays
                M = Mn;
                if (t > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_PV + ((g - 1) & 1)), (uint32_t)((g - 1) >> 1) & 1u, abort_flag));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int ch = 0; ch < HD; ch += 32) {
                        float o[32];
                        tmem_ld32(lO + ch, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= alpha;
                        tmem_st32(lO + ch, o);
                    }
                }
                const float up = mr - Mr + kUnit;
                l += whole ? weight_pass<false>(lS, ks, q_unscale, 0, mr, up)
                           : weight_pass<true>(lS, ks, q_unscale, limit - j0, mr, up);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_PF + (g & 1)));
            }
            if (!ok) break;
            // the commit of an item's last PV covers the ones before it
            ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_PV + ((g - 1) & 1)), (uint32_t)((g - 1) >> 1) & 1u, abort_flag));
            if (!ok) break;
            tc_fence_after();
            if (shares && n_kt < t_all) {   // a part: the sums as they are
                float* part = p.parts + (2LL * blockIdx.x + (t_first == 0 ? 1 : 0)) * PromptSlot<HD>::FLOATS;
#pragma unroll 1
                for (int ch = 0; ch < HD; ch += 32) {
                    float o[32];
                    tmem_ld32(lO + ch, o);
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4*>(part + row * HD + ch + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
                part += TROWS * HD;
                part[row] = m;
                part[TROWS + row] = l;
                part[2 * TROWS + row] = M;
                if (t_first == 0 && row == 0) {   // its first part; the share is at its end
                    const long long all = *reinterpret_cast<const long long*>(p.list + 2);
                    const long long share = (all + gridDim.x - 1) / gridDim.x;
                    const long long end = (blockIdx.x + 1LL) * share - n_kt + t_all;
                    p.desc[blockIdx.x] = PromptDesc{r.row0, r.n, r.q_lo, head, (int)((end - 1) / share), r.b, r.kv_len, r.keys};
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_OF));
                ++it;
                continue;
            }
            // O is in units of 2^(M - 11); l is 0 for a row that saw no key, and NaN when a score was
            const float f = l == 0.f ? 0.f : exp2f((M == -INFINITY ? 0.f : M) - (m == -INFINITY ? 0.f : m)) / l;
            bf16* dst = p.out + ((long long)(r.row0 + r.q_lo + qi) * p.nq + head * p.G + hq) * HD;
#pragma unroll 1
            for (int ch = 0; ch < HD; ch += 32) {
                float o[32];
                tmem_ld32(lO + ch, o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = o[e] * 0x1p-11f * f;
                if (ch == 32 * (quad % (HD / 32))) {   // (a NaN of V is in every row's sum of its dim)
                    float2 t2 = make_float2(o[0], o[1]);
#pragma unroll
                    for (int e = 2; e < 32; e += 2) t2 = add2(t2, make_float2(o[e], o[e + 1]));
                    if (t2.x != t2.x || t2.y != t2.y) *nan_out = 1;
                }
                if (row_ok) {
                    if (p.v8) {
                        st_global_32(dst + ch, pack8(o), pack8(o + 8));
                        st_global_32(dst + ch + 16, pack8(o + 16), pack8(o + 24));
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) *reinterpret_cast<uint4*>(dst + ch + e) = pack8(o + e);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::B_OF));
            ++it;
        }
    } else {
        // ---- Q of each item, then its V tiles
        const int w = warp - 6;
        // V: keys 16 w .. 16 w + 15 of a tile, one block; this lane's codes are 16 of the rows kq and 8 + kq
        constexpr int HALVES = HD / 64;
        const int kq = ((lane >> 2) & 1) + 2 * (lane >> 3), c16 = lane & 3;
        const long long page_bytes = 2LL * c.n_kv * c.page_size * HD;
        constexpr int LPR = HD / 16, RPP = 32 / LPR;
        const int x = lane % LPR, qi_first = (w * 32 + lane / LPR) / p.G, hq_first = w * 32 + lane / LPR - qi_first * p.G;
        const int rpp_qi = RPP / p.G, rpp_hq = RPP - rpp_qi * p.G;
        int g = 0, it = 0;
        for (int k = 0; ok; ++k) {
            const int n_kt = item(k, r, head);
            if (n_kt == 0) break;
            uint4 raw[2][2 * HALVES];   // the codes of two tiles on their way
            const uint8_t* head_v = c.codes + kv8_code_at(c, 0, 1, head, 0) + kq * HD + c16 * 16;
            const int32_t* table = c.table + (long long)r.b * c.max_pages;
            auto page_of = [&](int t) {
                const int pos = (t_first + t) * TK + w * kKv8Block;
                if (pos >= r.keys) return -1;   // below it: inside the row of the table
                const int page = table[pos >> c.page_shift];
                return page < c.n_pages ? page : -1;
            };
            auto request = [&](uint4(&v)[2 * HALVES], int t, int page) {
                const int pos = (t_first + t) * TK + w * kKv8Block;
                const uint8_t* src = head_v + (long long)max(page, 0) * page_bytes + (pos & (c.page_size - 1)) * HD;
                if (page >= 0 && pos + kKv8Block <= r.keys) {
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int h = 0; h < HALVES; ++h)
                            v[y * HALVES + h] = *reinterpret_cast<const uint4*>(src + 8 * y * HD + h * 64);
                } else {
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int h = 0; h < HALVES; ++h) {
                            uint4 u = make_uint4(0u, 0u, 0u, 0u);
                            if (page >= 0 && pos + 8 * y + kq < r.keys)
                                u = *reinterpret_cast<const uint4*>(src + 8 * y * HD + h * 64);
                            v[y * HALVES + h] = u;
                        }
                }
            };
            int page = page_of(0), page1 = page_of(1);
            {   // Q: hi and lo codes of rows 32 w .. 32 w + 31, LPR lanes a row, 16 elements a lane
                int qi = qi_first, hq = hq_first;   // of this lane's row of a pass
#pragma unroll 1
                for (int p0 = 0; p0 < LPR; p0 += 4) {
                    uint4 u[4][2];   // four passes in flight; the first ones while the item before still runs
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        u[y][0] = u[y][1] = make_uint4(0u, 0u, 0u, 0u);
                        if (qi < p.QT && r.q_lo + qi < r.n) {
                            const uint4* src = reinterpret_cast<const uint4*>(
                                p.q + (long long)(r.row0 + r.q_lo + qi) * p.row_stride + (long long)(head * p.G + hq) * HD + 16 * x);
                            u[y][0] = src[0];
                            u[y][1] = src[1];
                        }
                        qi += rpp_qi;   // RPP rows on
                        hq += rpp_hq;
                        if (hq >= p.G) {
                            hq -= p.G;
                            ++qi;
                        }
                    }
                    if (p0 == 0 && it >= 1)
                        ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_QE), (uint32_t)(it - 1) & 1u, abort_flag));
                    if (!ok) break;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int row = w * 32 + (p0 + y) * RPP + lane / LPR;
                        const uint32_t in[8] = {u[y][0].x, u[y][0].y, u[y][0].z, u[y][0].w,
                                                u[y][1].x, u[y][1].y, u[y][1].z, u[y][1].w};
                        // the row's largest magnitude: bf16 bits without their sign order like the values
                        uint32_t top = 0u;
#pragma unroll
                        for (int e = 0; e < 8; ++e) top = __vmaxu2(top, in[e] & 0x7FFF7FFFu);
                        top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
                        for (int o = 1; o < LPR; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                        const uint32_t s = kv8_scale_bits(min(top, 0x7F7Fu) << 16);
                        const float inv = __uint_as_float((254u << 23) - s);   // 1 / s: a power of two
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            uint32_t hc[2], lc[2];
#pragma unroll
                            for (int z = 0; z < 2; ++z) {   // q / s fits f16 exactly, but for what is under 2^-25
                                const uint32_t v = pack_h2(__uint_as_float(in[e + z] << 16) * inv,
                                                           __uint_as_float(in[e + z] & 0xFFFF0000u) * inv);
                                hc[z] = f16x2_e4m3x2(v);
                                const uint32_t back = e4m3x2_f16x2(hc[z]);
                                const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&back));
                                lc[z] = f16x2_e4m3x2(*reinterpret_cast<const uint32_t*>(&d));
                            }
                            hi[e >> 1] = __byte_perm(hc[0], hc[1], 0x5410);
                            lo[e >> 1] = __byte_perm(lc[0], lc[1], 0x5410);
                        }
                        const int at = row * HD + ((HD == 128 ? x ^ (row & 7) : x ^ ((row >> 1) & 3)) << 4);
                        *reinterpret_cast<uint4*>(smem + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(smem + C::QB + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        // a row with an infinity or a NaN gives NaN
                        if (x == 0) qs[(it % NQS) * TROWS + row] = __uint_as_float(top < 0x7F80u ? s : 0x7FC00000u);
                    }
                }
                if (!ok) break;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(C::B_QF));
                    mbar_arrive(bar(C::B_QS + it % NQS));
                }
            }
            request(raw[0], 0, page);
            request(raw[1], 1, page1);
            page = page_of(2);
            // tile t from v, tile t + 2 into it
            auto turn = [&](uint4(&v)[2 * HALVES], int t) {
                if (g >= 2) ok = __all_sync(0xffffffffu, mbar_wait(bar(C::B_PV + (g & 1)), (uint32_t)((g >> 1) - 1) & 1u, abort_flag));
                if (!ok) return;
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int h = 0; h < HALVES; ++h) {
                        const uint4 u = v[y * HALVES + h];
                        uint32_t f[8];
                        e4m3x4_f16x4(u.x, f[0], f[1]);
                        e4m3x4_f16x4(u.y, f[2], f[3]);
                        e4m3x4_f16x4(u.z, f[4], f[5]);
                        e4m3x4_f16x4(u.w, f[6], f[7]);
                        const int key = w * kKv8Block + 8 * y + kq;
                        uint8_t* at = smem + C::OFF_V + (g & 1) * C::VB + h * TK * 128 + key * 128;
                        *reinterpret_cast<uint4*>(at + (((2 * c16) ^ (key & 7)) << 4)) =
                            make_uint4(f[0], f[1], f[2], f[3]);
                        *reinterpret_cast<uint4*>(at + (((2 * c16 + 1) ^ (key & 7)) << 4)) =
                            make_uint4(f[4], f[5], f[6], f[7]);
                    }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::B_VF + (g & 1)));
                if (t + 2 < n_kt) request(v, t + 2, page);
                if (t + 3 < n_kt) page = page_of(t + 3);
                ++g;
            };
            for (int t = 0; t < n_kt && ok; t += 2) {
                turn(raw[0], t);
                if (t + 1 < n_kt && ok) turn(raw[1], t + 1);
            }
            ++it;
        }
    }
    if (!ok) {
        *abort_flag = 1;
        raise_error(c.err, HRA_DEVERR_WAIT_TIMEOUT);
    }

    // ---- teardown: on abort, let every requested copy and every MMA land first
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
        volatile int never = 0;
        if (*abort_flag)
            for (int g = max(0, *issued - NK); g < *issued; ++g) (void)mbar_wait(bar(C::B_KF + g % NK), (uint32_t)(g / NK) & 1u, &never);
        (void)mbar_wait(bar(C::B_IDLE), 0u, &never);
    }
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tS, 256);
    }
    if (*nan_out && !*abort_flag) outputs_again<HD>(p, first_s);
}

// The parts of the item that begins in share blockIdx.x and goes on behind it, in order; 8 rows a CTA.
template <int HD>
__global__ void __launch_bounds__(256) kv8_prompt_join_kernel(const __grid_constant__ PromptArgs p) {
    pdl_launch();
    pdl_wait();
    const int c0 = blockIdx.x;
    const PromptDesc d = p.desc[c0];
    if (d.row0 < 0) return;
    const int row = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int qi = row / p.G, hq = row - qi * p.G;
    if (qi >= p.QT || d.q_lo + qi >= d.n) return;
    constexpr int E = HD / 32;
    const int parts = d.last - c0 + 1;
    auto slot = [&](int i) { return p.parts + (2LL * (c0 + i) + (i == 0 ? 1 : 0)) * PromptSlot<HD>::FLOATS; };
    float m = -INFINITY, M = -INFINITY;
    for (int i = 0; i < parts; ++i) {
        const float* q = slot(i) + TROWS * HD + row;
        m = fmaxf(m, q[0]);
        M = fmaxf(M, q[2 * TROWS]);
    }
    const float mr = m == -INFINITY ? 0.f : m, Mr = M == -INFINITY ? 0.f : M;
    float l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
        const float* q = slot(i) + TROWS * HD + row;
        const float* x = slot(i) + row * HD + lane * E;
        l += q[TROWS] * ex2(q[0] - mr);
        const float f = ex2(q[2 * TROWS] - Mr);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += x[e] * f;
    }
    const float f = l == 0.f ? 0.f : exp2f(Mr - mr) / l;
    bf16* dst = p.out + ((long long)(d.row0 + d.q_lo + qi) * p.nq + d.head * p.G + hq) * HD + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t*>(dst + e) = pack_bf2(o[e] * 0x1p-11f * f, o[e + 1] * 0x1p-11f * f);
    bool nan = false;
#pragma unroll
    for (int e = 0; e < E; ++e) nan |= o[e] != o[e];
    if (nan) look_again(p, PromptRec{d.b, d.row0, d.n, d.q_lo, d.kv_len, d.keys, 0}, d.head, row, lane * E, E, dst);
}

int prompt_slots() { return 2 * device_sm_count(); }

// Equal shares where the items are long and so few that the CTAs' turns would not come out even.
bool prompt_shares(long long pairs, int n_kv, int max_len) {
    return max_len > kSharesFrom && pairs * n_kv < 8LL * prompt_slots();
}
long long most_pairs(int batch, int total_rows, int QT, int max_new) {
    return std::min((long long)((max_new + QT - 1) / QT) * batch, (long long)total_rows / QT + batch);
}

// Sequences that share no rows have sum ceil(n / QT) <= total / QT + batch tiles.
long long list_pairs(int batch, int total_rows, int G) { return (long long)total_rows / (TROWS / G) + batch; }
size_t list_bytes(int batch, int total_rows, int G) {
    return (size_t)(list_pairs(batch, total_rows, G) + 1) * kRecWords * sizeof(int32_t);
}

template <int HD>
cudaError_t launch_hd(const Kv8AttnArgs& a, int G, int QT, int short_rows, cudaStream_t st) {
    using C = Cfg<HD>;
    alignas(64) CUtensorMap map;
    const long long rows = 2LL * a.view.n_pages * a.view.n_kv * a.view.page_size;
    if (!make_map_codes(&map, a.view.codes, rows, HD, kKv8Block)) return cudaErrorInvalidValue;
    static bool configured[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(kv8_prompt_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::ALLOC);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    int32_t* list = reinterpret_cast<int32_t*>(a.scratch);
    const long long pairs = most_pairs(a.batch, a.total_rows, QT, a.max_new);
    const bool shares = prompt_shares(pairs, a.view.n_kv, a.max_len);
    HRA_LAUNCH(kv8_schedule_kernel, dim3(1), dim3(1024), 0, st, a, G, QT, short_rows, shares ? 1 : 0,
               (int)list_pairs(a.batch, a.total_rows, G), list);
    PromptArgs p{};
    p.view = a.view;
    p.q = a.q;
    p.row_stride = a.row_stride;
    p.out = a.out;
    p.list = list;
    p.scale_log2 = a.scale_log2;
    p.nq = a.nq;
    p.G = G;
    p.QT = QT;
    p.v8 = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0 ? 1 : 0;
    const int grid = shares ? prompt_slots() : (int)std::max<long long>(1, std::min<long long>(pairs * a.view.n_kv, prompt_slots()));
    if (shares) {
        uint8_t* at = reinterpret_cast<uint8_t*>(a.scratch) + list_bytes(a.batch, a.total_rows, G);
        p.desc = reinterpret_cast<PromptDesc*>(at);
        p.parts = reinterpret_cast<float*>(at + grid * sizeof(PromptDesc));
    }
    HRA_LAUNCH(kv8_prompt_kernel<HD>, dim3(grid), dim3(kThreads), C::ALLOC, st, map, p);
    if (shares) HRA_LAUNCH(kv8_prompt_join_kernel<HD>, dim3(grid, TROWS / 8), dim3(256), 0, st, p);
    return cudaGetLastError();
}

}  // namespace

// Never less for more of anything, so that a caller may size it for the most: the shares' slots also where there are so
// many pairs that they are not used.
size_t kv8_prompt_scratch_bytes(const Kv8View& c, int batch, int total_rows, int G, int max_len) {
    size_t n = list_bytes(batch, total_rows, G);
    if (max_len > kSharesFrom)
        n += (size_t)prompt_slots() * (sizeof(PromptDesc) + 2 * sizeof(float) * TROWS * (c.head_dim + 3));
    return n;
}

cudaError_t launch_kv8_prompt(const Kv8AttnArgs& a, int short_rows, cudaStream_t st) {
    const int G = a.nq / a.view.n_kv, QT = TROWS / G;
    return a.view.head_dim == 128 ? launch_hd<128>(a, G, QT, short_rows, st) : launch_hd<64>(a, G, QT, short_rows, st);
}

}  // namespace hra
