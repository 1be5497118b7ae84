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
// The work is a line of units of 128 keys, sequence by sequence and head by head; every CTA takes an equal share
// of it, wherever the borders between sequences fall, so ragged lengths cost nothing and one long sequence
// spreads over the whole GPU.  An item (sequence, head) that lies inside one share is written at once; the parts
// of the others go to scratch as fp32 sums with their (m, l, M), and a second kernel joins them in order.
//
// A warp takes two blocks of 16 keys at a time.  The order of the dims inside a dot product, of the dims among the
// output rows and of the keys of a block is free, so it is chosen such that every lane reads its share of a block as
// whole 16-byte pieces that become MMA fragments with no exchange between lanes:
//   S = Q K^T   (m16n8k16): rows are up to 16 (position, head) pairs, lane (g, t) = (lane / 4, lane % 4)
//               reads pieces 16 t and 64 + 16 t of keys k(g) and k(g) + 8;
//   O^T = V^T P^T: lane (g, t) reads dims 16 g .. 16 g + 15 of keys k(2t), k(2t + 1) and those + 8, and the P^T
//               fragment is the lane's own S accumulators;
//   k(2 j) = 2 j, k(2 j + 1) = (2 j ^ 4) + 1: with the copies' 128-byte swizzle no read has a bank conflict.
// Each warp has its own ring of stages that TMA fills, one box of 16 rows for K and one for V a block, so a
// block costs one lane two instructions to request.  64 sequences of up to 8192 keys, 8 kv heads of 128, 4 q heads
// each (559 MB): 108 us, 5.2 TB/s; with the pieces copied by cp.async, an address a lane each, 140 us; one block at a
// time 117-124 us (both against 112 then).  What is left is the warps' own work: 48% of issue slots, 12 warps an SM.
// Through a window of 2048 and 4 sinks the same 64 rows, of up to 32,768 positions (254 MB seen), take 58 us, 4.4 TB/s.  Heads of 128 in two
// column groups are at the limit of their registers: 100 bytes spilled a thread, 142-158 through a window.
#include <math.h>

#include <algorithm>

#include "kv8_parts.cuh"

namespace hra {

namespace {

// The positions that tokens see: all, a window's and the sinks', or those behind a shared prefix (and then only parts are written)
enum { kAll, kWindow, kOwn };
constexpr int kWarps = 4;
constexpr int kPair = 2;        // blocks a warp works on at once: two chains of MMAs and shuffles instead of one
constexpr int kStages = 2;      // pairs of a warp in shared memory: 12 warps an SM; with 3, 8 warps fit (121 us against 112)
constexpr int kUnit = kWarps * kPair * kKv8Block;   // keys of a unit: a pair of blocks a warp
constexpr int kMaxBatch = 1024;             // sequences whose units fit the CTA's table
// Items of at most so many units go whole, one a CTA, and need no second kernel.  One token, 8 kv heads of 128, in a graph,
// whole / split: 8 rows after 512 positions 8.6 / 10.2 us, after 768 11.2 / 10.3; 1 row 8.0 / 7.7 and 10.6 / 8.1; 64 rows
// after 512 19.6 / 24.0, after 1024 33.2 / 33.2.
constexpr int kWholeUnits = 4;
constexpr int kShortRows = 16;  // (position, head) rows of a kv head that fit this kernel's tile
// Keys that a short sequence may walk alone among prompts.  One prompt of 256 tokens beside single tokens, among the prompts /
// in this kernel: 8 of them after 1024 positions 25 / 32 us, after 2048 40 / 39, after 4096 83 / 54; 48 of them 49 / 60, 81 / 83
// and 277 / 126.
constexpr int kSerialKeys = 2048;
constexpr float kPScale = kRowsUnit;   // log2 of the largest p
static_assert(kUnit == 128, "units of kv8_own");

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// A stage: K and V of a pair of blocks as TMA writes them (rows of HD bytes, swizzled over the row: 1024- or
// 512-byte atoms), and the blocks' scales, a copy a lane.
template <int HD>
struct Ring {
    static constexpr int BLOCK = kKv8Block * HD;               // K (or V) of a block
    static constexpr int CODES = kPair * 2 * BLOCK;            // of a stage: [pair][K, V]
    static constexpr int SCALES = kPair * 32 * 8;
    static constexpr int ALL_CODES = kWarps * kStages * CODES;
    static constexpr int BYTES = ALL_CODES + kWarps * kStages * SCALES;
    // byte offset of 16-byte chunk `chunk` of row `row`
    static __device__ __forceinline__ int at(int row, int chunk) {
        return row * HD + ((HD == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3)) << 4);
    }
};

// Parts of split items: CTA c has slots 2 c (the item that its share begins in) and 2 c + 1 (the one it ends in).
// desc[c]: the item whose first part is CTA c's slot 2 c + 1 and
// the last CTA that has a part of it.
struct SplitDesc {
    int row0, n, head, last;   // n: tokens; row0 < 0: no item begins in this share and goes on behind it
    int b, pad[3];
};
struct SplitArgs {
    Kv8AttnArgs a;
    SplitDesc* desc;
    float* parts;
    int G, max_rows;   // sequences with at most max_rows (position, head) rows a kv head
    int whole;         // one item a CTA: blockIdx = (head, sequence)
    // behind a shared prefix: blockIdx = (head, tile of a sequence's tokens, split)
    const SharedRow* shared;
    int row_tiles, own_units;
};

// Dims d and d + 1 of row r, written to dst, are or hold a NaN: see kv8_row_again.
__device__ __noinline__ void look_again(const SplitArgs& s, int b, int head, int r, int d, bf16* dst) {
    const Kv8View& c = s.a.view;
    int row0, n;
    kv8_rows(s.a.cu, b, s.a.total_rows, row0, n);
    const int qi = r / s.G, hq = r - qi * s.G;
    const int before = min(c.max_pages << c.page_shift, max(0, s.a.kv_len[b])) - n;   // positions before the first token
    const bf16* q = s.a.q + (long long)(row0 + qi) * s.a.row_stride + (long long)(head * s.G + hq) * c.head_dim;
    const int lo = s.a.window > 0 ? before + qi + 1 - s.a.window : 0;
    kv8_row_again(c, q, b, head, before + qi + 1, before + n, d, 2, s.a.scale_log2, dst, lo, s.a.sinks, max(0, lo - qi));
}

// NG x 8 rows of (position, head) pairs.  ONE: sequences of one new token, whose rows all see the same keys.  MODE: all
// positions, or those of a window and the sinks, or those behind a shared prefix: then units, blocks and lengths below count what
// some token of the sequence sees, kv8_unit_at says which block that is, and only blocks at the window's edge look at its
// border.
template <int HD, int NG, bool ONE, int MODE>
__global__ void __launch_bounds__(kWarps * 32, 3) kv8_attn_kernel(const __grid_constant__ CUtensorMap codes_map,
                                                                  const __grid_constant__ SplitArgs s) {
    pdl_launch();
    pdl_wait();
    using R = Ring<HD>;
    constexpr int KS = HD / 16;       // k steps of S
    constexpr int DT = HD / 16;       // 16-dim tiles of O^T
    constexpr int ROWS = 8 * NG;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t bars[kWarps * kStages];
    __shared__ int abort_flag;
    __shared__ int before[kMaxBatch + 1];   // units of one head of the sequences before
    __shared__ int warp_total[kWarps];
    const Kv8AttnArgs& a = s.a;
    const Kv8View& c = a.view;
    const int G = s.G;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int room = c.max_pages << c.page_shift;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kWarps * kStages; ++i) mbar_init(smem_u32(bars + i), 1);
        abort_flag = 0;
        mbar_fence_init();
        tma_prefetch_map(&codes_map);
    }
    __syncthreads();
    auto length = [&](int b) { return min(room, max(0, a.kv_len[b])); };
    auto skipped = [&](int len, int n) {   // blocks that no token sees of a sequence of `len` positions, n of them new
        return MODE == kWindow ? kv8_skip(len - n, a.window, a.sinks, kKv8Block) : Kv8Skip{0, 0};
    };

    // ---- this CTA's share
    long long u = 0, u_end = 1;
    long long share = 0;
    if (MODE != kOwn && !s.whole) {
        // units of the sequences, summed up front: consecutive sequences a thread, then across threads
        const int per = (a.batch + kWarps * 32 - 1) / (kWarps * 32);
        const int b0 = threadIdx.x * per;
        int mine = 0;
        for (int i = 0; i < per; ++i) {
            const int b = b0 + i;
            int units = 0;
            if (b < a.batch) {
                int row0, n;
                kv8_rows(a.cu, b, a.total_rows, row0, n);
                // a sequence with new tokens but no keys has one unit: its rows get 0
                if (n > 0 && n <= s.max_rows / G) {
                    const int len = length(b);
                    units = max(1, (len - skipped(len, n).by * kKv8Block + kUnit - 1) / kUnit);
                }
                before[b] = units;
            }
            mine += units;
        }
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) warp_total[warp] = incl;
        __syncthreads();
        int run = incl - mine;
        for (int w = 0; w < warp; ++w) run += warp_total[w];
        for (int i = 0; i < per; ++i) {
            const int b = b0 + i;
            if (b < a.batch) {
                const int v = before[b];
                before[b] = run;
                run += v;
            }
        }
        if (threadIdx.x == kWarps * 32 - 1) before[a.batch] = run;
        __syncthreads();
        const long long all = (long long)before[a.batch] * c.n_kv;
        share = (all + gridDim.x - 1) / gridDim.x;
        u = blockIdx.x * share;
        u_end = min(all, u + share);
        if (threadIdx.x == 0) s.desc[blockIdx.x].row0 = -1;
        if (u >= u_end) return;
    }

    uint8_t* ring = sm + warp * kStages * R::CODES;
    uint8_t* ring_scales = sm + R::ALL_CODES + warp * kStages * R::SCALES + lane * 8;
    const uint32_t ring_bar = smem_u32(bars + warp * kStages);
    uint32_t phases = 0u;      // the next phase of each stage's barrier
    const int page_rows = 2 * c.n_kv * c.page_size, v_rows = c.n_kv * c.page_size;   // rows of the tensor map
    const int page_scales = 2 * c.n_kv * (c.page_size / kKv8Block), v_scales = page_scales / 2;
    const int key_g = g & 1 ? ((g - 1) ^ 4) + 1 : g;   // k(g), k(2 t), k(2 t + 1)
    const int key_0 = 2 * t4, key_1 = (key_0 ^ 4) + 1;
    bool bad_page = false;

    while (u < u_end) {
        // ---- the segment: units [i0, i1) of item (b, head)
        int b, head, i0 = 0, i1, row0, n;
        bool first_part = true, last_part = true;
        Kv8Own own{};
        if (MODE == kOwn) {
            b = blockIdx.y / s.row_tiles;
            head = blockIdx.x;
            kv8_rows(a.cu, b, a.total_rows, row0, n);
            own = kv8_own(length(b), n, blockIdx.y - b * s.row_tiles, ROWS / G, a.max_new, s.shared[b].prefix, gridDim.z, s.own_units);
            if (own.tokens == 0 || blockIdx.z >= own.parts) return;
            i0 = blockIdx.z * own.per;
            i1 = i0 + own.per;
            row0 += own.t0;
            u = u_end;
        } else if (s.whole) {
            b = blockIdx.y;
            head = blockIdx.x;
            kv8_rows(a.cu, b, a.total_rows, row0, n);
            if (n == 0 || n > s.max_rows / G) return;
            i1 = 1 << 30;
            u = u_end;
        } else {
            const int ub = (int)(u / c.n_kv);
            int lo = 0, hi = a.batch;      // the last b with before[b] * n_kv <= u
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (before[mid] <= ub) lo = mid;
                else hi = mid;
            }
            b = lo;
            const int units = before[b + 1] - before[b];
            const int at = (int)(u - (long long)before[b] * c.n_kv);
            head = at / units;
            i0 = at - head * units;
            i1 = (int)min((long long)units, i0 + (u_end - u));
            first_part = i0 == 0;
            last_part = i1 == units;
            u += i1 - i0;
            kv8_rows(a.cu, b, a.total_rows, row0, n);
        }
        const int kv_len = length(b);
        if (head == 0 && threadIdx.x == 0 && first_part && blockIdx.z == 0 && own.t0 == 0 &&
            (a.kv_len[b] != kv_len || n > a.max_new))
            raise_error(c.err, HRA_DEVERR_POS_RANGE);
        const int q_n = MODE == kOwn ? own.tokens : min(min(ROWS / G, n), a.max_new);   // tokens beyond max_new get no output
        const int first = kv_len - n + own.t0;         // position of the first token
        const int keys = max(0, first + q_n);          // positions below the last of them
        const Kv8Skip skip = MODE == kOwn ? Kv8Skip{0, s.shared[b].prefix / kKv8Block} : skipped(kv_len, n);
        auto first_key = [&](int x) { return (MODE == kAll ? x : kv8_unit_at(skip, x)) * kKv8Block; };   // of block x
        const int blk1 = min((keys + kKv8Block - 1) / kKv8Block - skip.by, i1 >= (1 << 28) ? 1 << 28 : i1 * (kWarps * kPair));
        const int lo0 = first + 1 - a.window;          // window: the first position of the first token's
        int blk = (i0 * kWarps + warp) * kPair;
        constexpr int STEP = kWarps * kPair;

        // ---- page numbers two turns of this warp ahead of the use, requests kStages - 1 ahead
        const int32_t* table = c.table + (long long)b * c.max_pages;
        struct Pages {
            int p[kPair];
        };
        auto pages_of = [&](int x) {   // -1: no page of the pool; -2: behind the last block
            Pages r;
#pragma unroll
            for (int y = 0; y < kPair; ++y) {
                r.p[y] = -2;
                if (x + y < blk1) {   // first_key(x + y) < keys <= max_pages * page_size
                    const int page = table[first_key(x + y) >> c.page_shift];
                    r.p[y] = page >= 0 && page < c.n_pages ? page : -1;
                }
            }
            return r;
        };
        const float* head_scales = c.scales + head * (c.page_size / kKv8Block);
        // blocks x0, x0 + 1 into stage st; one without a page gets scales of -1 and is masked below
        auto request = [&](int x0, const Pages& pages, int st) {
            int boxes = 0;
#pragma unroll
            for (int y = 0; y < kPair; ++y) {
                const int page = pages.p[y];
                bad_page |= page == -1;
                boxes += page >= 0 ? 2 : 0;
                const int slot0 = first_key(x0 + y) & (c.page_size - 1);
                const float* sp = head_scales + (long long)max(page, 0) * page_scales + (slot0 / kKv8Block);
                const uint32_t to = smem_u32(ring_scales + st * R::SCALES + y * 32 * 8);
                if (page >= 0) {
                    cp_async4(to, sp);
                    cp_async4(to + 4, sp + v_scales);
                } else {   // (this lane's own slot, whose last copy it has waited for)
                    *reinterpret_cast<float2*>(ring_scales + st * R::SCALES + y * 32 * 8) = make_float2(-1.f, -1.f);
                }
            }
            if (lane == 0) {
                const uint32_t bar = ring_bar + 8 * st;
                if (boxes)
                    mbar_expect_tx(bar, boxes * R::BLOCK);
                else
                    mbar_arrive(bar);
#pragma unroll
                for (int y = 0; y < kPair; ++y) {
                    if (pages.p[y] >= 0) {   // rows of the map are counted in 32 bits (checked before the launch)
                        const int row = pages.p[y] * page_rows + head * c.page_size + (first_key(x0 + y) & (c.page_size - 1));
                        const uint32_t to = smem_u32(ring + st * R::CODES + 2 * y * R::BLOCK);
                        tma_load_2d(to, &codes_map, bar, 0, row);
                        tma_load_2d(to + R::BLOCK, &codes_map, bar, 0, row + v_rows);
                    }
                }
            }
        };
        // q rows, on their way beside the page numbers
        uint4 q_raw[NG][HD / 64][2];
#pragma unroll
        for (int x = 0; x < NG; ++x) {
            const int r = g + 8 * x, qi = r / G, hq = r - qi * G;
            const bool ok = qi < q_n;
            const bf16* src = a.q + (long long)(row0 + (ok ? qi : 0)) * a.row_stride + (long long)(head * G + hq) * HD;
#pragma unroll
            for (int h = 0; h < HD / 64; ++h) {
                q_raw[x][h][0] = q_raw[x][h][1] = make_uint4(0u, 0u, 0u, 0u);
                if (ok) {
                    q_raw[x][h][0] = *reinterpret_cast<const uint4*>(src + h * 64 + t4 * 16);
                    q_raw[x][h][1] = *reinterpret_cast<const uint4*>(src + h * 64 + t4 * 16 + 8);
                }
            }
        }
        int ahead = blk;
        Pages page0 = pages_of(ahead), page1 = pages_of(ahead + STEP);
#pragma unroll
        for (int st = 0; st < kStages - 1; ++st) {
            const Pages page2 = pages_of(ahead + 2 * STEP);
            if (ahead < blk1) request(ahead, page0, st);
            cp_async_commit();
            ahead += STEP;
            page0 = page1;
            page1 = page2;
        }

        // ---- q fragments: f16, each row scaled by a power of two
        uint32_t qa[KS][2 * NG];
        float q_unscale[NG];
        int limit[NG];             // keys below this one count for the row
#pragma unroll
        for (int x = 0; x < NG; ++x) {
            const int r = g + 8 * x, qi = r / G, hq = r - qi * G;
            const bool ok = qi < q_n;
            limit[x] = ok ? min(keys, first + qi + 1) : 0;
            const uint4(&raw)[HD / 64][2] = q_raw[x];
            uint32_t top = 0u;     // bf16 bits without their sign order like the values
#pragma unroll
            for (int h = 0; h < HD / 64; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint4 w = raw[h][e];
                    top = __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                                 __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu)));
                }
            top = max(top & 0xFFFFu, top >> 16);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^(14 - floor(log2 of it)), its exponent kept inside fp32's normal range
            const int ex = min(254, max(14, (int)(top >> 7)));
            const float mul = __uint_as_float((uint32_t)(268 - ex) << 23);
            q_unscale[x] = __uint_as_float((uint32_t)max(1, ex - 14) << 23) * a.scale_log2;
#pragma unroll
            for (int h = 0; h < HD / 64; ++h) {
                float f[16], f1[8];
                unpack8(raw[h][0], f1);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = f1[e];
                unpack8(raw[h][1], f1);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[8 + e] = f1[e];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    qa[h * 4 + q][x] = pack_h2(f[4 * q] * mul, f[4 * q + 1] * mul);
                    qa[h * 4 + q][NG + x] = pack_h2(f[4 * q + 2] * mul, f[4 * q + 3] * mul);
                }
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

        int st = 0, st_in = kStages - 1;
#pragma unroll 1
        for (; blk < blk1; blk += STEP) {
            {
                const Pages page2 = pages_of(ahead + 2 * STEP);
                __syncwarp();   // every lane's pieces of the stage before are in its MMAs: the stage may be filled
                if (ahead < blk1) request(ahead, page0, st_in);
                page0 = page1;
                page1 = page2;
            }
            cp_async_commit();
            ahead += STEP;
            st_in = st_in + 1 == kStages ? 0 : st_in + 1;
            cp_async_wait<kStages - 1>();
            if (!__all_sync(0xffffffffu, mbar_wait(ring_bar + 8 * st, (phases >> st) & 1u, &abort_flag))) {
                // no further request; the copies under way land, or are waited for as long, before the CTA goes
                abort_flag = 1;
                raise_error(c.err, HRA_DEVERR_WAIT_TIMEOUT);
                volatile int never = 0;
                const int under_way = kv8_turns_left(blk, blk1, STEP, kStages);
                for (int i = 0; i < under_way; ++i, st = st + 1 == kStages ? 0 : st + 1)
                    (void)mbar_wait(ring_bar + 8 * st, (phases >> st) & 1u, &never);
                break;
            }
            phases ^= 1u << st;
            const uint8_t* codes = ring + st * R::CODES;
            const uint8_t* scales = ring_scales + st * R::SCALES;
            st = st + 1 == kStages ? 0 : st + 1;

            float sv[kPair][2][4];
            float2 sc[kPair];
            int key0[kPair];
#pragma unroll
            for (int y = 0; y < kPair; ++y) key0[y] = first_key(blk + y);
#pragma unroll
            for (int y = 0; y < kPair; ++y) {
                sc[y] = *reinterpret_cast<const float2*>(scales + y * 32 * 8);
#pragma unroll
                for (int i = 0; i < 2; ++i) sv[y][i][0] = sv[y][i][1] = sv[y][i][2] = sv[y][i][3] = 0.f;
            }
#pragma unroll
            for (int h = 0; h < HD / 64; ++h)
#pragma unroll
                for (int y = 0; y < kPair; ++y)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4 w = *reinterpret_cast<const uint4*>(codes + 2 * y * R::BLOCK + R::at(key_g + 8 * i, t4 + 4 * h));
                        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t b0, b1;
                            e4m3x4_f16x4(ww[q], b0, b1);
                            if (NG == 1)
                                mma_f16(sv[y][i], qa[h * 4 + q][0], 0u, qa[h * 4 + q][1], 0u, b0, b1);
                            else
                                mma_f16(sv[y][i], qa[h * 4 + q][0], qa[h * 4 + q][NG - 1], qa[h * 4 + q][NG],
                                        qa[h * 4 + q][2 * NG - 1], b0, b1);
                        }
                    }
            uint32_t pb[kPair][NG][2];
            float al[NG];
            bool moved = false;
            float ev[kPair], vm[kPair];
#pragma unroll
            for (int y = 0; y < kPair; ++y) {
                ev[y] = exponent_of(sc[y].y);
                vm[y] = mantissa_of(sc[y].y);
            }
#pragma unroll
            for (int x = 0; x < NG; ++x) {
                float z[kPair][4];
                float mx[kPair];
#pragma unroll
                for (int y = 0; y < kPair; ++y) {
                    const float coef = q_unscale[x] * sc[y].x;
                    // a scale of -1: the block is absent
                    const int lim = sc[y].x >= 0.f ? limit[x] - key0[y] : 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        z[y][e] = (e & 1 ? key_1 : key_0) + 8 * (e >> 1) < lim ? sv[y][e >> 1][2 * x + (e & 1)] * coef : -INFINITY;
                    if (MODE == kWindow && key0[y] < lo0 + q_n - 1 && key0[y] + kKv8Block > a.sinks) {   // some row's border
                        const int lo = limit[x] - a.window - key0[y], sinks = a.sinks - key0[y];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int k = (e & 1 ? key_1 : key_0) + 8 * (e >> 1);
                            if (k < lo && k >= sinks) z[y][e] = -INFINITY;
                        }
                    }
                    mx[y] = fmaxf(fmaxf(z[y][0], z[y][1]), fmaxf(z[y][2], z[y][3]));
                }
                float top = mx[0], Top = mx[0] + ev[0];
#pragma unroll
                for (int y = 1; y < kPair; ++y) {
                    top = fmaxf(top, mx[y]);
                    Top = fmaxf(Top, mx[y] + ev[y]);
                }
#pragma unroll
                for (int o2 = 1; o2 < 4; o2 <<= 1) {
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o2));
                    Top = fmaxf(Top, __shfl_xor_sync(0xffffffffu, Top, o2));
                }
                const float mn = fmaxf(m[x], top), Mn = fmaxf(M[x], Top);
                const float mr = mn == -INFINITY ? 0.f : mn, Mr = Mn == -INFINITY ? 0.f : Mn;
                al[x] = ex2(M[x] - Mr);
                l[x] *= ex2(m[x] - mr);
                moved |= al[x] != 1.f;
                m[x] = mn;
                M[x] = Mn;
#pragma unroll
                for (int y = 0; y < kPair; ++y) {
                    const float off = ev[y] + kPScale - Mr;
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        l[x] += ex2(z[y][e] - mr);
                        w[e] = ex2(z[y][e] + off) * vm[y];
                    }
                    pb[y][x][0] = pack_h2(w[0], w[1]);
                    pb[y][x][1] = pack_h2(w[2], w[3]);
                }
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
#pragma unroll
            for (int y = 0; y < kPair; ++y) {
                uint32_t vw[4][HD / 32];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = (i & 1 ? key_1 : key_0) + 8 * (i >> 1);
                    const uint8_t* at = codes + (2 * y + 1) * R::BLOCK;
                    if (HD == 128) {
                        const uint4 w = *reinterpret_cast<const uint4*>(at + R::at(key, g));
                        vw[i][0] = w.x;
                        vw[i][1] = w.y;
                        vw[i][HD / 32 - 2] = w.z;
                        vw[i][HD / 32 - 1] = w.w;
                    } else {
                        const uint2 w = *reinterpret_cast<const uint2*>(at + R::at(key, g >> 1) + 8 * (g & 1));
                        vw[i][0] = w.x;
                        vw[i][1] = w.y;
                    }
                }
                // keys that do not count: whatever their slots hold (a NaN times a weight of 0 is none)
                const int left = sc[y].x >= 0.f ? keys - key0[y] : 0;
                if (left < kKv8Block) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if ((i & 1 ? key_1 : key_0) + 8 * (i >> 1) >= left)
#pragma unroll
                            for (int j = 0; j < HD / 32; ++j) vw[i][j] = 0u;
                }
                if (MODE == kWindow && key0[y] < lo0 && key0[y] + kKv8Block > a.sinks) {   // behind every row's window
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = key0[y] + (i & 1 ? key_1 : key_0) + 8 * (i >> 1);
                        if (k < lo0 && k >= a.sinks)
#pragma unroll
                            for (int j = 0; j < HD / 32; ++j) vw[i][j] = 0u;
                    }
                }
#pragma unroll
                for (int j = 0; j < HD / 32; ++j) {
                    uint32_t a0, a1, a2, a3, c0, c1, c2, c3;
                    e4m3x4_f16x4(__byte_perm(vw[0][j], vw[1][j], 0x5140), a0, a1);
                    e4m3x4_f16x4(__byte_perm(vw[2][j], vw[3][j], 0x5140), a2, a3);
                    e4m3x4_f16x4(__byte_perm(vw[0][j], vw[1][j], 0x7362), c0, c1);
                    e4m3x4_f16x4(__byte_perm(vw[2][j], vw[3][j], 0x7362), c2, c3);
#pragma unroll
                    for (int x = 0; x < NG; ++x) {
                        mma_f16(o[x][2 * j], a0, a1, a2, a3, pb[y][x][0], pb[y][x][1]);
                        mma_f16(o[x][2 * j + 1], c0, c1, c2, c3, pb[y][x][0], pb[y][x][1]);
                    }
                }
            }
        }
        cp_async_wait<0>();
        __syncthreads();   // the rings are empty: the warps' results go over them
        if (abort_flag) return;   // a wait ran out: nothing is stored

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
        const bool whole = MODE != kOwn && first_part && last_part;
        const long long slot = MODE == kOwn ? ((long long)blockIdx.y * c.n_kv + head) * gridDim.z + blockIdx.z
                                            : 2LL * blockIdx.x + (first_part ? 1 : 0);
        float* part = s.parts + slot * Slot<HD, NG>::FLOATS;
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
            if (whole) {
                // L is 0 for a row that saw no key, and NaN when a score was
                const float f = L == 0.f ? 0.f : exp2f(Mr - mr) / L;
                bf16* dst = a.out + ((long long)(row0 + qi) * a.nq + head * G + hq) * HD + d;
                *reinterpret_cast<uint32_t*>(dst) = pack_bf2(x0 * 0x1p-15f * f, x1 * 0x1p-15f * f);
                if (!ONE && (x0 != x0 || x1 != x1)) look_again(s, b, head, r, d, dst);
            } else {
                *reinterpret_cast<float2*>(part + r * HD + d) = make_float2(x0, x1);
                if (d == 0) {
                    float* at = part + ROWS * HD + r * 3;
                    at[0] = mm;
                    at[1] = L;
                    at[2] = MM;
                }
            }
        }
        if (MODE != kOwn && first_part && !last_part && threadIdx.x == 0) {
            const long long end = (long long)before[b] * c.n_kv + (long long)(head + 1) * (before[b + 1] - before[b]);
            s.desc[blockIdx.x] = SplitDesc{row0, q_n, head, (int)((end - 1) / share), b, {0, 0, 0}};
        }
        fence_proxy_async_smem();   // the sums below the next copies
        __syncthreads();            // the results are read: the rings may be filled again
    }
    if (bad_page) raise_error(c.err, HRA_DEVERR_PAGE_RANGE);
}

// One CTA per share: the item that begins in it and goes on behind it.  The rows' maxima and sums over all parts
// come first (a warp a row, a lane a part), then every thread adds its columns, parts in order, with the loads free of
// each other and the first ones under way before (8 rows after 1024-2112 positions, both kernels in a graph over 36
// layers: 15.6 us, and 17.0 with one under way instead of eight).
template <int HD, int NG, bool ONE>
__global__ void __launch_bounds__(256) kv8_join_kernel(const __grid_constant__ SplitArgs s) {
    pdl_launch();
    pdl_wait();
    constexpr int ROWS = 8 * NG;
    __shared__ float s_m[ROWS], s_M[ROWS], s_l[ROWS];
    const int c0 = blockIdx.x;
    const SplitDesc d = s.desc[c0];
    if (d.row0 < 0) return;
    const int rows = d.n * s.G, parts = d.last - c0 + 1;
    // part i: the end of share c0, then the beginnings of the shares behind it
    auto slot = [&](int i) { return s.parts + (2LL * (c0 + i) + (i == 0 ? 1 : 0)) * Slot<HD, NG>::FLOATS; };
    // this thread's first columns of the first parts, on their way while the rows' maxima are found
    constexpr int AHEAD = 8;
    float2 ahead[AHEAD];
    float ahead_M[AHEAD];
    const int r0 = min((int)threadIdx.x / (HD / 2), ROWS - 1), d0 = ((int)threadIdx.x % (HD / 2)) * 2;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
        ahead[k] = make_float2(0.f, 0.f);
        ahead_M[k] = 0.f;
        if (k < parts && r0 < rows) {
            ahead[k] = *reinterpret_cast<const float2*>(slot(k) + r0 * HD + d0);
            ahead_M[k] = slot(k)[ROWS * HD + r0 * 3 + 2];
        }
    }
    for (int r = threadIdx.x >> 5; r < rows; r += 8) {
        const int lane = threadIdx.x & 31;
        float m = -INFINITY, M = -INFINITY, l = 0.f;
        for (int i = lane; i < parts; i += 32) {
            const float* q = slot(i) + ROWS * HD + r * 3;
            const float mn = fmaxf(m, q[0]);
            const float mr = mn == -INFINITY ? 0.f : mn;
            l = l * ex2(m - mr) + q[1] * ex2(q[0] - mr);
            m = mn;
            M = fmaxf(M, q[2]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
            const float mn = fmaxf(m, m2);
            const float mr = mn == -INFINITY ? 0.f : mn;
            // the lower lane's term first on both sides: every lane has the same sum
            const float x = l * ex2(m - mr), y = l2 * ex2(m2 - mr);
            l = (lane & o) ? y + x : x + y;
            m = mn;
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        }
        if (lane == 0) {
            s_m[r] = m == -INFINITY ? 0.f : m;
            s_M[r] = M == -INFINITY ? 0.f : M;
            s_l[r] = l;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (HD / 2); i += 256) {
        const int r = i / (HD / 2), dd = (i - r * (HD / 2)) * 2;
        const int qi = r / s.G, hq = r - qi * s.G;
        const float Mr = s_M[r], L = s_l[r];
        float x0 = 0.f, x1 = 0.f;
        const bool held = i < 256;
        if (held) {
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                if (k < parts) {
                    const float f = ex2(ahead_M[k] - Mr);
                    x0 += ahead[k].x * f;
                    x1 += ahead[k].y * f;
                }
            }
        }
#pragma unroll 8
        for (int k = held ? AHEAD : 0; k < parts; ++k) {
            const float* p = slot(k);
            const float2 ov = *reinterpret_cast<const float2*>(p + r * HD + dd);
            const float f = ex2(p[ROWS * HD + r * 3 + 2] - Mr);
            x0 += ov.x * f;
            x1 += ov.y * f;
        }
        const float f = L == 0.f ? 0.f : exp2f(Mr - s_m[r]) / L;
        bf16* dst = s.a.out + ((long long)(d.row0 + qi) * s.a.nq + d.head * s.G + hq) * HD + dd;
        *reinterpret_cast<uint32_t*>(dst) = pack_bf2(x0 * 0x1p-15f * f, x1 * 0x1p-15f * f);
        if (!ONE && (x0 != x0 || x1 != x1)) look_again(s, d.b, d.head, r, dd, dst);
    }
}

int split_grid() { return 3 * device_sm_count(); }

template <int HD, int NG, bool ONE, int MODE>
cudaError_t launch_ng(const SplitArgs& s, cudaStream_t st, int splits = 1) {
    constexpr int join = kWarps * 8 * NG * (HD + 3) * 4;
    constexpr int smem = (Ring<HD>::BYTES > join ? Ring<HD>::BYTES : join) + 1024;   // aligned up to 1024 bytes
    alignas(64) CUtensorMap map;
    if (!make_map_codes(&map, s.a.view.codes, 2LL * s.a.view.n_pages * s.a.view.n_kv * s.a.view.page_size, HD, kKv8Block))
        return cudaErrorInvalidValue;
    static bool configured[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(kv8_attn_kernel<HD, NG, ONE, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    if (MODE == kOwn) {
        const dim3 grid((unsigned)s.a.view.n_kv, (unsigned)(s.a.batch * s.row_tiles), (unsigned)splits);
        HRA_LAUNCH((kv8_attn_kernel<HD, NG, ONE, MODE>), grid, dim3(kWarps * 32), smem, st, map, s);
        return cudaGetLastError();
    }
    if (s.whole) {
        const dim3 grid((unsigned)s.a.view.n_kv, (unsigned)s.a.batch);
        HRA_LAUNCH((kv8_attn_kernel<HD, NG, ONE, MODE>), grid, dim3(kWarps * 32), smem, st, map, s);
        return cudaGetLastError();
    }
    const dim3 grid((unsigned)split_grid());
    HRA_LAUNCH((kv8_attn_kernel<HD, NG, ONE, MODE>), grid, dim3(kWarps * 32), smem, st, map, s);
    HRA_LAUNCH((kv8_join_kernel<HD, NG, ONE>), grid, dim3(256), 0, st, s);
    return cudaGetLastError();
}

template <int HD, int NG>
cudaError_t launch_tokens(const SplitArgs& s, cudaStream_t st) {
    if (s.a.window > 0) return s.a.max_new == 1 ? launch_ng<HD, NG, true, kWindow>(s, st) : launch_ng<HD, NG, false, kWindow>(s, st);
    return s.a.max_new == 1 ? launch_ng<HD, NG, true, kAll>(s, st) : launch_ng<HD, NG, false, kAll>(s, st);
}

// Items go whole, one a CTA, while they are short, and where the sequences do not fit the table of a CTA.
bool goes_whole(int batch, int max_len) { return max_len <= kWholeUnits * kUnit || batch > kMaxBatch; }

size_t split_scratch(const Kv8View& c, int ng) {
    const size_t grid = (size_t)split_grid();
    return grid * sizeof(SplitDesc) + grid * 2 * 8 * ng * (c.head_dim + 3) * sizeof(float);
}

}  // namespace

size_t kv8_attention_scratch_bytes(const Kv8View& c, int batch, int total_rows, int nq, int max_new, int max_len) {
    const int G = nq / c.n_kv;
    size_t n = 0;
    if ((long long)G * max_new > kShortRows) n = (kv8_prompt_scratch_bytes(c, batch, total_rows, G, max_len) + 255) & ~size_t(255);
    if (max_len > kWholeUnits * kUnit) n += split_scratch(c, column_groups(G, max_new));   // also where batch > kMaxBatch
    return n;
}

cudaError_t launch_kv8_own(const Kv8AttnArgs& a, const SharedCall& c, cudaStream_t st) {
    SplitArgs s{};
    s.a = a;
    s.G = a.nq / a.view.n_kv;
    s.parts = c.own_parts;
    s.shared = c.rows;
    s.row_tiles = c.row_tiles;
    s.own_units = c.own_units;
    const bool one = column_groups(s.G, a.max_new) == 1;
    if (a.view.head_dim == 128)
        return one ? launch_ng<128, 1, false, kOwn>(s, st, c.splits) : launch_ng<128, 2, false, kOwn>(s, st, c.splits);
    return one ? launch_ng<64, 1, false, kOwn>(s, st, c.splits) : launch_ng<64, 2, false, kOwn>(s, st, c.splits);
}

cudaError_t launch_kv8_attention(const Kv8AttnArgs& a, cudaStream_t st) {
    if (kv8_shares(a.view, a.batch, a.total_rows, a.nq, a.max_new, a.groups, a.max_prefix)) return launch_kv8_shared(a, st);
    const int G = a.nq / a.view.n_kv;
    const bool prompts = (long long)G * a.max_new > kShortRows;
    uint8_t* scratch = reinterpret_cast<uint8_t*>(a.scratch);
    if (prompts) {
        // short sequences go with the prompts unless they may hold many keys (and unless the counts say that there are none)
        const int most = kv8_most_seen(a.max_len, a.window, a.sinks, kShortRows + 2 * kKv8Block);
        const int short_rows = most > kSerialKeys && (long long)a.batch * a.max_new != a.total_rows ? kShortRows : 0;
        cudaError_t e = launch_kv8_prompt(a, short_rows, st);
        if (e != cudaSuccess || short_rows == 0) return e;
        scratch += (kv8_prompt_scratch_bytes(a.view, a.batch, a.total_rows, G, a.max_len) + 255) & ~size_t(255);
    }
    SplitArgs s{};
    s.a = a;
    s.G = G;
    s.max_rows = prompts ? kShortRows : 1 << 30;
    s.whole = goes_whole(a.batch, kv8_most_seen(a.max_len, a.window, a.sinks, kShortRows + 2 * kKv8Block)) ? 1 : 0;
    s.desc = reinterpret_cast<SplitDesc*>(scratch);
    s.parts = reinterpret_cast<float*>(scratch + split_grid() * sizeof(SplitDesc));
    const bool one = column_groups(G, a.max_new) == 1;
    if (a.view.head_dim == 128) return one ? launch_tokens<128, 1>(s, st) : launch_tokens<128, 2>(s, st);
    return one ? launch_tokens<64, 1>(s, st) : launch_tokens<64, 2>(s, st);
}

}  // namespace hra
