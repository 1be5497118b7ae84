// kv8_shared.cu -- attention of a batch whose groups of rows share the pages of a long prefix.
//
// With the positions of a row in two sets, P below its group's prefix and O behind it, softmax attention is the join
//   o = (2^(M_P - M) o_P + 2^(M_O - M) o_O) 2^(M - m) / (2^(m_P - m) l_P + 2^(m_O - m) l_O)
// of the two sets' sums (kv8_parts.cuh).  The (token, head) rows of all sequences of a group are one query tile after another
// over P, where no token is masked: K and V of the prefix leave HBM once a group and run on the tensor cores with 128 rows
// a tile (kv8_prompt.cu), while O, a few hundred positions each, goes row by row (kv8_attention.cu).  Four kernels:
//   plan    one CTA: each group's prefix in whole pages, its query tiles, and units of their key tiles, one a CTA
//   prefix  the units, each one's sums to scratch as a part
//   own     (sequence, head, split): the row's own positions, as parts
//   join    a warp a (token, head) row: its parts in order, prefix first (the last CTA of a sequence and head to do it, in the
//           place of a kernel of its own: 46 us against 43 for 46 rows in 8 groups, 78 against 76 for 64 in one, but 50 against 53 for
//           32 rows of 0-12 tokens, whose own positions are one part)
// 64 rows on 16,001 positions, 15-1000 of their own: 69 us (plan 6.5, prefix 29, own 23, join 10.5), row by row 330; 8 groups of 4-8
// rows on 1024-2112: 40 us (6.5, 16, 14, 5).  A pass plans once.  The prefix is bound by its chain of tiles, 45% of the issue slots
// and 27% of the tensor pipe; own positions and joins by latency.
#include <algorithm>
#include <math.h>

#include "kv8_parts.cuh"

namespace hra {

namespace {

// (token, head) rows of a sequence from which its own prompt tiles are at least half full: it then shares nothing.  32 rows of 8 / 12 / 16 /
// 20 / 24 / 31 tokens, 4 q heads a kv head, after 4096 shared positions 62 / 76 / 98 / 139 / 152 / 172 us, row by row 92 in all; 8 rows of
// 16 / 20 / 31 after 8192 52 / 57 / 81, row by row 54 / 56 / 61; 16 q heads, 32 rows of 4 / 5 / 8 after 8192 49 / 55 / 77, row by row 55 / 57 / 62;
// one q head, 16 rows of 32 / 64 / 80 after 4096 43 / 61 / 73, row by row 55 / 57 / 58.
constexpr int kMostRows = 64;
constexpr int kMostParts = 32;  // of a prefix: what the lanes of a joining warp look at in one turn
// Bytes of K and V that a call has to save: below them its three further kernels cost more.  8 kv heads of 128, 4 q heads each, 200
// own positions, in a graph, once a group / row by row: 16 rows after 4096 shared positions (126 MB) 35 / 33 us, after 8192 38 / 53;
// 64 after 1024 (132 MB) 38 / 39; 8 groups of 6 after 1024 (84 MB) 34 / 34, after 2048 39 / 47; 64 rows after 16384 59 / 330.
// Tokens of more than 8 rows take twice as long row by row: 16 rows of 8 tokens after 2048 (63 MB) 40 / 49.  Other heads, single tokens, once a
// group / row by row: 2 kv heads of 128, 64 rows after 4096 (126 MB) 29 / 34 us; 8 of 64 with 4 q heads, 64 rows after 1024 (63 MB) 23 / 32,
// 16 after 4096 (60 MB) 25 / 28, 4 after 16384 (48 MB) 30 / 29: with heads of 64 half as much would do.
constexpr long long kLeastSaved = 96LL << 20;
// ... and for each (token, head) row of such tokens, in units of head_dim^2 / 8, what its own positions and its join cost: 64 rows of
// 4 / 8 / 16 tokens after 1024 (252 MB, counted twice) 45 / 64 / 106 us, row by row 63 / 57 / 57, of 16 after 4096 (1008 MB) 164 / 170; with
// heads of 64 31 / 44 / 72 (126 MB), row by row 42 / 49 / 49, and 119 / 146 (504 MB).
constexpr long long kSavedARow = 5;
constexpr int kHeldRows = 1024; // rows whose lengths the plan holds in shared memory
constexpr int kOwnSplits = 8;   // most CTAs that a row's own positions are split over
// Units of 128 keys that a CTA takes of a row's own positions at least: more where the CTAs are more than the SMs hold at
// once.  The whole call with 2 / 4 units (8 kv heads of 128): 16 rows of 1000 own positions on one prefix (512 CTAs of 2) 38.8 / 40.9 us,
// 32 rows of 500 (512) 41.6 / 42.5, 8 groups of 6 with 300 (768) 38.2 / 36.9 and with 700 (1152) 49.9 / 47.3, 64 rows of 2000 (4096)
// 106 / 96.
constexpr int kFewUnits = 2, kMoreUnits = 4, kManyCtas = 4;

__global__ void __launch_bounds__(1024) kv8_shared_plan_kernel(const Kv8AttnArgs a, int QT, const SharedCall s) {
    pdl_launch();
    pdl_wait();
    __shared__ int first_s[kKv8MaxGroups + 1];   // the groups' first rows, made ascending
    __shared__ int prefix_s[kKv8MaxGroups], row0_s[kKv8MaxGroups], n_s[kKv8MaxGroups], pairs_s[kKv8MaxGroups];
    __shared__ int lead_s[kKv8MaxGroups];
    const Kv8View& c = a.view;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int room = c.max_pages << c.page_shift;
    const int threads = blockDim.x, warps = threads >> 5;
    // every array at once, where they fit: one way to memory and back
    const bool held = a.batch <= kHeldRows;
    __shared__ int cu_s[kHeldRows + 1], len_s[kHeldRows];
    if (held)
        for (int b = threadIdx.x; b <= a.batch; b += threads) {
            cu_s[b] = a.cu[b];
            if (b < a.batch) len_s[b] = a.kv_len[b];
        }
    for (int g = threadIdx.x; g <= a.groups; g += threads) {
        first_s[g] = a.group_cu[g];
        if (g < a.groups) prefix_s[g] = a.prefix[g];
    }
    for (int b = threadIdx.x; b < a.batch; b += threads) s.rows[b] = SharedRow{0, 0, 0, 0};
    const int32_t* const cu = held ? cu_s : a.cu;
    const int32_t* const kv_len = held ? len_s : a.kv_len;
    __syncthreads();
    if (warp == 0) {
        int run = 0;
        bool bad = false;
        for (int i0 = 0; i0 <= a.groups; i0 += 32) {
            const int i = i0 + lane;
            const int at = i <= a.groups ? first_s[i] : 0;
            int v = min(a.batch, max(0, at));
            bad |= i <= a.groups && v != at;
            const int mine = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v = max(v, u);
            }
            v = max(v, run);
            bad |= i <= a.groups && v != mine;
            if (i <= a.groups) first_s[i] = v;
            run = __shfl_sync(0xffffffffu, v, 31);
        }
        if (bad) raise_error(c.err, HRA_DEVERR_POS_RANGE);
    }
    __syncthreads();
    // a warp a group: no row reads more of the prefix than it holds before its new tokens
    for (int g = warp; g < a.groups; g += warps) {
        const int b0 = first_s[g], b1 = first_s[g + 1];
        int least = prefix_s[g], rows = 0, lead = a.batch;   // lead: the group's first row with new tokens
        int lo = cu[b0], hi = cu[b1];
        if (lane == 0 && least < 0) raise_error(c.err, HRA_DEVERR_POS_RANGE);
        for (int b = b0 + lane; b < b1; b += 32) {
            int row0, n;
            kv8_rows(cu, b, a.total_rows, row0, n);
            if (n > 0) {
                least = min(least, min(room, max(0, kv_len[b])) - n);
                ++rows;
                lead = min(lead, b);
            }
        }
        least = __reduce_min_sync(0xffffffffu, least);
        rows = __reduce_add_sync(0xffffffffu, rows);
        lead = __reduce_min_sync(0xffffffffu, lead);
        if (lane == 0) {
            lo = min(a.total_rows, max(0, lo));
            hi = rows > 0 ? min(a.total_rows, max(lo, hi)) : lo;
            prefix_s[g] = rows > 0 ? max(0, least) >> c.page_shift << c.page_shift : 0;
            lead_s[g] = lead;
            row0_s[g] = lo;
            n_s[g] = prefix_s[g] > 0 ? hi - lo : 0;
            pairs_s[g] = (n_s[g] + QT - 1) / QT;
        }
    }
    __syncthreads();
    // Units.  Items (query tile, kv head) of T key tiles go in parts of at most `per` tiles: a CTA that begins a second item
    // waits for its queries and writes its first one's sums (8 us of 25, measured), so as few tiles a CTA as leave one unit
    // each, or whole items where there are more of them than CTAs.
    __shared__ int unit_s[kKv8MaxGroups], parts_s[kKv8MaxGroups];
    __shared__ int total_s;
    if (warp == 0) {
        auto items_of = [&](int g) { return g < a.groups ? (long long)pairs_s[g] * c.n_kv : 0; };
        long long items = 0, tiles = 0;
        for (int g = lane; g < a.groups; g += 32) {
            items += items_of(g);
            tiles += items_of(g) * key_tiles(prefix_s[g]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            items += __shfl_xor_sync(0xffffffffu, items, o);
            tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
        }
        const long long most = max((long long)s.prefix_grid, items);
        auto count = [&](int per) {
            long long u = 0;
            for (int g = 0; g < a.groups; ++g) u += items_of(g) * ((key_tiles(prefix_s[g]) + per - 1) / per);
            return u;
        };
        // 32 sizes from equal shares on; beyond them the equal share of the CTAs that are left when each item has one, which
        // always fits
        int longest = 1;
        for (int g = lane; g < a.groups; g += 32) longest = max(longest, key_tiles(prefix_s[g]));
        longest = __reduce_max_sync(0xffffffffu, longest);
        const int whole = 1 << 24;   // more than any prefix has
        const int least = max((int)min((tiles + s.prefix_grid - 1) / s.prefix_grid, (long long)whole),
                              max(1, (longest + kMostParts - 1) / kMostParts));
        const unsigned int fits = __ballot_sync(0xffffffffu, count(least + lane) <= most);
        int per = whole;
        if (fits) per = least + __ffs(fits) - 1;
        else if (items < s.prefix_grid) per = (int)min((tiles + s.prefix_grid - items - 1) / (s.prefix_grid - items), (long long)whole);
        long long run = 0;
        for (int g0 = 0; g0 < a.groups; g0 += 32) {
            const int g = g0 + lane;
            const int parts = g < a.groups ? (key_tiles(prefix_s[g]) + per - 1) / per : 0;
            const long long mine = items_of(g) * parts;
            long long incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (g < a.groups) {
                // groups whose packed rows lie in one another's could have more units than there is room for
                if (run + incl > s.most_units) {
                    raise_error(c.err, HRA_DEVERR_POS_RANGE);
                    prefix_s[g] = 0;
                }
                unit_s[g] = (int)min(run + incl - mine, (long long)s.most_units);
                parts_s[g] = parts;
            }
            run += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) {
            total_s = (int)min(run, (long long)s.most_units);
            *s.n_units = total_s;
        }
    }
    __syncthreads();
    const int total = total_s;
    for (int u = threadIdx.x; u < max(total, s.prefix_grid); u += threads) {
        PrefixUnit unit{0, 0, 0, 0, 0, 0, 0, 0};
        if (u < total) {
            int lo = 0, hi = a.groups;   // the last group with a first unit <= u: it has units
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (unit_s[mid] <= u) lo = mid;
                else hi = mid;
            }
            const int p = parts_s[lo], keys = prefix_s[lo], all_tiles = key_tiles(keys), len = (all_tiles + p - 1) / p;
            const int item = (u - unit_s[lo]) / p, part = (u - unit_s[lo]) % p, pair = item / c.n_kv;
            if (keys > 0)
                unit = PrefixUnit{lead_s[lo], row0_s[lo], n_s[lo], pair * QT, keys, item % c.n_kv, part * len,
                                  max(0, min(len, all_tiles - part * len))};
        }
        int4* to = reinterpret_cast<int4*>(s.units + u);
        to[0] = make_int4(unit.b, unit.row0, unit.n, unit.q_lo);
        to[1] = make_int4(unit.keys, unit.head, unit.t_first, unit.count);
    }
    for (int x = warp; x < a.groups; x += warps) {
        if (prefix_s[x] == 0) continue;
        for (int b = first_s[x] + lane; b < first_s[x + 1]; b += 32) {
            int row0, n;
            kv8_rows(cu, b, a.total_rows, row0, n);
            if (n > 0 && row0 >= row0_s[x] && row0 + n <= row0_s[x] + n_s[x])
                s.rows[b] = SharedRow{prefix_s[x], unit_s[x], row0_s[x], parts_s[x]};
        }
    }
}

// A CTA a (kv head, tile of a sequence's tokens), a warp a row of it, or several that take its parts in turn: every load but the
// first few is free of the others, and the first parts are on their way while the row's maxima are found.
template <int HD, int NG>
__global__ void __launch_bounds__(256 * NG) kv8_shared_join_kernel(const Kv8AttnArgs a, int G, int QT, const SharedCall s) {
    pdl_launch();
    pdl_wait();
    constexpr int ROWS = 8 * NG, E = HD / 32, AHEAD = 8;
    const Kv8View& c = a.view;
    const int lane = threadIdx.x & 31;
    const int head = blockIdx.x, b = blockIdx.y / s.row_tiles;
    int row0, n;
    kv8_rows(a.cu, b, a.total_rows, row0, n);
    const int kv_len = min(c.max_pages << c.page_shift, max(0, a.kv_len[b]));
    const SharedRow sh = s.rows[b];
    const Kv8Own o = kv8_own(kv_len, n, blockIdx.y - b * s.row_tiles, ROWS / G, a.max_new, sh.prefix, s.splits, s.own_units);
    const int rows = o.tokens * G;
    if (rows == 0) return;
    // warps a row: one where it has all parts on their way at once (with more, 4.6 -> 5.4 us at 8 groups of 4-8 rows); several
    // where there are more parts (64 rows, 38 of a prefix of 16,001: 14 -> 10.9 us)
    const int each = (sh.prefix > 0 ? sh.parts : 0) + o.parts <= AHEAD || rows > ROWS / 2 ? 1 : rows > ROWS / 4 ? 2 : 4;
    const int r = (threadIdx.x >> 5) / each, sub = (threadIdx.x >> 5) % each;
    __shared__ float acc_s[ROWS][HD + 1];   // a warp's sums and their l
    if (r >= rows) return;   // (whole warps of rows that are not waited for)
    row0 += o.t0;
    const float* own = s.own_parts + ((long long)blockIdx.y * c.n_kv + head) * s.splits * Slot<HD, NG>::FLOATS;
    const int qi = r / G, hq = r - qi * G;
    const int parts = sh.prefix > 0 ? sh.parts : 0, x0 = row0 + qi - sh.row0, prow = (x0 % QT) * G + hq;
    const float* at = s.prefix_parts + (sh.unit0 + ((long long)(x0 / QT) * c.n_kv + head) * parts) * PromptSlot<HD>::FLOATS;
    const int count = parts + o.parts;
    // prefix sums are in units of 2^-11, the row's own of 2^-15
    auto stats = [&](int i, float& m, float& l, float& M) {
        if (i < parts) {
            const float* q = at + (long long)i * PromptSlot<HD>::FLOATS + kTileRows * HD + prow;
            m = q[0];
            l = q[kTileRows];
            M = q[2 * kTileRows];
        } else {
            const float* q = own + (long long)(i - parts) * Slot<HD, NG>::FLOATS + ROWS * HD + r * 3;
            m = q[0];
            l = q[1];
            M = q[2];
        }
    };
    auto part = [&](int k, float (&v)[E]) {
        const float* p = k < parts ? at + (long long)k * PromptSlot<HD>::FLOATS + prow * HD + lane * E
                                   : own + (long long)(k - parts) * Slot<HD, NG>::FLOATS + r * HD + lane * E;
        if constexpr (E == 4) {
            const float4 x = *reinterpret_cast<const float4*>(p);
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        } else {
            const float2 x = *reinterpret_cast<const float2*>(p);
            v[0] = x.x, v[1] = x.y;
        }
    };
    float ahead[AHEAD][E];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
        if (sub + k * each < count) part(sub + k * each, ahead[k]);
    float pm0 = -INFINITY, pl0 = 0.f, pM0 = -INFINITY;   // part `lane`'s
    if (lane < count) stats(lane, pm0, pl0, pM0);
    float m = pm0, M = pM0;
    for (int i = lane + 32; i < count; i += 32) {
        float pm, pl, pM;
        stats(i, pm, pl, pM);
        m = fmaxf(m, pm);
        M = fmaxf(M, pM);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    }
    const float mr = m == -INFINITY ? 0.f : m, Mr = M == -INFINITY ? 0.f : M;
    float L = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int i0 = 0; i0 < count; i0 += 32) {
        float f = 0.f, pl = 0.f;
        if (i0 + lane < count) {
            float pm = pm0, pM = pM0;
            pl = pl0;
            if (i0 > 0) stats(i0 + lane, pm, pl, pM);
            pl *= ex2(pm - mr);
            f = ex2(pM - Mr + (i0 + lane < parts ? kRowsUnit - kTileUnit : 0.f));
        }
        const int here = min(32, count - i0);
        auto add = [&](int i, const float (&v)[E]) {
            const float w = __shfl_sync(0xffffffffu, f, i);
            L += __shfl_sync(0xffffffffu, pl, i);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += v[e] * w;
        };
        if (i0 == 0) {
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (sub + k * each < here) add(sub + k * each, ahead[k]);
        }
#pragma unroll 4
        for (int i = sub + (i0 == 0 ? AHEAD * each : 0); i < here; i += each) {
            float v[E];
            part(i0 + i, v);
            add(i, v);
        }
    }
    if (each > 1) {   // the first warp of a row adds the others' sums, in order
        float* mine = acc_s[r * each + sub];
#pragma unroll
        for (int e = 0; e < E; ++e) mine[lane * E + e] = acc[e];
        if (lane == 0) mine[HD] = L;
        // (the row's warps alone)
        asm volatile("bar.sync %0, %1;" ::"r"(1 + r), "r"(32 * each) : "memory");
        if (sub != 0) return;
        for (int k = 1; k < each; ++k) {
            const float* other = acc_s[r * each + k];
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += other[lane * E + e];
            L += other[HD];
        }
    }
    const float f = L == 0.f ? 0.f : exp2f(Mr - mr) / L;
    bf16* dst = a.out + ((long long)(row0 + qi) * a.nq + head * G + hq) * HD + lane * E;
    bool nan = false;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        *reinterpret_cast<uint32_t*>(dst + e) = pack_bf2(acc[e] * 0x1p-15f * f, acc[e + 1] * 0x1p-15f * f);
        nan |= acc[e] != acc[e] || acc[e + 1] != acc[e + 1];
    }
    if (nan && o.tokens > 1) {   // of a later token's V, perhaps
        const bf16* q = a.q + (long long)(row0 + qi) * a.row_stride + (long long)(head * G + hq) * HD;
        kv8_row_again(c, q, b, head, kv_len - n + o.t0 + qi + 1, o.keys, lane * E, E, a.scale_log2, dst);
    }
}


int row_tiles(int G, int max_new) {
    const int tokens = 8 * column_groups(G, max_new) / G;
    return (max_new + tokens - 1) / tokens;
}
// Parts of a row's own positions, of `least` units of 128 keys while so many CTAs do.
int own_splits(int max_own, int least) {
    const long long units = std::max<long long>(1, ((long long)max_own + 127) / 128);
    return (int)std::min<long long>((units + least - 1) / least, kOwnSplits);
}
size_t up(size_t n) { return (n + 255) & ~size_t(255); }
int prefix_grid() { return 2 * device_sm_count(); }
// Packed rows of sequences of at most max_new tokens.
int most_rows(int batch, int total_rows, int max_new) { return (int)std::min<long long>(total_rows, (long long)batch * max_new); }
// Items of groups that share no packed rows: sum ceil(n / QT) <= total / QT + groups tiles a kv head.
long long most_units(const Kv8View& c, int total_rows, int G, int groups) {
    return std::max<long long>(prefix_grid(), ((long long)total_rows / (kTileRows / G) + groups) * c.n_kv);
}

}  // namespace

bool kv8_shares(const Kv8View& c, int batch, int total_rows, int nq, int max_new, int groups, int max_prefix) {
    const int G = nq / c.n_kv;
    if (groups < 1 || groups >= batch || (long long)G * max_new > kMostRows) return false;
    if (max_prefix < c.page_size || (long long)batch * row_tiles(G, max_new) > 65535) return false;
    const long long held = std::min<long long>(max_prefix, (long long)c.max_pages * c.page_size);
    const long long saved = 2LL * c.n_kv * c.head_dim * held * (batch - groups);   // bytes, if the groups are alike
    if (column_groups(G, max_new) == 1) return saved >= kLeastSaved;
    return 2 * saved >= kLeastSaved + (long long)most_rows(batch, total_rows, max_new) * nq * (c.head_dim * c.head_dim / 8 * kSavedARow);
}

size_t kv8_shared_scratch_bytes(const Kv8View& c, int batch, int total_rows, int nq, int max_new, int max_len, int groups,
                                int max_prefix, int max_own) {
    size_t n = kv8_attention_scratch_bytes(c, batch, total_rows, nq, max_new, max_len);
    if (groups < 1 || max_prefix < c.page_size) return n;
    // also for calls that then share nothing, and the most of as many or fewer heads (their tiles divide unevenly), so that the
    // size never falls
    size_t units = 0, tiles = 0;
    for (int G = 1; G <= nq / c.n_kv; ++G) {
        const int most = std::min(max_new, std::max(1, kMostRows / G));
        units = std::max(units, (size_t)most_units(c, most_rows(batch, total_rows, most), G, groups));
        tiles = std::max(tiles, (size_t)row_tiles(G, most));
    }
    const size_t slots = (size_t)batch * tiles * c.n_kv * own_splits(max_own, kFewUnits);
    n = up(n) + 512 + up(units * sizeof(PrefixUnit)) + up(batch * sizeof(SharedRow));
    n += up(4 * units * kTileRows * (c.head_dim + 3));
    return n + 4 * slots * 16 * (c.head_dim + 3);
}

cudaError_t launch_kv8_shared(const Kv8AttnArgs& a, cudaStream_t st) {
    const Kv8View& c = a.view;
    const int G = a.nq / c.n_kv, QT = kTileRows / G;
    SharedCall s{};
    s.prefix_grid = prefix_grid();
    s.most_units = (int)most_units(c, most_rows(a.batch, a.total_rows, a.max_new), G, a.groups);
    s.row_tiles = row_tiles(G, a.max_new);
    const int own = std::min(a.max_own, a.max_len);
    const long long ctas = (long long)a.batch * s.row_tiles * c.n_kv * own_splits(own, kFewUnits);
    s.own_units = ctas > kManyCtas * device_sm_count() ? kMoreUnits : kFewUnits;
    s.splits = own_splits(own, s.own_units);
    uint8_t* at = reinterpret_cast<uint8_t*>(up(reinterpret_cast<uintptr_t>(a.scratch)));
    auto take = [&](size_t n) {
        uint8_t* p = at;
        at += up(n);
        return p;
    };
    s.n_units = reinterpret_cast<int32_t*>(take(4));
    s.units = reinterpret_cast<PrefixUnit*>(take(s.most_units * sizeof(PrefixUnit)));
    s.rows = reinterpret_cast<SharedRow*>(take(a.batch * sizeof(SharedRow)));
    s.prefix_parts = reinterpret_cast<float*>(take(4ull * s.most_units * kTileRows * (c.head_dim + 3)));
    s.own_parts = reinterpret_cast<float*>(at);
    if (!a.planned) HRA_LAUNCH(kv8_shared_plan_kernel, dim3(1), dim3(a.batch <= 256 && a.groups <= 64 ? 256 : 1024), 0, st, a, QT, s);
    cudaError_t e = launch_kv8_prefix(a, s, st);
    if (e != cudaSuccess) return e;
    e = launch_kv8_own(a, s, st);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)c.n_kv, (unsigned)(a.batch * s.row_tiles));
    const bool one = column_groups(G, a.max_new) == 1;
    if (c.head_dim == 128) {
        if (one) HRA_LAUNCH((kv8_shared_join_kernel<128, 1>), grid, dim3(256), 0, st, a, G, QT, s);
        else HRA_LAUNCH((kv8_shared_join_kernel<128, 2>), grid, dim3(512), 0, st, a, G, QT, s);
    } else {
        if (one) HRA_LAUNCH((kv8_shared_join_kernel<64, 1>), grid, dim3(256), 0, st, a, G, QT, s);
        else HRA_LAUNCH((kv8_shared_join_kernel<64, 2>), grid, dim3(512), 0, st, a, G, QT, s);
    }
    return cudaGetLastError();
}

}  // namespace hra
