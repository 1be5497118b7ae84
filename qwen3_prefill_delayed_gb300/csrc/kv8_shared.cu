// kv8_shared.cu -- attention of a batch whose groups of rows share the pages of a long prefix.
//
// With the positions of a row in two sets, P below its group's prefix and O behind it, softmax attention is the join
//   o = (2^(M_P - M) o_P + 2^(M_O - M) o_O) 2^(M - m) / (2^(m_P - m) l_P + 2^(m_O - m) l_O)
// of the two sets' sums (kv8_parts.cuh).  The (token, head) rows of all sequences of a group are one query tile after another
// over P, where no token is masked: K and V of the prefix leave HBM once a group and run on the tensor cores with 128 rows
// a tile (kv8_prompt.cu), while O, a few hundred positions each, goes row by row (kv8_attention.cu).  Four kernels:
//   plan    one CTA: each group's prefix in whole pages, its query tiles, and the tiles' place in the line of all key tiles
//   prefix  equal shares of that line; every item's sums go to scratch as parts
//   own     (sequence, head, split): the row's own positions, as parts
//   join    a warp a (token, head) row: its parts in order, prefix first
#include <algorithm>
#include <math.h>

#include "kv8_parts.cuh"

namespace hra {

namespace {

// (token, head) rows of a sequence from which its own prompt tiles are at least half full: it then shares nothing
constexpr int kMostRows = 64;
constexpr int kOwnCtas = 3;    // CTAs an SM of the kernel over the rows' own positions

__global__ void __launch_bounds__(1024) kv8_shared_plan_kernel(const Kv8AttnArgs a, int QT, const SharedCall s) {
    pdl_launch();
    pdl_wait();
    __shared__ int first_s[kKv8MaxGroups + 1];   // the groups' first rows, made ascending
    __shared__ int prefix_s[kKv8MaxGroups], row0_s[kKv8MaxGroups], n_s[kKv8MaxGroups];
    const Kv8View& c = a.view;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int room = c.max_pages << c.page_shift;
    for (int b = threadIdx.x; b < a.batch; b += 1024) s.rows[b] = SharedRow{0, 0, 0, 0};
    if (warp == 0) {
        int run = 0;
        bool bad = false;
        for (int i0 = 0; i0 <= a.groups; i0 += 32) {
            const int i = i0 + lane;
            const int at = i <= a.groups ? a.group_cu[i] : 0;
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
    for (int g = warp; g < a.groups; g += 32) {
        const int b0 = first_s[g], b1 = first_s[g + 1];
        int least = a.prefix[g], rows = 0;
        if (lane == 0 && least < 0) raise_error(c.err, HRA_DEVERR_POS_RANGE);
        for (int b = b0 + lane; b < b1; b += 32) {
            int row0, n;
            kv8_rows(a.cu, b, a.total_rows, row0, n);
            if (n > 0) {
                least = min(least, min(room, max(0, a.kv_len[b])) - n);
                ++rows;
            }
        }
        least = __reduce_min_sync(0xffffffffu, least);
        rows = __reduce_add_sync(0xffffffffu, rows);
        if (lane == 0) {
            int lo = 0, hi = 0;
            if (rows > 0) {
                lo = min(a.total_rows, max(0, a.cu[b0]));
                hi = min(a.total_rows, max(lo, a.cu[b1]));
            }
            prefix_s[g] = max(0, least) >> c.page_shift << c.page_shift;
            row0_s[g] = lo;
            n_s[g] = prefix_s[g] > 0 ? hi - lo : 0;
        }
    }
    __syncthreads();
    // pairs of the groups before, and their tiles; enough of both for groups that share no packed rows
    __shared__ int pair_s[kKv8MaxGroups], pairs_s[kKv8MaxGroups];
    __shared__ long long before_s[kKv8MaxGroups];
    const int g = threadIdx.x;
    const bool in = g < a.groups;
    int all;
    const int want = in ? (n_s[g] + QT - 1) / QT : 0;
    const int at = min(s.most_pairs, block_scan(want, all));
    const int mine = min(want, s.most_pairs - at);
    if (threadIdx.x == 0 && all > s.most_pairs) raise_error(c.err, HRA_DEVERR_POS_RANGE);
    long long tiles;
    const long long before = block_scan((long long)mine * (in ? key_tiles(prefix_s[g]) : 0), tiles);
    if (in) {
        pair_s[g] = at;
        pairs_s[g] = mine;
        before_s[g] = before * c.n_kv;
    }
    if (threadIdx.x == 0) {
        s.list[0] = min(all, s.most_pairs);
        *reinterpret_cast<long long*>(s.list + 2) = tiles * c.n_kv;
    }
    __syncthreads();
    for (int x = warp; x < a.groups; x += 32) {
        const int b0 = first_s[x], b1 = first_s[x + 1], keys = prefix_s[x], T = key_tiles(keys);
        for (int p = lane; p < pairs_s[x]; p += 32) {
            const long long line = before_s[x] + (long long)p * T * c.n_kv;
            int4* to = reinterpret_cast<int4*>(s.list + kRecWords * (1 + (long long)(pair_s[x] + p)));
            to[0] = make_int4(b0, row0_s[x], n_s[x], p * QT);
            to[1] = make_int4(keys, keys, (int)(line & 0xFFFFFFFFll), (int)(line >> 32));
        }
        const int end = row0_s[x] + min(n_s[x], pairs_s[x] * QT);
        for (int b = b0 + lane; b < b1; b += 32) {
            int row0, n;
            kv8_rows(a.cu, b, a.total_rows, row0, n);
            if (n > 0 && row0 >= row0_s[x] && row0 + n <= end) s.rows[b] = SharedRow{keys, pair_s[x], row0_s[x], T};
        }
    }
}

// A CTA a (kv head, tile of a sequence's tokens), a warp a row of it.
template <int HD, int NG>
__global__ void __launch_bounds__(128) kv8_shared_join_kernel(const Kv8AttnArgs a, int G, int QT, const SharedCall s) {
    pdl_launch();
    pdl_wait();
    constexpr int ROWS = 8 * NG, E = HD / 32;
    const Kv8View& c = a.view;
    const int head = blockIdx.x, b = blockIdx.y / s.row_tiles, tile = blockIdx.y - b * s.row_tiles;
    int row0, n;
    kv8_rows(a.cu, b, a.total_rows, row0, n);
    const int kv_len = min(c.max_pages << c.page_shift, max(0, a.kv_len[b]));
    const SharedRow sh = s.rows[b];
    const Kv8Own o = kv8_own(kv_len, n, tile, ROWS / G, a.max_new, sh.prefix, s.splits);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float* own = s.own_parts + ((long long)blockIdx.y * c.n_kv + head) * s.splits * Slot<HD, NG>::FLOATS;
    const long long all = *reinterpret_cast<const long long*>(s.list + 2);
    const long long share = (all + s.prefix_grid - 1) / s.prefix_grid;
    for (int r = warp; r < o.tokens * G; r += 4) {
        const int qi = r / G, hq = r - qi * G;
        // the prefix's parts: the end of a share, then the beginnings of the ones behind it; or the item's own slot
        int parts = 0, prow = 0;
        long long c0 = 0, item = 0;
        if (sh.prefix > 0) {
            const int x = row0 + o.t0 + qi - sh.row0, pair = sh.pair0 + x / QT;
            prow = (x % QT) * G + hq;
            item = (long long)pair * c.n_kv + head;
            const long long u = *reinterpret_cast<const long long*>(s.list + kRecWords * (1 + (long long)pair) + 6) + (long long)head * sh.tiles;
            c0 = u / share;
            parts = (int)((u + sh.tiles - 1) / share - c0) + 1;
        }
        auto slot = [&](int i) {
            const long long k = parts == 1 ? 2LL * s.prefix_grid + item : 2 * (c0 + i) + (i == 0 ? 1 : 0);
            return s.prefix_parts + k * PromptSlot<HD>::FLOATS;
        };
        const int count = parts + o.parts;
        // the parts' m, l and M; prefix sums are in units of 2^-11, the row's own of 2^-15
        auto stats = [&](int i, float& m, float& l, float& M) {
            if (i < parts) {
                const float* q = slot(i) + kTileRows * HD + prow;
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
        float m = -INFINITY, M = -INFINITY;
        for (int i = lane; i < count; i += 32) {
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
                float pm, pM;
                stats(i0 + lane, pm, pl, pM);
                pl *= ex2(pm - mr);
                f = ex2(pM - Mr + (i0 + lane < parts ? kRowsUnit - kTileUnit : 0.f));
            }
            const int here = min(32, count - i0);
#pragma unroll 8
            for (int i = 0; i < here; ++i) {   // in order, so that the sums are the same at every call
                const int k = i0 + i;
                const float* p = k < parts ? slot(k) + prow * HD : own + (long long)(k - parts) * Slot<HD, NG>::FLOATS + r * HD;
                const float w = __shfl_sync(0xffffffffu, f, i);
                L += __shfl_sync(0xffffffffu, pl, i);
                alignas(16) float v[E];
                if constexpr (E == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(p + lane * E);
                else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(p + lane * E);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += v[e] * w;
            }
        }
        const float f = L == 0.f ? 0.f : exp2f(Mr - mr) / L;
        bf16* dst = a.out + ((long long)(row0 + o.t0 + qi) * a.nq + head * G + hq) * HD + lane * E;
        bool nan = false;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            *reinterpret_cast<uint32_t*>(dst + e) = pack_bf2(acc[e] * 0x1p-15f * f, acc[e + 1] * 0x1p-15f * f);
            nan |= acc[e] != acc[e] || acc[e + 1] != acc[e + 1];
        }
        if (nan && o.tokens > 1) {   // of a later token's V, perhaps
            const bf16* q = a.q + (long long)(row0 + o.t0 + qi) * a.row_stride + (long long)(head * G + hq) * HD;
            kv8_row_again(c, q, b, head, kv_len - n + o.t0 + qi + 1, o.keys, lane * E, E, a.scale_log2, dst);
        }
    }
}

int row_tiles(int G, int max_new) {
    const int tokens = 8 * column_groups(G, max_new) / G;
    return (max_new + tokens - 1) / tokens;
}
// Splits of a row's own positions: CTAs for the whole GPU, but units of 128 keys at least.
int own_splits(long long ctas, int max_own) {
    const long long fill = (kOwnCtas * (long long)device_sm_count() + ctas - 1) / ctas;
    const long long units = std::max<long long>(1, ((long long)max_own + 127) / 128);
    return (int)std::max<long long>(1, std::min({fill, units, 16LL}));
}
size_t up(size_t n) { return (n + 255) & ~size_t(255); }
long long most_pairs(int total_rows, int G, int groups) { return (long long)total_rows / (kTileRows / G) + groups; }

}  // namespace

bool kv8_shares(const Kv8View& c, int batch, int nq, int max_new, int groups, int max_prefix) {
    const int G = nq / c.n_kv;
    return groups > 0 && groups < batch && (long long)G * max_new <= kMostRows && max_prefix >= c.page_size &&
           (long long)batch * row_tiles(G, max_new) <= 65535;
}

size_t kv8_shared_scratch_bytes(const Kv8View& c, int batch, int total_rows, int nq, int max_new, int max_len, int groups,
                                int max_prefix, int max_own) {
    (void)max_own;   // splits are bounded by what fills the GPU
    size_t n = kv8_attention_scratch_bytes(c, batch, total_rows, nq, max_new, max_len);
    if (groups < 1 || max_prefix < c.page_size) return n;
    // also for calls that then share nothing, so that the size never falls
    const int G = nq / c.n_kv, most = std::min(max_new, std::max(1, kMostRows / G));
    const long long pairs = most_pairs(total_rows, G, groups);
    const long long slots = (long long)batch * row_tiles(G, most) * c.n_kv + 2LL * kOwnCtas * device_sm_count();
    n = up(n) + up(4 * kRecWords * (pairs + 1)) + up(batch * sizeof(SharedRow));
    n += 4 * (2LL * 2 * device_sm_count() + pairs * c.n_kv) * kTileRows * (c.head_dim + 3);
    return up(n) + 4 * slots * 16 * (c.head_dim + 3);
}

cudaError_t launch_kv8_shared(const Kv8AttnArgs& a, cudaStream_t st) {
    const Kv8View& c = a.view;
    const int G = a.nq / c.n_kv, QT = kTileRows / G;
    SharedCall s{};
    s.prefix_grid = 2 * device_sm_count();
    s.row_tiles = row_tiles(G, a.max_new);
    s.splits = own_splits((long long)a.batch * s.row_tiles * c.n_kv, std::min(a.max_own, a.max_len));
    s.most_pairs = (int)most_pairs(a.total_rows, G, a.groups);
    uint8_t* at = reinterpret_cast<uint8_t*>(a.scratch);
    auto take = [&](size_t n) {
        uint8_t* p = at;
        at += up(n);
        return p;
    };
    s.list = reinterpret_cast<int32_t*>(take(4 * kRecWords * ((size_t)s.most_pairs + 1)));
    s.rows = reinterpret_cast<SharedRow*>(take(a.batch * sizeof(SharedRow)));
    s.prefix_parts = reinterpret_cast<float*>(
        take(4 * (2ull * s.prefix_grid + (size_t)s.most_pairs * c.n_kv) * kTileRows * (c.head_dim + 3)));
    s.own_parts = reinterpret_cast<float*>(at);
    HRA_LAUNCH(kv8_shared_plan_kernel, dim3(1), dim3(1024), 0, st, a, QT, s);
    cudaError_t e = launch_kv8_prefix(a, s, st);
    if (e != cudaSuccess) return e;
    e = launch_kv8_own(a, s, st);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)c.n_kv, (unsigned)(a.batch * s.row_tiles));
    const bool one = column_groups(G, a.max_new) == 1;
    if (c.head_dim == 128) {
        if (one) HRA_LAUNCH((kv8_shared_join_kernel<128, 1>), grid, dim3(128), 0, st, a, G, QT, s);
        else HRA_LAUNCH((kv8_shared_join_kernel<128, 2>), grid, dim3(128), 0, st, a, G, QT, s);
    } else {
        if (one) HRA_LAUNCH((kv8_shared_join_kernel<64, 1>), grid, dim3(128), 0, st, a, G, QT, s);
        else HRA_LAUNCH((kv8_shared_join_kernel<64, 2>), grid, dim3(128), 0, st, a, G, QT, s);
    }
    return cudaGetLastError();
}

}  // namespace hra
