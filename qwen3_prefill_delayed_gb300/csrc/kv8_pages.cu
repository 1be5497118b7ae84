// kv8_pages.cu -- the pages of the 8-bit cache: rows forked, reordered, freed and extended, and the
// pool compacted.
//
// update: new row b is a copy of old row parents[b] (-1: empty).  A page whose page_size tokens are all
//   filled is never written again, so copies of a row share it and its count in refs goes up.  The pages
//   behind (the part-filled one and those reserved) belong to one row: of the rows with one parent the
//   lowest keeps them, the others get fresh pages and the part-filled one is copied in every layer.
//   Pages that no new row lists are free; rows then get fresh pages for room[b] more tokens.  Fresh pages
//   are the lowest-numbered free ones, in (row, index) order, so the result is one function of the
//   inputs.  When too few are free, or a row's table is too short, nothing changes at all.
//   Where a window bounds what is seen, the pages of a row that no later token sees are dropped before all this: the row
//   neither keeps them nor needs fresh ones in their place.
// compact: with U pages in use, the i-th used page with number >= U (ascending) moves to the i-th free
//   page with number < U.  Sources and destinations are disjoint, so the copies need no order.
//
// A plan kernel of one CTA, or a cluster of eight for large tables and pools, works out the tables in scratch; the copy
// kernel then moves the pages (16-byte copies, persistent over (move, layer, part) items) and brings the tables out,
// which is why the outputs may be the inputs.
#include <algorithm>

#include "kv8_device.cuh"

namespace hra {

namespace {

constexpr int kPlanThreads = 1024;   // what block_scan takes
constexpr int kPart = 16384;   // bytes of one copy item
constexpr int kRun = 8;        // pages a thread takes at once
constexpr int kCells = 4;      // table cells a lane has in flight
constexpr int kTeam = 8;       // CTAs of a large plan
// Table cells + pages from which an update's plan takes a cluster, and pages from which a compaction's does.  In a captured
// graph, one CTA against eight: update of 64 x 128 cells, 10,000 pages 11.7 / 12.7 us; 64 x 256, 20,000 13.0 / 13.0; 256 x
// 2048, 300,000 239 / 49; compaction of 4,096 pages 9.3 / 10.5 us; 10,000 16.8 / 11.0; 300,000 362 / 64.
constexpr long long kTeamFrom = 1LL << 15;
constexpr int kTeamPages = 5120;

constexpr int kHead = 4 + 2 * kTeam;

// Scratch of both operations, in 4-byte words.
struct PlanScratch {
    int32_t* head;     // [0] moves, [1] 1 = write the outputs; of a cluster: [2] a row too long, [3] pages needed,
                       // [4 + r], [12 + r] counts of CTA r's pages
    int32_t* first;    // [rows] lowest child of each old row
    int32_t* base;     // [rows + 1] fresh pages before each row
    int32_t* lens;     // [rows]
    int32_t* refs;     // [n_pages]
    int32_t* list;     // [n_pages] free pages in order (update), new number of each page (compact)
    int2* moves;       // [max(rows, n_pages)]
    int32_t* table;    // [rows][max_pages]
    __host__ __device__ PlanScratch(void* p, int rows, int n_pages) {
        head = reinterpret_cast<int32_t*>(p);
        moves = reinterpret_cast<int2*>(head + kHead);
        const int mv = rows > n_pages ? rows : n_pages;
        first = head + kHead + 2 * mv;
        base = first + rows;
        lens = base + rows + 1;
        refs = lens + rows;
        list = refs + n_pages;
        table = list + n_pages;
    }
};
// What one CTA's update keeps in shared memory instead: first, base, lens, refs and list, and the rows' parents.
size_t one_cta_bytes(int rows, int n_pages) { return 4 * (4 * (size_t)rows + 2 * (size_t)n_pages); }
constexpr size_t kOneCtaMost = 200 * 1024;

// The CTAs of a plan: CS of them, one cluster.
template <int CS>
struct Team {
    int rank = CS == 1 ? 0 : (int)cta_rank_in_cluster();
    int tid = rank * kPlanThreads + (int)threadIdx.x;
    static constexpr int kThreads = CS * kPlanThreads, kWarps = kThreads / 32;
    __device__ void sync() const {
        if (CS == 1) __syncthreads();
        else cluster_barrier_sync();
    }
    // this CTA's pages
    __device__ int page_lo(int n) const { return (int)((long long)n * rank / CS); }
    __device__ int page_hi(int n) const { return (int)((long long)n * (rank + 1) / CS); }
    // each CTA's count, published and (after a sync) summed below this one and in all
    __device__ void publish(int32_t* at, int v) const {
        if (CS > 1 && threadIdx.x == 0) at[rank] = v;
    }
    __device__ void sums(const int32_t* at, int& below, int& all) const {
        below = all = 0;
        for (int r = 0; r < CS; ++r) {
            const int v = at[r];
            below += r < rank ? v : 0;
            all += v;
        }
    }
};

// WINDOW: pages that no later token sees are dropped (looked for in every update, that takes 0.6 us of 16)
template <int CS, bool WINDOW>
__global__ void __launch_bounds__(kPlanThreads) kv8_update_plan_kernel(const Kv8PagesArgs a) {
    pdl_launch();
    pdl_wait();
    PlanScratch s(a.scratch, a.rows, a.n_pages);
    const Team<CS> team;
    __shared__ unsigned int bad;
    __shared__ int moved;   // one CTA's moves
    extern __shared__ int32_t words[];
    int32_t* const refs_out = s.refs;
    int32_t* const lens_out = s.lens;
    int32_t* const parents = words;
    if (CS == 1) {
        s.first = words + a.rows;
        s.base = s.first + a.rows;
        s.lens = s.base + a.rows;
        s.refs = s.lens + a.rows;
        s.list = s.refs + a.n_pages;
    }
    const int warp = team.tid >> 5, lane = threadIdx.x & 31;
    const int R = a.rows, W = a.max_pages, P = 1 << a.page_shift;
    if (threadIdx.x == 0) {
        bad = 0u;
        moved = 0;
    }
    if (team.tid == 0) {
        s.head[0] = 0;
        s.head[1] = 1;
        s.head[2] = 0;
    }
    for (int p = team.tid; p < a.n_pages; p += team.kThreads) s.refs[p] = 0;
    for (int b = team.tid; b < R; b += team.kThreads) s.first[b] = R;
    team.sync();
    auto parent = [&](int b) {
        if (CS == 1) return parents[b];
        const int p = a.parents ? a.parents[b] : b;
        return p >= 0 && p < R ? p : -1;
    };
    for (int b = team.tid; b < R; b += team.kThreads) {
        int p = a.parents ? a.parents[b] : b;
        if (p < 0 || p >= R) p = -1;
        if (CS == 1) parents[b] = p;
        if (p < 0 && a.parents[b] != -1) atomicOr(&bad, HRA_DEVERR_PARENT_RANGE);
        int len = 0;
        if (p >= 0) {
            atomicMin(&s.first[p], b);
            len = a.lens[p];
            if (len < 0 || len > ((long long)W << a.page_shift)) {
                atomicOr(&bad, HRA_DEVERR_POS_RANGE);
                len = 0;
            }
        }
        s.lens[b] = len;
        if (CS == 1) lens_out[b] = len;
    }
    team.sync();
    // the row's old pages i0 + 32 c + lane, -1 where there is none or (wrong) it is no page of the pool
    auto old_pages = [&](int p, int i0, int (&old)[kCells], bool& wrong) {
#pragma unroll
        for (int c = 0; c < kCells; ++c) {
            const int i = i0 + 32 * c + lane;
            old[c] = p >= 0 && i < W ? a.table[(long long)p * W + i] : -1;
        }
#pragma unroll
        for (int c = 0; c < kCells; ++c) {
            if (old[c] >= a.n_pages || old[c] < -1) {
                wrong = true;
                old[c] = -1;
            }
        }
    };
    // pages [gone_lo, gone_hi) of a row of `len` positions: behind the window of every later token and no sinks
    const int gone_lo = WINDOW ? (int)(((long long)a.sinks + P - 1) >> a.page_shift) : 0;
    auto gone_hi = [&](int len) { return WINDOW && len >= a.window ? (len - a.window + 1) >> a.page_shift : 0; };
    // the pages each new row keeps, and how many fresh ones it needs: one warp a row
    bool too_long = false, wrong = false;
    for (int b = warp; b < R; b += team.kWarps) {
        const int p = parent(b), len = s.lens[b];
        const int more = p >= 0 && a.room ? max(0, a.room[b]) : 0;
        const long long ends = ((long long)len + more + P - 1) >> a.page_shift;
        const bool heir = p >= 0 && s.first[p] == b;
        const int gone = gone_hi(len);
        too_long |= p >= 0 && ends > W;
        int need = 0;
        for (int i0 = 0; i0 < W; i0 += 32 * kCells) {
            int old[kCells];
            old_pages(p, i0, old, wrong);
#pragma unroll
            for (int c = 0; c < kCells; ++c) {
                const int i = i0 + 32 * c + lane;
                const bool out = WINDOW && i >= gone_lo && i < gone;
                const bool keep = !out && old[c] >= 0 && (heir || i < (len >> a.page_shift));
                if (keep) atomicAdd(&s.refs[old[c]], 1);
                need += __popc(__ballot_sync(0xffffffffu, p >= 0 && i < ends && i < W && !keep && !out));
            }
        }
        if (lane == 0) s.base[b] = need;
    }
    if (wrong) atomicOr(&bad, HRA_DEVERR_PAGE_RANGE);
    bool fail_long = __syncthreads_or(too_long);
    if (CS > 1 && fail_long && threadIdx.x == 0) atomicOr(&s.head[2], 1);
    if (CS > 1) team.sync();
    int need_all = 0, free_all = 0;
    if (team.rank == 0) {
        for (int b0 = 0; b0 < R; b0 += kPlanThreads) {
            const int b = b0 + (int)threadIdx.x;
            int total;
            const int at = block_scan(b < R ? s.base[b] : 0, total);
            if (b < R) s.base[b] = need_all + at;
            need_all += total;
        }
        if (CS > 1 && threadIdx.x == 0) s.head[3] = need_all;
    }
    // the free pages from `lo` on, in order, from place `at` of the list on, until there are enough (or only counted)
    auto free_pages = [&](int lo, int hi, int at, int enough, bool write) {
        for (int p0 = lo; p0 < hi && at < enough; p0 += kRun * kPlanThreads) {
            const int p = p0 + kRun * (int)threadIdx.x;
            unsigned int free_here = 0u;
#pragma unroll
            for (int e = 0; e < kRun; ++e)
                if (p + e < hi && s.refs[p + e] == 0) free_here |= 1u << e;
            int total;
            int to = at + block_scan(__popc(free_here), total);
#pragma unroll
            for (int e = 0; e < kRun; ++e)
                if (free_here >> e & 1u) {
                    if (write) s.list[to] = p + e;
                    ++to;
                }
            at += total;
        }
        return at;
    };
    const int lo = team.page_lo(a.n_pages), hi = team.page_hi(a.n_pages);
    if (CS == 1) {
        free_all = free_pages(0, a.n_pages, 0, need_all, true);
    } else {
        team.publish(s.head + 4, free_pages(lo, hi, 0, 1 << 30, false));
        team.sync();
        int below;
        team.sums(s.head + 4, below, free_all);
        need_all = s.head[3];
        fail_long = s.head[2] != 0;
        (void)free_pages(lo, hi, below, need_all, true);
    }
    const bool fail = fail_long || need_all > free_all;
    team.sync();
    if (!fail) {
        for (int b = warp; b < R; b += team.kWarps) {
            const int p = parent(b), len = s.lens[b];
            const int more = p >= 0 && a.room ? max(0, a.room[b]) : 0;
            const long long ends = ((long long)len + more + P - 1) >> a.page_shift;
            const bool heir = p >= 0 && s.first[p] == b;
            const int gone = gone_hi(len);
            int at = s.base[b];
            for (int i0 = 0; i0 < W; i0 += 32 * kCells) {
                int old[kCells];
                old_pages(p, i0, old, wrong);
#pragma unroll
                for (int c = 0; c < kCells; ++c) {
                    const int i = i0 + 32 * c + lane;
                    const bool out = WINDOW && i >= gone_lo && i < gone;
                    const bool keep = !out && old[c] >= 0 && (heir || i < (len >> a.page_shift));
                    const bool fresh = p >= 0 && i < ends && i < W && !keep && !out;
                    const unsigned int mask = __ballot_sync(0xffffffffu, fresh);
                    int now = keep ? old[c] : -1;
                    if (fresh) {
                        now = s.list[at + __popc(mask & ((1u << lane) - 1u))];
                        s.refs[now] = 1;
                        if (old[c] >= 0 && ((long long)i << a.page_shift) < len)
                            s.moves[atomicAdd(CS == 1 ? &moved : &s.head[0], 1)] = make_int2(old[c], now);
                    }
                    at += __popc(mask);
                    if (i < W) s.table[(long long)b * W + i] = now;
                }
            }
        }
    } else if (team.tid == 0) {
        s.head[1] = 0;
    }
    if (CS == 1) {
        __syncthreads();
        for (int p = threadIdx.x; p < a.n_pages; p += kPlanThreads) refs_out[p] = s.refs[p];
    }
    if (threadIdx.x == 0) {
        if (CS == 1) s.head[0] = moved;
        if (fail) bad |= HRA_DEVERR_PAGES_SPENT;
        if (bad) raise_error(a.err, bad);
    }
}

// One CTA (RUN pages a thread at once, its moves in shared memory) or a cluster.
template <int CS, int RUN>
__global__ void __launch_bounds__(kPlanThreads) kv8_compact_plan_kernel(const Kv8PagesArgs a) {
    pdl_launch();
    pdl_wait();
    const PlanScratch s(a.scratch, a.rows, a.n_pages);
    const Team<CS> team;
    __shared__ int2 moves_s[CS == 1 ? kTeamPages / 2 + 1 : 1];
    int2* const moves_at = CS == 1 ? moves_s : s.moves;
    const int lo = team.page_lo(a.n_pages), hi = team.page_hi(a.n_pages);
    int used = 0;
    for (int p0 = lo; p0 < hi; p0 += RUN * kPlanThreads)
#pragma unroll
        for (int e = 0; e < RUN; ++e) {   // in any order: neighbours to neighbouring threads
            const int p = p0 + e * kPlanThreads + (int)threadIdx.x;
            used += p < hi && a.refs[p] > 0 ? 1 : 0;
        }
    int U;
    (void)block_scan(used, U);
    if (CS > 1) {
        int below;
        team.publish(s.head + 4, U);
        team.sync();
        team.sums(s.head + 4, below, U);
        team.sync();   // the words are written again
    }
    // holes: .y of moves; movers: .x
    auto walk = [&](int& holes, int& movers, bool write) {
        for (int p0 = lo; p0 < hi; p0 += RUN * kPlanThreads) {
            const int p = p0 + RUN * (int)threadIdx.x;
            int r[RUN], mine = 0;
#pragma unroll
            for (int e = 0; e < RUN; ++e) r[e] = p + e < hi ? a.refs[p + e] : 0;
#pragma unroll
            for (int e = 0; e < RUN; ++e)
                if (p + e < hi) mine += p + e < U ? (r[e] <= 0 ? 1 : 0) : (r[e] > 0 ? 1 << 16 : 0);
            int total;
            const int at = block_scan(mine, total);
            int h = holes + (at & 0xFFFF), m = movers + (at >> 16);
#pragma unroll
            for (int e = 0; e < RUN; ++e) {
                if (!write || p + e >= hi) continue;
                if (p + e < U && r[e] <= 0) moves_at[h++].y = p + e;
                if (p + e >= U && r[e] > 0) moves_at[m++].x = p + e;
                s.list[p + e] = p + e;
                s.refs[p + e] = p + e < U ? max(r[e], 0) : 0;
            }
            holes += total & 0xFFFF;
            movers += total >> 16;
        }
    };
    static_assert(RUN * kPlanThreads < 1 << 15, "two counts in one word");
    int holes = 0, movers = 0;
    if (CS > 1) {
        walk(holes, movers, false);
        team.publish(s.head + 4, holes);
        team.publish(s.head + 4 + kTeam, movers);
        team.sync();
        int all;
        team.sums(s.head + 4, holes, all);
        team.sums(s.head + 4 + kTeam, movers, all);
    }
    walk(holes, movers, true);
    team.sync();
    int moves = movers;
    if (CS > 1) {
        int below;
        team.sums(s.head + 4 + kTeam, below, moves);
    }
    for (int i = team.tid; i < moves; i += team.kThreads) {
        const int2 mv = moves_at[i];
        if (CS == 1) s.moves[i] = mv;
        s.list[mv.x] = mv.y;
        s.refs[mv.y] = a.refs[mv.x];
    }
    if (team.tid == 0) {
        s.head[0] = moves;
        s.head[1] = 1;
    }
}

// The moves of the plan in every layer, and the plan's tables to the outputs (or, when the plan failed, the inputs).
// A compaction's table is the old one with each page's new number: a cell depends on itself alone.
template <bool COMPACT>
__global__ void __launch_bounds__(256) kv8_copy_kernel(const Kv8PagesArgs a) {
    pdl_launch();
    pdl_wait();
    const PlanScratch s(a.scratch, a.rows, a.n_pages);
    const int tid = threadIdx.x;
    const long long t0 = (long long)blockIdx.x * blockDim.x + tid, step = (long long)gridDim.x * blockDim.x;
    const bool ok = s.head[1] != 0;
    const long long cells = (long long)a.rows * a.max_pages;
    if (COMPACT) {
        bool wrong = false;
        for (long long i = t0; i < cells; i += step) {
            const int p = a.table[i];
            const bool in = p >= 0 && p < a.n_pages;
            wrong |= !in && p != -1;
            a.table_out[i] = in ? s.list[p] : p;
        }
        if (wrong) raise_error(a.err, HRA_DEVERR_PAGE_RANGE);
    } else {
        for (long long i = t0; i < cells; i += step) a.table_out[i] = ok ? s.table[i] : a.table[i];
    }
    for (long long i = t0; i < a.rows; i += step) a.lens_out[i] = ok && !COMPACT ? s.lens[i] : a.lens[i];
    for (long long i = t0; i < a.n_pages; i += step) a.refs_out[i] = ok ? s.refs[i] : a.refs[i];
    const int moves = s.head[0];
    const int parts = (int)((a.code_page + kPart - 1) / kPart);
    const long long items = (long long)moves * a.n_layers * parts;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int part = (int)(it % parts);
        const long long ml = it / parts;
        const int layer = (int)(ml % a.n_layers);
        const int2 mv = s.moves[ml / a.n_layers];
        const long long lay = (long long)layer * a.n_pages;
        const int bytes = (int)min((long long)kPart, a.code_page - (long long)part * kPart);
        const uint4* src = reinterpret_cast<const uint4*>(a.codes + (lay + mv.x) * a.code_page + (long long)part * kPart);
        uint4* dst = reinterpret_cast<uint4*>(a.codes + (lay + mv.y) * a.code_page + (long long)part * kPart);
        const int n16 = bytes >> 4;
        uint4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (q * 256 + tid < n16) v[q] = src[q * 256 + tid];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (q * 256 + tid < n16) dst[q * 256 + tid] = v[q];
        if (part == 0) {
            const float* sp = a.scales + (lay + mv.x) * a.scale_page;
            float* dp = a.scales + (lay + mv.y) * a.scale_page;
            for (int i = tid; i < a.scale_page; i += 256) dp[i] = sp[i];
        }
    }
}

static_assert(kPart == 4 * 256 * 16, "four 16-byte pieces a thread");

template <bool COMPACT>
cudaError_t launch_copy(const Kv8PagesArgs& a, int most_moves, cudaStream_t st) {
    const long long parts = (a.code_page + kPart - 1) / kPart;
    const long long items = (long long)most_moves * a.n_layers * parts;
    const long long tables = ((long long)a.rows * a.max_pages + 1023) / 1024;   // four cells a thread
    const int grid = (int)std::min<long long>(std::max(items, tables), 8LL * device_sm_count());
    HRA_LAUNCH(kv8_copy_kernel<COMPACT>, dim3(grid), dim3(256), 0, st, a);
    return cudaGetLastError();
}

template <typename K>
cudaError_t launch_team(K kernel, const Kv8PagesArgs& a, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kTeam);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kTeam;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <bool WINDOW>
cudaError_t launch_update_plan(const Kv8PagesArgs& a, cudaStream_t st) {
    const size_t bytes = one_cta_bytes(a.rows, a.n_pages);
    if ((long long)a.rows * a.max_pages + a.n_pages >= kTeamFrom || bytes > kOneCtaMost)
        return launch_team(kv8_update_plan_kernel<kTeam, WINDOW>, a, st);
    static bool configured[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(kv8_update_plan_kernel<1, WINDOW>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kOneCtaMost);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    HRA_LAUNCH((kv8_update_plan_kernel<1, WINDOW>), dim3(1), dim3(kPlanThreads), bytes, st, a);
    return cudaGetLastError();
}

}  // namespace

size_t kv8_pages_scratch_bytes(int rows, int max_pages, int n_pages) {
    const size_t mv = (size_t)std::max(rows, n_pages);
    return 4 * (kHead + 2 * mv + 3 * (size_t)rows + 1 + 2 * (size_t)n_pages + (size_t)rows * max_pages);
}

cudaError_t launch_kv8_update(const Kv8PagesArgs& a, cudaStream_t st) {
    const cudaError_t e = a.window > 0 ? launch_update_plan<true>(a, st) : launch_update_plan<false>(a, st);
    return e != cudaSuccess ? e : launch_copy<false>(a, a.rows, st);
}

cudaError_t launch_kv8_compact(const Kv8PagesArgs& a, cudaStream_t st) {
    if (a.n_pages >= kTeamPages) {
        const cudaError_t e = launch_team(kv8_compact_plan_kernel<kTeam, kRun>, a, st);
        if (e != cudaSuccess) return e;
    } else if (a.n_pages > 2 * kPlanThreads) {
        HRA_LAUNCH((kv8_compact_plan_kernel<1, kRun>), dim3(1), dim3(kPlanThreads), 0, st, a);
    } else {
        HRA_LAUNCH((kv8_compact_plan_kernel<1, 1>), dim3(1), dim3(kPlanThreads), 0, st, a);
    }
    return launch_copy<true>(a, a.n_pages / 2 + 1, st);
}

}  // namespace hra
