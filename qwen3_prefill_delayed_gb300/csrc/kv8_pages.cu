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
// compact: with U pages in use, the i-th used page with number >= U (ascending) moves to the i-th free
//   page with number < U.  Sources and destinations are disjoint, so the copies need no order.
//
// A plan kernel of one CTA works out the tables in scratch; the copy kernel then moves the pages
// (16-byte copies, persistent over (move, layer, part) items) and brings the tables out, which is why
// the outputs may be the inputs.
#include <algorithm>

#include "kv8_device.cuh"

namespace hra {

namespace {

constexpr int kPlanThreads = 1024;   // what block_scan takes
constexpr int kPart = 16384;   // bytes of one copy item

// Scratch of both operations, in 4-byte words.
struct PlanScratch {
    int32_t* head;     // [0] moves, [1] 1 = write the outputs
    int32_t* first;    // [rows] lowest child of each old row
    int32_t* base;     // [rows + 1] fresh pages before each row
    int32_t* lens;     // [rows]
    int32_t* refs;     // [n_pages]
    int32_t* list;     // [n_pages] free pages in order (update), new number of each page (compact)
    int2* moves;       // [max(rows, n_pages)]
    int32_t* table;    // [rows][max_pages]
    __host__ __device__ PlanScratch(void* p, int rows, int n_pages) {
        head = reinterpret_cast<int32_t*>(p);
        moves = reinterpret_cast<int2*>(head + 4);
        const int mv = rows > n_pages ? rows : n_pages;
        first = head + 4 + 2 * mv;
        base = first + rows;
        lens = base + rows + 1;
        refs = lens + rows;
        list = refs + n_pages;
        table = list + n_pages;
    }
};

__global__ void __launch_bounds__(kPlanThreads) kv8_update_plan_kernel(const Kv8PagesArgs a) {
    pdl_launch();
    pdl_wait();
    const PlanScratch s(a.scratch, a.rows, a.n_pages);
    __shared__ unsigned int bad;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int R = a.rows, W = a.max_pages, P = 1 << a.page_shift;
    if (tid == 0) bad = 0u;
    for (int p = tid; p < a.n_pages; p += kPlanThreads) s.refs[p] = 0;
    for (int b = tid; b < R; b += kPlanThreads) s.first[b] = R;
    __syncthreads();
    auto parent = [&](int b) {
        const int p = a.parents ? a.parents[b] : b;
        return p >= 0 && p < R ? p : -1;
    };
    for (int b = tid; b < R; b += kPlanThreads) {
        const int p = parent(b);
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
    }
    __syncthreads();
    // the pages each new row keeps, and how many fresh ones it needs: one warp a row
    bool too_long = false;
    for (int b = warp; b < R; b += kPlanThreads / 32) {
        const int p = parent(b), len = s.lens[b];
        const int more = p >= 0 && a.room ? max(0, a.room[b]) : 0;
        const long long ends = ((long long)len + more + P - 1) >> a.page_shift;
        const bool heir = p >= 0 && s.first[p] == b;
        too_long |= p >= 0 && ends > W;
        int need = 0;
        for (int i0 = 0; i0 < W; i0 += 32) {
            const int i = i0 + lane;
            int old = -1;
            if (p >= 0 && i < W) {
                old = a.table[(long long)p * W + i];
                if (old >= a.n_pages || old < -1) {
                    atomicOr(&bad, HRA_DEVERR_PAGE_RANGE);
                    old = -1;
                }
            }
            const bool keep = old >= 0 && (heir || i < (len >> a.page_shift));
            if (keep) atomicAdd(&s.refs[old], 1);
            need += __popc(__ballot_sync(0xffffffffu, p >= 0 && i < ends && i < W && !keep));
        }
        if (lane == 0) s.base[b] = need;
    }
    const bool fail_long = __syncthreads_or(too_long);
    int need_all = 0;
    for (int b0 = 0; b0 < R; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int total;
        const int at = block_scan(b < R ? s.base[b] : 0, total);
        if (b < R) s.base[b] = need_all + at;
        need_all += total;
    }
    int free_all = 0;
    for (int p0 = 0; p0 < a.n_pages; p0 += kPlanThreads) {
        const int p = p0 + tid;
        const int is_free = p < a.n_pages && s.refs[p] == 0 ? 1 : 0;
        int total;
        const int at = block_scan(is_free, total);
        if (is_free) s.list[free_all + at] = p;
        free_all += total;
    }
    __syncthreads();
    const bool fail = fail_long || need_all > free_all;
    if (tid == 0) {
        s.head[0] = 0;
        s.head[1] = fail ? 0 : 1;
    }
    __syncthreads();
    if (!fail) {
        for (int b = warp; b < R; b += kPlanThreads / 32) {
            const int p = parent(b), len = s.lens[b];
            const int more = p >= 0 && a.room ? max(0, a.room[b]) : 0;
            const long long ends = ((long long)len + more + P - 1) >> a.page_shift;
            const bool heir = p >= 0 && s.first[p] == b;
            int at = s.base[b];
            for (int i0 = 0; i0 < W; i0 += 32) {
                const int i = i0 + lane;
                int old = -1;
                if (p >= 0 && i < W) {
                    old = a.table[(long long)p * W + i];
                    if (old >= a.n_pages || old < -1) old = -1;
                }
                const bool keep = old >= 0 && (heir || i < (len >> a.page_shift));
                const bool fresh = p >= 0 && i < ends && i < W && !keep;
                const unsigned int mask = __ballot_sync(0xffffffffu, fresh);
                int now = keep ? old : -1;
                if (fresh) {
                    now = s.list[at + __popc(mask & ((1u << lane) - 1u))];
                    s.refs[now] = 1;
                    if (old >= 0 && ((long long)i << a.page_shift) < len)
                        s.moves[atomicAdd(&s.head[0], 1)] = make_int2(old, now);
                }
                at += __popc(mask);
                if (i < W) s.table[(long long)b * W + i] = now;
            }
        }
    }
    if (tid == 0) {
        if (fail) bad |= HRA_DEVERR_PAGES_SPENT;
        if (bad) raise_error(a.err, bad);
    }
}

__global__ void __launch_bounds__(kPlanThreads) kv8_compact_plan_kernel(const Kv8PagesArgs a) {
    pdl_launch();
    pdl_wait();
    const PlanScratch s(a.scratch, a.rows, a.n_pages);
    const int tid = threadIdx.x;
    int used = 0;
    for (int p = tid; p < a.n_pages; p += kPlanThreads) used += a.refs[p] > 0 ? 1 : 0;
    int U;
    (void)block_scan(used, U);
    // holes: .x of moves; movers: .y, swapped into (source, destination) by the copy
    int holes = 0, movers = 0;
    for (int p0 = 0; p0 < a.n_pages; p0 += kPlanThreads) {
        const int p = p0 + tid;
        const bool in = p < a.n_pages;
        const int r = in ? a.refs[p] : 0;
        const int hole = in && p < U && r <= 0, mover = in && p >= U && r > 0;
        int total;
        const int at = block_scan(hole | mover << 16, total);
        if (hole) s.moves[holes + (at & 0xFFFF)].y = p;
        if (mover) s.moves[movers + (at >> 16)].x = p;
        if (in) {
            s.list[p] = p;
            s.refs[p] = p < U ? max(r, 0) : 0;
        }
        holes += total & 0xFFFF;
        movers += total >> 16;
    }
    __syncthreads();
    for (int i = tid; i < movers; i += kPlanThreads) {
        const int2 mv = s.moves[i];
        s.list[mv.x] = mv.y;
        s.refs[mv.y] = a.refs[mv.x];
    }
    if (tid == 0) {
        s.head[0] = movers;
        s.head[1] = 1;
    }
    __syncthreads();
    bool bad = false;
    const long long cells = (long long)a.rows * a.max_pages;
    for (long long i = tid; i < cells; i += kPlanThreads) {
        const int p = a.table[i];
        const bool ok = p >= 0 && p < a.n_pages;
        bad |= !ok && p != -1;
        s.table[i] = ok ? s.list[p] : p;
    }
    for (int b = tid; b < a.rows; b += kPlanThreads) s.lens[b] = a.lens[b];
    if (bad) raise_error(a.err, HRA_DEVERR_PAGE_RANGE);
}

// The moves of the plan in every layer, and the plan's tables to the outputs (or, when the plan
// failed, the inputs to the outputs).
__global__ void __launch_bounds__(256) kv8_copy_kernel(const Kv8PagesArgs a) {
    pdl_launch();
    pdl_wait();
    const PlanScratch s(a.scratch, a.rows, a.n_pages);
    const int tid = threadIdx.x;
    const long long t0 = (long long)blockIdx.x * blockDim.x + tid, step = (long long)gridDim.x * blockDim.x;
    const bool ok = s.head[1] != 0;
    const long long cells = (long long)a.rows * a.max_pages;
    for (long long i = t0; i < cells; i += step) a.table_out[i] = ok ? s.table[i] : a.table[i];
    for (long long i = t0; i < a.rows; i += step) a.lens_out[i] = ok ? s.lens[i] : a.lens[i];
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

cudaError_t launch_copy(const Kv8PagesArgs& a, int most_moves, cudaStream_t st) {
    const long long parts = (a.code_page + kPart - 1) / kPart;
    const long long items = std::max<long long>(1, (long long)most_moves * a.n_layers * parts);
    const int grid = (int)std::min<long long>(items, 8LL * device_sm_count());
    HRA_LAUNCH(kv8_copy_kernel, dim3(grid), dim3(256), 0, st, a);
    return cudaGetLastError();
}

}  // namespace

size_t kv8_pages_scratch_bytes(int rows, int max_pages, int n_pages) {
    const size_t mv = (size_t)std::max(rows, n_pages);
    return 4 * (4 + 2 * mv + 3 * (size_t)rows + 1 + 2 * (size_t)n_pages + (size_t)rows * max_pages);
}

cudaError_t launch_kv8_update(const Kv8PagesArgs& a, cudaStream_t st) {
    HRA_LAUNCH(kv8_update_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, a);
    return launch_copy(a, a.rows, st);
}

cudaError_t launch_kv8_compact(const Kv8PagesArgs& a, cudaStream_t st) {
    HRA_LAUNCH(kv8_compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, a);
    return launch_copy(a, a.n_pages / 2 + 1, st);
}

}  // namespace hra
