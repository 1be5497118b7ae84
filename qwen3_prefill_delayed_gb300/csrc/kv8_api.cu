// kv8_api.cu -- the extern "C" entry points of the paged 8-bit K/V cache declared in include/hra.h:
// argument checks before the first launch, then one launch function per operation.  No allocation,
// no synchronisation.
#include <cmath>

#include <algorithm>

#include "internal.h"
#include "kv8_host.h"

using namespace hra;

namespace hra {

namespace {

inline bool aligned(const void* p, uintptr_t n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct Range {
    const void* at;
    size_t n;
};
inline bool overlap(const Range& a, const Range& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
    return x < y + b.n && y < x + a.n;
}

}  // namespace

int kv8_check(const hra_kv8_cache* c) {
    if (c == nullptr || !aligned(c->codes, 16) || !aligned(c->scales, 16) || !aligned(c->page_table, 4) ||
        !aligned(c->lens, 4) || !aligned(c->errors, 4) || (c->refs != nullptr && !aligned(c->refs, 4)))
        return HRA_ERR_INVALID_ARG;
    if (c->n_layers < 1 || c->n_pages < 1 || c->n_kv_heads < 1 || c->rows < 1 || c->max_pages < 1)
        return HRA_ERR_INVALID_ARG;
    if ((c->head_dim != 64 && c->head_dim != 128) || c->page_size < 16 || c->page_size > 128 ||
        (c->page_size & (c->page_size - 1)) != 0 || c->n_kv_heads > 1024 || c->rows > 65535)
        return HRA_ERR_UNSUPPORTED;
    if ((long long)c->max_pages * c->page_size > (1 << 30) || (long long)c->rows * c->max_pages > (1 << 30) ||
        2LL * c->n_pages * c->n_kv_heads * c->page_size >= (1LL << 31) ||
        (long long)c->max_pages * c->page_size * c->n_kv_heads > (1LL << 37))
        return HRA_ERR_UNSUPPORTED;   // positions, table cells, scratch words, a layer's rows and a sequence's units of
                                      // 128 keys over all heads stay inside 32 bits
    return HRA_OK;
}

int kv8_reach_check(const hra_kv8_reach* r, int batch) {
    if (r == nullptr) return HRA_OK;
    if (r->window < 0 || r->sinks < 0 || (r->window == 0 && r->sinks != 0) || r->groups < 0) return HRA_ERR_INVALID_ARG;
    if (r->window > (1 << 30) || r->sinks > (1 << 30)) return HRA_ERR_RANGE;
    if (r->groups == 0) return HRA_OK;
    if (r->window > 0 || r->groups > kKv8MaxGroups) return HRA_ERR_UNSUPPORTED;
    if (!aligned(r->group_cu_dev, 4) || !aligned(r->prefix_dev, 4) || r->groups > batch || r->max_prefix < 0 || r->max_own < 0)
        return HRA_ERR_INVALID_ARG;
    return HRA_OK;
}

bool kv8_reach_touches(const hra_kv8_reach* r, const void* at, size_t n) {
    if (r == nullptr || r->groups == 0) return false;
    return overlap({r->group_cu_dev, 4 * ((size_t)r->groups + 1)}, {at, n}) || overlap({r->prefix_dev, 4 * (size_t)r->groups}, {at, n});
}

void kv8_set_reach(Kv8AttnArgs& a, const hra_kv8_reach* r) {
    if (r == nullptr) return;
    a.window = r->window;
    a.sinks = r->sinks;
    a.groups = r->groups;
    a.group_cu = r->group_cu_dev;
    a.prefix = r->prefix_dev;
    a.max_prefix = r->max_prefix;
    a.max_own = r->max_own;
}

Kv8View kv8_view(const hra_kv8_cache& c, int layer) {
    Kv8View v{};
    const long long codes = 2LL * c.n_kv_heads * c.page_size * c.head_dim;
    const long long scales = 2LL * c.n_kv_heads * (c.page_size / kKv8Block);
    v.codes = reinterpret_cast<uint8_t*>(c.codes) + (long long)layer * c.n_pages * codes;
    v.scales = c.scales + (long long)layer * c.n_pages * scales;
    v.table = c.page_table;
    v.err = c.errors;
    v.n_pages = c.n_pages;
    v.n_kv = c.n_kv_heads;
    v.head_dim = c.head_dim;
    v.page_size = c.page_size;
    for (v.page_shift = 0; (1 << v.page_shift) < c.page_size; ++v.page_shift) {
    }
    v.max_pages = c.max_pages;
    return v;
}

}  // namespace hra

namespace {

int status(cudaError_t e) { return e == cudaSuccess ? HRA_OK : HRA_ERR_CUDA; }

// Packed rows of a batch: the counts that the host knows.
int rows_check(const hra_kv8_cache& c, const int32_t* cu, const int32_t* per_row, int batch, int total, int max_new) {
    if (!aligned(cu, 4) || !aligned(per_row, 4) || batch < 1 || total < 0 || max_new < 0) return HRA_ERR_INVALID_ARG;
    if (batch > c.rows) return HRA_ERR_INVALID_ARG;
    if (total > (1 << 30) || max_new > (1 << 30)) return HRA_ERR_RANGE;
    if (total > 0 && (max_new < 1 || max_new > total)) return HRA_ERR_INVALID_ARG;
    return HRA_OK;
}

size_t attention_scratch(const Kv8View& v, int batch, int total, int nq, int max_new, int max_len, const hra_kv8_reach* r) {
    if (r == nullptr || r->groups == 0) return kv8_attention_scratch_bytes(v, batch, total, nq, max_new, max_len);
    return kv8_shared_scratch_bytes(v, batch, total, nq, max_new, max_len, r->groups, r->max_prefix, r->max_own);
}

bool heads_dims_ok(int nq, int nkv) { return nq >= 1 && nq % nkv == 0 && nq / nkv <= 16; }

int pages_impl(const hra_kv8_cache* cache, const int32_t* parents, const int32_t* room, int32_t* table_out,
               int32_t* lens_out, int32_t* refs_out, void* workspace, size_t workspace_bytes, void* stream, bool update,
               const hra_kv8_reach* reach = nullptr) {
    int rc = kv8_check(cache);
    if (rc != HRA_OK) return rc;
    if (reach != nullptr && reach->groups != 0) return HRA_ERR_INVALID_ARG;
    rc = kv8_reach_check(reach, 0);
    if (rc != HRA_OK) return rc;
    const hra_kv8_cache& c = *cache;
    if (c.refs == nullptr || !aligned(table_out, 4) || !aligned(lens_out, 4) || !aligned(refs_out, 4) ||
        !aligned(workspace, 16))
        return HRA_ERR_INVALID_ARG;
    if ((parents != nullptr && !aligned(parents, 4)) || (room != nullptr && !aligned(room, 4)))
        return HRA_ERR_INVALID_ARG;
    const size_t need = hra_kv8_pages_workspace_size(cache);
    if (workspace_bytes < need) return HRA_ERR_WORKSPACE;
    // an output is its own input, or apart from every input and from the other outputs
    const size_t n_table = 4 * (size_t)c.rows * c.max_pages, n_rows = 4 * (size_t)c.rows, n_refs = 4 * (size_t)c.n_pages;
    const Range in[3] = {{c.page_table, n_table}, {c.lens, n_rows}, {c.refs, n_refs}};
    const Range out[4] = {{table_out, n_table}, {lens_out, n_rows}, {refs_out, n_refs}, {workspace, need}};
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 3; ++j)
            if ((i != j && overlap(out[i], out[j])) || (overlap(out[i], in[j]) && (i != j || out[i].at != in[j].at)))
                return HRA_ERR_INVALID_ARG;
    // parents and room are read before any output is written, but while the workspace is
    for (const int32_t* p : {parents, room})
        if (p != nullptr && overlap(out[3], {p, n_rows})) return HRA_ERR_INVALID_ARG;
    const Kv8View v = kv8_view(c, 0);
    Kv8PagesArgs a{};
    a.codes = v.codes;
    a.scales = v.scales;
    a.table = c.page_table;
    a.lens = c.lens;
    a.refs = c.refs;
    a.parents = parents;
    a.room = room;
    a.table_out = table_out;
    a.lens_out = lens_out;
    a.refs_out = refs_out;
    a.err = c.errors;
    a.scratch = workspace;
    a.code_page = 2LL * c.n_kv_heads * c.page_size * c.head_dim;
    a.scale_page = 2 * c.n_kv_heads * (c.page_size / kKv8Block);
    a.n_layers = c.n_layers;
    a.n_pages = c.n_pages;
    a.page_shift = v.page_shift;
    a.rows = c.rows;
    a.max_pages = c.max_pages;
    if (reach != nullptr) {
        a.window = reach->window;
        a.sinks = reach->sinks;
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return status(update ? launch_kv8_update(a, st) : launch_kv8_compact(a, st));
}

}  // namespace

extern "C" {

int hra_kv8_append(const hra_kv8_cache* cache, int32_t layer, const void* k_dev, const void* v_dev, int64_t row_stride,
                   const int32_t* cu_dev, const int32_t* start_dev, int32_t batch, int32_t total_rows, int32_t max_new,
                   void* stream) {
    int rc = kv8_check(cache);
    if (rc != HRA_OK) return rc;
    const hra_kv8_cache& c = *cache;
    if (layer < 0 || layer >= c.n_layers) return HRA_ERR_INVALID_ARG;
    rc = rows_check(c, cu_dev, start_dev, batch, total_rows, max_new);
    if (rc != HRA_OK) return rc;
    if (total_rows == 0) return HRA_OK;
    if (!aligned(k_dev, 16) || !aligned(v_dev, 16) || row_stride < (int64_t)c.n_kv_heads * c.head_dim ||
        row_stride % 8 != 0)
        return HRA_ERR_INVALID_ARG;
    // every CTA of a row reads start and cu, and one of them writes the row's length
    const Range lens{c.lens, 4 * (size_t)c.rows};
    if (overlap(lens, {start_dev, 4 * (size_t)batch}) || overlap(lens, {cu_dev, 4 * ((size_t)batch + 1)}))
        return HRA_ERR_INVALID_ARG;
    Kv8AppendArgs a{};
    a.view = kv8_view(c, layer);
    a.k = reinterpret_cast<const bf16*>(k_dev);
    a.v = reinterpret_cast<const bf16*>(v_dev);
    a.row_stride = row_stride;
    a.cu = cu_dev;
    a.start = start_dev;
    a.lens = c.lens;
    a.batch = batch;
    a.total_rows = total_rows;
    a.max_new = max_new;
    return status(launch_kv8_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t hra_kv8_attention_reach_workspace_size(const hra_kv8_cache* cache, int32_t batch, int32_t total_rows,
                                              int32_t n_q_heads, int32_t max_new, int32_t max_len,
                                              const hra_kv8_reach* reach) {
    if (kv8_check(cache) != HRA_OK || batch < 1 || batch > cache->rows || total_rows < 0 || max_new < 0 ||
        max_new > total_rows || max_len < 0 || !heads_dims_ok(n_q_heads, cache->n_kv_heads))
        return 0;
    if (kv8_reach_check(reach, batch) != HRA_OK) return 0;
    return 256 + attention_scratch(kv8_view(*cache, 0), batch, total_rows, n_q_heads, max_new, max_len, reach);
}
size_t hra_kv8_attention_workspace_size(const hra_kv8_cache* cache, int32_t batch, int32_t total_rows,
                                        int32_t n_q_heads, int32_t max_new, int32_t max_len) {
    return hra_kv8_attention_reach_workspace_size(cache, batch, total_rows, n_q_heads, max_new, max_len, nullptr);
}

int hra_kv8_attention(const hra_kv8_cache* cache, int32_t layer, const void* q_dev, int64_t q_row_stride,
                      int32_t n_q_heads, float scale, const int32_t* cu_dev, const int32_t* kv_len_dev, int32_t batch,
                      int32_t total_rows, int32_t max_new, int32_t max_len, void* out_dev, void* workspace,
                      size_t workspace_bytes, void* stream) {
    return hra_kv8_attention_reach(cache, layer, q_dev, q_row_stride, n_q_heads, scale, cu_dev, kv_len_dev, batch, total_rows,
                                   max_new, max_len, nullptr, out_dev, workspace, workspace_bytes, stream);
}

int hra_kv8_attention_reach(const hra_kv8_cache* cache, int32_t layer, const void* q_dev, int64_t q_row_stride,
                            int32_t n_q_heads, float scale, const int32_t* cu_dev, const int32_t* kv_len_dev,
                            int32_t batch, int32_t total_rows, int32_t max_new, int32_t max_len,
                            const hra_kv8_reach* reach, void* out_dev, void* workspace, size_t workspace_bytes,
                            void* stream) {
    int rc = kv8_check(cache);
    if (rc != HRA_OK) return rc;
    const hra_kv8_cache& c = *cache;
    if (layer < 0 || layer >= c.n_layers || !std::isfinite(scale) || scale < 0.f) return HRA_ERR_INVALID_ARG;
    if (!heads_dims_ok(n_q_heads, c.n_kv_heads)) return HRA_ERR_UNSUPPORTED;
    rc = rows_check(c, cu_dev, kv_len_dev, batch, total_rows, max_new);
    if (rc != HRA_OK) return rc;
    if (max_len < 0 || max_len > (long long)c.max_pages * c.page_size) return HRA_ERR_RANGE;
    rc = kv8_reach_check(reach, batch);
    if (rc != HRA_OK) return rc;
    if (total_rows == 0) return HRA_OK;
    if (!aligned(q_dev, 16) || !aligned(out_dev, 16) || q_row_stride < (int64_t)n_q_heads * c.head_dim ||
        q_row_stride % 8 != 0 || !aligned(workspace, 16))
        return HRA_ERR_INVALID_ARG;
    Kv8AttnArgs a{};
    a.view = kv8_view(c, layer);
    if (workspace_bytes < 256 + attention_scratch(a.view, batch, total_rows, n_q_heads, max_new, max_len, reach))
        return HRA_ERR_WORKSPACE;
    // q is read again behind the output of a row with a NaN (kv8_row_again)
    const size_t q_row = 2 * (size_t)n_q_heads * c.head_dim;
    if (overlap({q_dev, 2 * (size_t)q_row_stride * (total_rows - 1) + q_row}, {out_dev, q_row * total_rows}))
        return HRA_ERR_INVALID_ARG;
    if (kv8_reach_touches(reach, workspace, workspace_bytes) || kv8_reach_touches(reach, out_dev, q_row * total_rows))
        return HRA_ERR_INVALID_ARG;
    a.q = reinterpret_cast<const bf16*>(q_dev);
    a.row_stride = q_row_stride;
    a.out = reinterpret_cast<bf16*>(out_dev);
    a.cu = cu_dev;
    a.kv_len = kv_len_dev;
    a.scale_log2 = (scale == 0.f ? 1.0f / std::sqrt((float)c.head_dim) : scale) * 1.4426950408889634f;
    a.batch = batch;
    a.total_rows = total_rows;
    a.nq = n_q_heads;
    a.max_new = max_new;
    a.max_len = max_len;
    a.scratch = workspace;
    kv8_set_reach(a, reach);
    return status(launch_kv8_attention(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t hra_kv8_pages_workspace_size(const hra_kv8_cache* cache) {
    if (kv8_check(cache) != HRA_OK) return 0;
    return kv8_pages_scratch_bytes(cache->rows, cache->max_pages, cache->n_pages);
}

int hra_kv8_update(const hra_kv8_cache* cache, const int32_t* parents_dev, const int32_t* room_dev,
                   int32_t* table_out, int32_t* lens_out, int32_t* refs_out, void* workspace, size_t workspace_bytes,
                   void* stream) {
    return pages_impl(cache, parents_dev, room_dev, table_out, lens_out, refs_out, workspace, workspace_bytes, stream,
                      true);
}

int hra_kv8_update_reach(const hra_kv8_cache* cache, const int32_t* parents_dev, const int32_t* room_dev,
                         const hra_kv8_reach* reach, int32_t* table_out, int32_t* lens_out, int32_t* refs_out,
                         void* workspace, size_t workspace_bytes, void* stream) {
    return pages_impl(cache, parents_dev, room_dev, table_out, lens_out, refs_out, workspace, workspace_bytes, stream,
                      true, reach);
}

int hra_kv8_compact(const hra_kv8_cache* cache, int32_t* table_out, int32_t* lens_out, int32_t* refs_out,
                    void* workspace, size_t workspace_bytes, void* stream) {
    return pages_impl(cache, nullptr, nullptr, table_out, lens_out, refs_out, workspace, workspace_bytes, stream, false);
}

}  // extern "C"
