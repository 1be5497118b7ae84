// kv8.cuh -- layout of the paged 8-bit K/V cache and the index arithmetic its kernels share.
//
// A pool holds n_pages pages per layer; a page holds page_size consecutive tokens of one sequence
// for every kv head: codes [2][n_kv][page_size][head_dim] (0 = K, 1 = V; E4M3) and scales
// [2][n_kv][page_size / 16] (fp32, 0 or a power of two, one for each block of 16 tokens and head).  The value of an
// element is code * scale.  Row b of the page table lists the pages of sequence b in order.
//
// Everything here is plain integer arithmetic and compiles as host code too, so that a test
// without a GPU can check it against the buffers' sizes.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KV8_HD __host__ __device__ __forceinline__
#else
#define KV8_HD inline
#endif

namespace hra {

constexpr int kKv8Block = 16;       // tokens that share a scale
constexpr float kKv8Top = 448.0f;   // largest E4M3 value

// One layer of the cache.
struct Kv8View {
    uint8_t* codes;
    float* scales;
    const int32_t* table;    // [rows][max_pages]
    unsigned int* err;       // sticky error bits (may be null)
    int n_pages, n_kv, head_dim, page_size, page_shift, max_pages;
};

// Offset (elements) of token `slot` of head `head` in a page's codes; which: 0 = K, 1 = V.  Pools
// pass 2^31 elements, so the product is 64 bits wide from the first factor on.
KV8_HD long long kv8_code_at(const Kv8View& c, int page, int which, int head, int slot) {
    return ((((long long)page * 2 + which) * c.n_kv + head) << c.page_shift) * c.head_dim +
           (long long)slot * c.head_dim;
}
KV8_HD long long kv8_scale_at(const Kv8View& c, int page, int which, int head, int slot) {
    return (((long long)page * 2 + which) * c.n_kv + head) * (c.page_size / kKv8Block) + slot / kKv8Block;
}
// Page of position `pos` of table row `row`; -1 when the position lies outside the row or its entry
// names no page of the pool.
KV8_HD int kv8_page_of(const Kv8View& c, int row, int pos) {
    const int i = pos >> c.page_shift;
    if (pos < 0 || i >= c.max_pages) return -1;
    const int page = c.table[(long long)row * c.max_pages + i];
    return page >= 0 && page < c.n_pages ? page : -1;
}
// Rows [lo, hi) of sequence b in packed tensors of `total` rows, from a cu array whose contents
// nobody has checked: always inside the tensor.
KV8_HD void kv8_rows(const int32_t* cu, int b, int total, int& lo, int& n) {
    int a = cu[b], z = cu[b + 1];
    a = a < 0 ? 0 : a > total ? total : a;
    z = z < a ? a : z > total ? total : z;
    lo = a;
    n = z - a;
}
// The smallest power of two s with a <= 448 s, at least 2^-126 (448 = 1.75 * 2^8): from the bits
// of a finite a >= 0.
KV8_HD uint32_t kv8_scale_bits(uint32_t a_bits) {
    const int e = (int)(a_bits >> 23) - 8 + ((a_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)(e < 1 ? 1 : e) << 23;
}
// Turns blk, blk + step, ... below blk1, at most `most`: with a ring of `most` stages of which one is requested at the start of a
// turn, the copies under way before turn blk has taken its own.
KV8_HD int kv8_turns_left(int blk, int blk1, int step, int most) {
    const int left = blk < blk1 ? (blk1 - blk - 1) / step + 1 : 0;
    return left < most ? left : most;
}
// Most blocks of 16 that n >= 1 consecutive positions can touch.
KV8_HD int kv8_max_blocks(int n) { return (n + kKv8Block - 2) / kKv8Block + 1; }

}  // namespace hra
