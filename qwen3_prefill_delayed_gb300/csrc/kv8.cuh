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
constexpr int kKv8MaxGroups = 1024; // of rows that share a prefix
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
// i / d for 0 <= i < 2^31 and 1 <= d <= 2^30: with 2^(b - 1) < d <= 2^b and m = ceil(2^(31 + b) / d), i m / 2^(31 + b) exceeds i / d
// by less than 1 / d.
struct Kv8Div {
    uint32_t mul;
    int shift;
};
KV8_HD Kv8Div kv8_div(int d) {
    int b = 0;
    while ((1 << b) < d) ++b;
    return {(uint32_t)(((1ull << (31 + b)) + d - 1) / d), 31 + b};
}
KV8_HD int kv8_over(const Kv8Div& d, int i) { return (int)((unsigned long long)(uint32_t)i * d.mul >> d.shift); }
// Positions that a window hides.  A token at position p sees those of [0, p] from p - window + 1 on and those below `sinks`; of
// tokens from position `first` on, the units of `per` positions that hold anything they see are 0 .. from - 1 and then
// from + by, from + by + 1, ...  window 0: everything is seen.
struct Kv8Skip {
    int from, by;
};
KV8_HD Kv8Skip kv8_skip(int first, int window, int sinks, int per) {
    const int near = window > 0 && first >= window ? (first - window + 1) / per : 0;
    const int keep = (sinks + per - 1) / per;
    const int from = near < keep ? near : keep;
    return {from, near - from};
}
KV8_HD int kv8_unit_at(const Kv8Skip& s, int i) { return i < s.from ? i : i + s.by; }
// Most positions that tokens within a span of `tokens` see of max_len.
KV8_HD int kv8_most_seen(int max_len, int window, int sinks, int tokens) {
    const long long n = (long long)window + sinks + tokens;
    return window > 0 && n < max_len ? (int)n : max_len;
}
// Tile `tile` of the n new tokens (of which max_new count) of a sequence of kv_len positions, over its positions from `prefix`
// (whole blocks) on in units of 128 keys, in parts of `least` units or, where more than `splits` of
// them would do, in `splits`: its tokens t0 .. t0 + tokens - 1, the positions below the last
// of them, the blocks, the units of a part, and how many parts there are.
struct Kv8Own {
    int t0, tokens, keys, blocks, per, parts;
};
KV8_HD Kv8Own kv8_own(int kv_len, int n, int tile, int tile_tokens, int max_new, int prefix, int splits, int least) {
    Kv8Own o;
    const int count = n < max_new ? n : max_new;
    o.t0 = tile * tile_tokens;
    o.tokens = count - o.t0 < tile_tokens ? count - o.t0 : tile_tokens;
    if (o.tokens < 0) o.tokens = 0;
    o.keys = kv_len - n + o.t0 + o.tokens;
    if (o.keys < 0) o.keys = 0;
    o.blocks = (o.keys + kKv8Block - 1) / kKv8Block - prefix / kKv8Block;
    if (o.blocks < 0) o.blocks = 0;
    const int units = o.blocks > 0 ? (o.blocks + 7) / 8 : 1;
    o.per = (units + splits - 1) / splits;
    if (o.per < least) o.per = least;
    o.parts = (units + o.per - 1) / o.per;
    return o;
}
// Most blocks of 16 that n >= 1 consecutive positions can touch.
KV8_HD int kv8_max_blocks(int n) { return (n + kKv8Block - 2) / kKv8Block + 1; }

}  // namespace hra
