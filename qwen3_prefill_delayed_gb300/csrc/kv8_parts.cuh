// kv8_parts.cuh -- partial results of attention over the paged 8-bit cache, which the kernels that write them share with the
// ones that join them.
//
// A part of an output row is the sum over some of its keys: m, the largest score s; l, the sum of 2^(s - m); M, the largest
// s + log2 of its block's V scale; and per dim the sum of 2^(s - M) times V, in units of 2^-15 (kv8_attention.cu) or 2^-11
// (kv8_prompt.cu).
#pragma once

#include "kv8_device.cuh"

namespace hra {

constexpr int kTileRows = 128;     // (position, head) rows of a prompt item
constexpr int kTileKeys = 64;      // keys of its tiles
constexpr float kTileUnit = 11.f;  // log2 of the weight of the reference maximum in a prompt's sums ...
constexpr float kRowsUnit = 15.f;  // ... and in a short sequence's

struct PromptRec {   // 32 bytes: one (query tile, sequence) pair
    int b, row0, n, q_lo, kv_len, keys;
    long long before;   // equal shares: tiles of the items of the pairs before
};
constexpr int kRecWords = 8;
__host__ __device__ __forceinline__ int key_tiles(int keys) {   // an item without keys has one empty tile: its rows get 0
    return keys > 0 ? (keys + kTileKeys - 1) / kTileKeys : 1;
}

// A prompt item's part: [kTileRows][HD] sums, then m, l and M of the rows.
template <int HD>
struct PromptSlot {
    static constexpr int FLOATS = kTileRows * (HD + 3);
};
// A short sequence's part: [ROWS][HD] sums, then [ROWS][3] (m, l, M).
template <int HD, int NG>
struct Slot {
    static constexpr int ROWS = 8 * NG;
    static constexpr int FLOATS = ROWS * (HD + 3);
};

// Shared prefixes (kv8_shared.cu).  A unit: part of the key tiles of one (query tile, group, kv head).
struct PrefixUnit {
    int b, row0, n, q_lo;             // the group's first row with new tokens, its packed rows, the tile's first token
    int keys, head, t_first, count;   // the prefix, and the unit's tiles (0: no unit)
};
// Of batch row b: the positions that it reads through another row of its group, the group's first unit and packed row, and the
// units of each (query tile, kv head).
struct SharedRow {
    int prefix, unit0, row0, parts;
};
// What the kernels of one call share in scratch.
struct SharedCall {
    PrefixUnit* units;   // [most_units]; unit u is CTA u % prefix_grid's
    int32_t* n_units;
    SharedRow* rows;     // [batch]
    float* prefix_parts; // PromptSlots: [most_units]
    float* own_parts;    // Slots: [batch][row_tiles][n_kv][splits]
    int prefix_grid, most_units, row_tiles, splits;
    int own_units;       // of 128 keys, that a CTA takes of a row's own positions at least
};
cudaError_t launch_kv8_prefix(const Kv8AttnArgs& a, const SharedCall& c, cudaStream_t st);   // kv8_prompt.cu
cudaError_t launch_kv8_own(const Kv8AttnArgs& a, const SharedCall& c, cudaStream_t st);      // kv8_attention.cu
cudaError_t launch_kv8_shared(const Kv8AttnArgs& a, cudaStream_t st);                        // kv8_shared.cu
// Whether a call's prefixes are read once; if not, launch_kv8_attention goes row by row.
bool kv8_shares(const Kv8View& c, int batch, int total_rows, int nq, int max_new, int groups, int max_prefix);
// Rows of a short sequence's tile: one n = 8 column group of the MMAs while its (position, head) rows fit, else two.
inline int column_groups(int G, int max_new) { return (long long)G * max_new <= 8 ? 1 : 2; }

}  // namespace hra
