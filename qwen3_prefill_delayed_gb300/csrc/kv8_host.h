// kv8_host.h -- host helpers of the paged 8-bit cache shared by its entry points and the path.
#pragma once

#include "internal.h"

namespace hra {

// HRA_OK, or the status a call with this cache returns.
int kv8_check(const hra_kv8_cache* c);
// The kernels' view of one layer.
Kv8View kv8_view(const hra_kv8_cache& c, int layer);

// HRA_OK, or the status a call of `batch` rows with this reach (null: every position) returns.
int kv8_reach_check(const hra_kv8_reach* reach, int batch);
// Whether a reach's group arrays touch the n bytes at `at`, which the call writes.
bool kv8_reach_touches(const hra_kv8_reach* reach, const void* at, size_t n);
// The reach in the kernels' terms.
void kv8_set_reach(Kv8AttnArgs& a, const hra_kv8_reach* reach);

}  // namespace hra
