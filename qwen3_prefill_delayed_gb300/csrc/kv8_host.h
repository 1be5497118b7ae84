// kv8_host.h -- host helpers of the paged 8-bit cache shared by its entry points and the path.
#pragma once

#include "internal.h"

namespace hra {

// HRA_OK, or the status a call with this cache returns.
int kv8_check(const hra_kv8_cache* c);
// The kernels' view of one layer.
Kv8View kv8_view(const hra_kv8_cache& c, int layer);

}  // namespace hra
