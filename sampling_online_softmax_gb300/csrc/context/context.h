// context.h -- what the host and the kernels on the paged cache share.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../host.h"

namespace spec {
namespace context {

// spec_cache as the kernels take it; [0] the keys, [1] the values.
struct CacheView {
    unsigned char *data[2];
    uint8_t *scale[2];
    const int32_t *table;
    int pages, page_bits, kv_heads, table_width;
};

}  // namespace context
}  // namespace spec
