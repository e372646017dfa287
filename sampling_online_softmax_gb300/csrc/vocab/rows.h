// rows.h -- what the host and the kernels on rows of logits share: launch
// constants and the parameter block.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../host.h"

namespace spec {
namespace vocab {

constexpr int kThreads = 256;
// CTAs of a row kernel per SM.  With 3 (80 registers) sampling spills 78 words in bf16 and
// 14 in fp32, the largest logits none: 48 flat rows of 50257 fp32 take
// 61 us against 65 with 4, the 64 largest of 2304 rows of 129280 bf16 134 against 141, top-p alone over 64
// rows of 128256 bf16 58 against 71, one row 10.7 against 11.7; 4 hide more of each other's tails where rows are
// many (512 rows of 152064 by top-p: 55 against 60) or short (1293 rows of 2695 bf16: 20.3 against 21.3).
constexpr int kRowCtas = 3;
constexpr int kMaxCluster = 8;    // CTAs per row (the portable limit)
constexpr int kMaxList = 2048;    // entries of a cluster's list

constexpr float kMinTemperature = 1e-6f, kMaxTemperature = 1e6f;

struct RowArgs {
    const unsigned char *base;  // [B, V] logits
    const unsigned char *end;   // one past their last byte
    int B, V;
    int cluster;                // CTAs per row
    int part;                   // 16-byte vectors of a row per CTA
    int U;                      // weights in units of 2^-U
    uint32_t *status;
    // filtered sampling, one entry a row
    const float *temperature, *u;
    const int32_t *top_k;       // null: no limit
    const float *top_p, *min_p;
    int32_t *tokens;
    // the largest logits
    int K;
    float temp;
    float *values;              // [B, K]
    int32_t *ids;
    float *lse;                 // [B] or null
};

enum RowOp : int { kSampleRows = 0, kTopRows = 1 };

template <int EB, int OP>
spec_status launch_rows(const RowArgs &a, cudaStream_t stream);

}  // namespace vocab
}  // namespace spec
