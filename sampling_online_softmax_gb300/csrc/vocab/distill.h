// distill.h -- the parameter block of the distillation kernels.
#pragma once

#include <cuda_bf16.h>

#include "rows.h"

namespace spec {
namespace vocab {

constexpr int kDThreads = 256;
constexpr int kPartBytes = 64 * 1024;  // of a row, at most, in a CTA's shared memory (loss and gradient)

struct DistillArgs {
    const unsigned char *student, *student_end;  // [N, V] logits
    const int32_t *ids;      // [N, K] the teacher's tokens, -1 in an empty slot
    const float *top;        // [N, K] the teacher's logits
    const float *lse;        // [N] the teacher's log-normaliser, or null
    const float *weight;     // [N] or null
    const float *grad_loss;  // [N] (backward alone)
    int N, V, K;
    int cluster, part;       // CTAs per row, vectors per CTA
    float T;
    float *loss;             // [N]
    float *stats;            // [N, 2]
    unsigned char *grad;     // [N, V], the logits' type
    uint32_t *status;
};

enum DistillForm : int { kLoss = 0, kLossGrad = 1, kBackward = 2 };

template <int EB>
spec_status launch_distill(const DistillArgs &a, int form, cudaStream_t stream);

}  // namespace vocab
}  // namespace spec
