// distill.h -- the parameter block of the distillation kernels.
#pragma once

#include <cuda_bf16.h>

#include "rows.h"

namespace spec {
namespace vocab {

constexpr int kDThreads = 256;
constexpr int kTrainCtas = 3;             // CTAs of the loss and gradient kernel per SM
constexpr int kPartBytes = 64 * 1024;  // of a row, at most, in a CTA's shared memory (loss and gradient)

constexpr int kLossBytes = 320 * 1024, kBackwardBytes = 96 * 1024;  // of a row per CTA: loss alone, gradient alone
constexpr int kWaves = 4;                 // a row is shared further where there are fewer CTAs than this an SM

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
    uint32_t zero;           // 0, for a dependence that the compiler cannot see through
};

enum DistillForm : int { kLoss = 0, kLossGrad = 1, kBackward = 2 };

// Clusters of a launch that fit the device at a time (cached; 0: unknown).
int resident_clusters(int dev, const void *kernel, const cudaLaunchConfig_t &cfg);

template <int EB>
spec_status launch_distill(const DistillArgs &a, int form, cudaStream_t stream);

}  // namespace vocab
}  // namespace spec
