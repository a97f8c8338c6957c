// mixture.h -- the router's and the combination's problems, as the host
// dispatcher hands them to the kernel launchers (all argument checks done).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "grouped.h"  // kOutF32, kOutBf16, kOutF16: a matrix's type
#include "internal.h"

namespace gemm {

constexpr int kMaxExperts = 1024, kMaxChoices = 32, kMaxExpertGroups = 32;

enum : int { kSoftmax = 0, kSigmoid = 1 };  // = gemm_score_t

// SMs of the current device (1 if that cannot be asked).
int sm_count();

struct RouteProblem {
    int64_t tokens;
    int experts, k;
    const void *logits;
    int64_t ld;
    int type;
    int score, renorm;
    float scale;
    const float *bias;  // forward
    int groups, kept, top;
    int32_t *chosen;  // forward: written; gradient: read
    float *weights;
    const float *dweights;  // gradient
    void *dlogits;
    int64_t ld_d;
};
cudaError_t launch_route(const RouteProblem &p, cudaStream_t stream, const char **name);
cudaError_t launch_route_grad(const RouteProblem &p, cudaStream_t stream, const char **name);

// D(t, :) = residual(t, :) + sum_j w(t, j) Y(position(t, j), :); the gradient's dD is D here.
struct CombineProblem {
    int64_t tokens, k, N;
    const void *Y;
    int64_t ldy, rows_y;
    int y_type;
    const int32_t *position;
    const float *weights;  // or null
    const void *residual;  // or null
    int64_t ld_r;
    void *D;  // gradient: read
    int64_t ldd;
    int d_type;
    void *dY;  // or null
    int64_t ld_dy;
    float *dweights;  // or null
};
cudaError_t launch_combine(const CombineProblem &p, cudaStream_t stream, const char **name);
cudaError_t launch_combine_grad(const CombineProblem &p, cudaStream_t stream, const char **name);
// Reads and clears the combination's device status word (after a sync).
cudaError_t combine_read_and_clear_status(cudaStream_t stream, int *status);

}  // namespace gemm
