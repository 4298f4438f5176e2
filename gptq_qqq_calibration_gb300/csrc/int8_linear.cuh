// Parameters and launchers of the 8-bit integer linear layer's kernels, and the
// gradients kernel it shares with the gated feed-forward projections.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "hess.h"

namespace hk {

// How many pairs of SMs run at once, and what a caller of ff_gradients_single
// provides for the tiles that are split: one piece (256 KB) per pair, two arrival
// counts per pair, all zero before the first call.
hess_status ff_resident_pairs(int dev, int* pairs, int* sms);
constexpr size_t kFfPieceBytes = 256 * 256 * sizeof(float);

// dX = dY W (dY [n, f], W [f, d], dX [n, d]) and dW = dY^T X (X [n, d], dW [f, d]) of one
// 16-bit type, row-major and contiguous; dX or dW may be NULL.  Launches on `s`,
// nothing else (no argument checks, no ordering of the workspace's users).
struct FfSingle {
    const void *dY, *W, *X;
    void *dX, *dW;
    int64_t n, d, f;
    int32_t dtype;
    int pairs;
    float* pieces;
    uint32_t *arrived, *status;
    unsigned long long timeout_ns;
};
hess_status ff_gradients_single(const FfSingle& a, cudaStream_t s);

}  // namespace hk
