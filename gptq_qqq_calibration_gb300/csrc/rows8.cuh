// Launchers of the 8-bit row kernels that other parts of the library call (no
// argument checks; conventions: include/rows8.h).  They return at once.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace hk {

// Codes go to `codes` as int8, or, when that is NULL, to `wide` as float16 whole
// numbers (for the tensor cores, which take no int8 on this GPU at speed).
cudaError_t rows8_quantize_launch(const void* X, int64_t ldx, int64_t n, int64_t d, int32_t dtype, int32_t group,
                                  int8_t* codes, int64_t ldc, uint16_t* wide, int64_t ldw, float* scale,
                                  cudaStream_t s);
// Two matrices of 8-bit rows (the second may have no rows) restored by one launch.
// scale == NULL: every scale is 1.  early: the stream's next kernel may start before the
// work in front of this launch is done (it has to wait for this one before it reads
// anything).
struct RestoreRows {
    const int8_t* codes = nullptr;
    int64_t ldc = 0;
    const float* scale = nullptr;
    int64_t n = 0, d = 0;
    int32_t group = 0;
    void* x = nullptr;
    int64_t ldx = 0;
};
cudaError_t rows8_restore_launch(const RestoreRows& a, const RestoreRows& b, int32_t dtype, bool early, cudaStream_t s);

}  // namespace hk
