// m3_norm.h -- parameter block and launch functions of the root-mean-square norm's
// kernels (internal to the library; the public ABI is include/m3.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "m3.h"

namespace m3 {

// root-mean-square norm (k_norm.cu)
struct NormParams {
    long long rows;
    int width;
    float eps;
    const void* x;             // [row][width] io (gradient: the norm's input, the stored sum)
    const void* residual;      // io, nullable
    const float* weight;       // [width], nullable (ones)
    void* sum;                 // io, nullable
    void* y;                   // io, nullable
    uint8_t* y8;               // e4m3, nullable
    float* scale;              // [row][blocks]
    int block;                 // columns a scale: 0 = the row, or 128
    // gradient
    const void* dy;            // io
    const void* d_sum;         // io, nullable
    void* dx;                  // io
    float* dweight;            // [width], nullable
    float* part;               // [parts][width]
    int parts;
};
int norm_bwd_parts(long long rows, int width, int io_dtype);
cudaError_t launch_norm(int io_dtype, const NormParams& q, cudaStream_t st);
cudaError_t launch_norm_bwd(int io_dtype, const NormParams& q, cudaStream_t st);

}  // namespace m3
