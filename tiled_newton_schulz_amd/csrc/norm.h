// Internal declarations of layer normalisation (api_train.cpp, norm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace himuon {

constexpr int kMaxNormCols = 32768;   // matches HIMUON_MAX_NORM_COLS: a row is held by one workgroup

struct NormArgs {
    const void* x;         // N x D
    const void* weight;    // D, or null (1)
    const void* bias;      // D, or null (0); forward only
    int64_t x_ld;
    int32_t rows, cols;
    int32_t dtype;         // 0 bf16, 1 fp32
    float eps;
    void* y;               // forward: N x D
    int64_t y_ld;
    float* stats;          // N x 2: mean and 1 / std; written by a forward pass (or null), read by a gradient
    const void* dy;        // gradient: N x D
    int64_t dy_ld;
    void* dx;              // N x D, or null
    int64_t dx_ld;
    void* dw;              // D, or null
    void* db;              // D, or null
    float* part;           // workspace: 2 D sums of each workgroup
};

// Bytes of workspace a gradient needs where dw or db is asked for (else it takes none).
int64_t norm_grad_bytes(int32_t rows, int32_t cols, int32_t dtype);
hipError_t launch_layer_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_layer_norm_grad(const NormArgs& a, hipStream_t s);

}  // namespace himuon
