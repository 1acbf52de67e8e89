// Internal declarations of the AdamW step (api_train.cpp, adamw.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace himuon {

constexpr int kAdamwTensors = 256;     // tensors of a launch (kernel-argument table, 22 KB)
constexpr int64_t kAdamwBlock = 256;   // elements that share a scale (matches HIMUON_ADAMW_BLOCK)
constexpr int64_t kAdamwUnit = 4096;   // elements a workgroup takes at a time

struct AdamwTensor {
    void* w;
    const void* g;
    void* m;              // fp32, or e4m3 codes
    void* v;              // fp32, or e4m3 codes of sqrt(v)
    float* m_scale;       // 8 bits: one for each block
    float* v_scale;
    int64_t numel;
    int64_t cols;         // 0: both w and g are without gaps between rows
    int64_t w_ld, g_ld;
    uint32_t first;       // units of the launch before this tensor's
};
struct AdamwArgs {
    AdamwTensor t[kAdamwTensors];
    int32_t n;
    int32_t w_dtype, g_dtype;   // 0 bf16, 1 fp32
    int32_t bits;
    uint32_t units;             // of the launch
    uint32_t key;               // of the step's random bits
    float beta1, rest1;         // beta, 1 - beta
    float beta2, rest2;
    float keep;                 // 1 - lr weight_decay
    float rate;                 // lr / (1 - beta1^t)
    float root;                 // 1 / sqrt(1 - beta2^t)
    float eps;
    const float* grad_scale;    // device scalar, or null (1)
};

hipError_t launch_adamw(const AdamwArgs& a, hipStream_t s);

}  // namespace himuon
