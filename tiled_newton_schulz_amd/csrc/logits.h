// Internal declarations of the two losses over logits (api_model.cpp,
// logits.hip): distillation from a teacher's top logits and log probabilities
// of given tokens.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace himuon {

constexpr int kMaxEntries = 1024;   // teacher entries of a row (matches HIMUON_MAX_ENTRIES)
constexpr int kMaxTop = 64;         // alternatives of a row (matches HIMUON_MAX_TOP)

struct LogitsArgs {
    const void* z;            // N x V logits
    void* dz;                 // gradient, or null
    int64_t z_ld, dz_ld;
    int32_t rows, cols;       // N, V
    int32_t dtype;            // 0 bf16, 1 fp32
    int32_t idx64;            // ids are int64
    float inv_temp;
    // distillation
    const void* idx;          // N x k ids
    const float* t;           // N x k teacher values
    int64_t t_ld;
    int32_t k, normalize;
    const float* weight;      // forward: null = 1; gradient: dL/dloss
    float* loss;
    float* lse;               // N x 2 (value, rest); written by a forward pass, read by a gradient (may be null in a forward pass)
    // token log probabilities
    const void* tokens;
    int32_t top;
    float* logp;
    float* entropy;           // written by the forward pass, read by the gradient
    int32_t* top_idx;
    float* top_logp;
    const float* g_logp;
    const float* g_entropy;
};

hipError_t launch_distill(const LogitsArgs& a, hipStream_t s);
hipError_t launch_distill_grad(const LogitsArgs& a, hipStream_t s);
hipError_t launch_logprobs(const LogitsArgs& a, hipStream_t s);
hipError_t launch_logprobs_grad(const LogitsArgs& a, hipStream_t s);

}  // namespace himuon
