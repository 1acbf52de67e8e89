// Internal declarations of the two losses over logits (api_model.cpp,
// logits.hip): distillation from a teacher's top logits and log probabilities
// of given tokens.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace himuon {

constexpr int kMaxEntries = 1024;   // teacher entries of a row (matches HIMUON_MAX_ENTRIES)
constexpr int kMaxTop = 64;         // alternatives of a row (matches HIMUON_MAX_TOP)

// How the rows are cut for the passes that read them in segments: one workgroup
// of 256 threads reads `chunks` 16-byte chunks, at most 256 * u.
struct SegPlan {
    int32_t segs;     // segments of a row
    int32_t chunks;   // chunks of a segment
    int32_t u;        // chunks of a thread: 1, 2, 4 or 8
};

// Result of a segment in the workspace (m the largest logit, the sums relative to it).
struct SegStats {
    float m, s, e, pad;
};

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
    float* lse;               // N x 2 (value, rest); written by a forward pass, read by a gradient (null: not wanted)
    // token log probabilities
    const void* tokens;
    int32_t top;
    float* logp;
    float* entropy;           // written by the forward pass, read by the gradient
    int32_t* top_idx;
    float* top_logp;
    const float* g_logp;
    const float* g_entropy;
    // segments
    SegPlan plan;
    SegStats* part;           // workspace: rows x segs (segs > 1)
    uint64_t* keys;           // workspace: rows x segs x top (segs > 1)
};

SegPlan seg_plan(int32_t rows, int32_t cols, int32_t dtype);
// True if himuon_distill with a gradient keeps every row on chip (one launch,
// one pass over the logits).
bool distill_on_chip(int32_t cols, int32_t dtype);

hipError_t launch_distill(const LogitsArgs& a, hipStream_t s);         // loss (and lse)
hipError_t launch_distill_on_chip(const LogitsArgs& a, hipStream_t s); // loss, lse and gradient
hipError_t launch_distill_grad(const LogitsArgs& a, hipStream_t s);
hipError_t launch_logprobs(const LogitsArgs& a, hipStream_t s);
hipError_t launch_logprobs_grad(const LogitsArgs& a, hipStream_t s);

}  // namespace himuon
