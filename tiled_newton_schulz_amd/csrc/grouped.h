// Internal declarations of the experts' products (api_model.cpp, grouped.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace himuon {

// Experts of one launch.  With the rows that belong to no expert as one more
// slot they fill four slots for each lane of a wave (find_tile in grouped.hip).
constexpr int kExperts = 255;

// Longest side: the kernels step past an end by less than this leaves to 2^31.
constexpr int64_t kMaxSide = INT32_MAX - 4096;

// One launch of Y = X W_e (or X W_e^T) or of G_e = X_e^T D_e.
struct GroupedArgs {
    const void* x;           // M x K
    const void* d;           // weight gradient: M x N
    void* y;                 // product: M x N
    int64_t x_ld, d_ld, y_ld;
    const int32_t* ends;     // device: end row of every expert of the call
    int32_t rows;            // M
    int32_t kdim, ndim;      // K, N
    int32_t e0, n;           // experts [e0, e0 + n) of the call
    int32_t total;           // experts of the call
    int32_t last;            // product: this launch also zeroes the rows past the last expert
    int32_t dtype;           // 0 bf16, 1 fp32
    int32_t vec;             // rows and widths allow 16-byte chunks
    float* sums;             // weight gradient: workspace of the parts' sums, or null
    int32_t parts;           // weight gradient: parts an expert's rows are cut into
    void* w[kExperts];       // product: weights; weight gradient: results
    int64_t w_ld[kExperts];
};

// True if a launch can hold the tiles (checked before any launch).
bool grouped_mm_fits(const GroupedArgs& a);
bool grouped_wgrad_fits(const GroupedArgs& a);
// Parts worth cutting the experts' rows of a weight gradient into (1: none), and
// the workspace of a part.
int32_t grouped_wgrad_parts(const GroupedArgs& a);
int64_t grouped_wgrad_part_bytes(const GroupedArgs& a);
hipError_t launch_grouped_mm(const GroupedArgs& a, bool trans_w, hipStream_t s);
hipError_t launch_grouped_wgrad(const GroupedArgs& a, hipStream_t s);

}  // namespace himuon
