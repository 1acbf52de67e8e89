// Internal declarations of the experts' products (api_model.cpp,
// grouped.hip, gated.hip, gated_grad.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace himuon {

// Experts of one launch.  With the rows that belong to no expert as one more
// slot they fill four slots for each lane of a wave (find_tile in grouped.hip).
constexpr int kExperts = 255;

// Longest side: the kernels step past an end by less than this leaves to 2^31.
constexpr int64_t kMaxSide = INT32_MAX - 4096;

// A product's part in a gated block (grouped.hip).
enum class Gate : int32_t {
    None,       // Y = X W_e
    Forward,    // W_e holds the gate's and the up projection: Y = act(G) * U
    Grad        // X W_e^T is the gradient of that Y: gradients of G and U
};

// What s is in act(g) = g s(g): sigmoid(k0 g), sigmoid(k0 g + k1 g^3), the integral of
// the normal distribution, or 1 above 0 and else 0.
enum class GateKind : int32_t { Linear, Cubic, Erf, Step };

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
    // gated block: N = ndim is the width of H; y is H (Forward) or D (Grad, M x 2N)
    Gate gate;
    int32_t nk;              // weights stored N x K (2N x K)
    void* p;                 // [G | U], M x 2N: written by Forward (or null), read by Grad
    void* h;                 // Grad: H, or null
    int64_t p_ld, h_ld;
    GateKind kind;           // act(g) = g s(g), with k0, k1
    float k0, k1;
    void* w[kExperts];       // product: weights; weight gradient: results
    int64_t w_ld[kExperts];
};

// Which kernel a product takes (rules and measurements: grouped.hip), the most
// workgroups or tiles of its launch, and the workgroups of the 256 x 256 kernel.
enum class GroupedKernel { Thin, Big, Staged128, Staged64, Split64 };
GroupedKernel grouped_mm_kernel(const GroupedArgs& a);
int grouped_thin_cols(const GroupedArgs& a);   // of a tile's result (Thin)
int64_t grouped_mm_grid(const GroupedArgs& a);
uint32_t grouped_big_grid(int64_t tiles);

// True if a launch can hold the tiles (checked before any launch).
bool grouped_mm_fits(const GroupedArgs& a);
bool grouped_wgrad_fits(const GroupedArgs& a);
// Parts worth cutting the experts' rows of a weight gradient into (1: none), and
// the workspace of a part.
int32_t grouped_wgrad_parts(const GroupedArgs& a);
int64_t grouped_wgrad_part_bytes(const GroupedArgs& a);
hipError_t launch_grouped_mm(const GroupedArgs& a, bool trans_w, hipStream_t s);
hipError_t launch_grouped_wgrad(const GroupedArgs& a, hipStream_t s);
// a.gate == Forward; a.gate == Grad.
hipError_t launch_grouped_gated(const GroupedArgs& a, hipStream_t s);
hipError_t launch_grouped_gated_grad(const GroupedArgs& a, hipStream_t s);

}  // namespace himuon
