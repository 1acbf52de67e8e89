// The gated experts' block on gfx950, forward pass (grouped_tiles.h has the kernels):
// launches.

#include "grouped_tiles.h"

namespace himuon {

template <int DT, bool WT>
static void staged(const GroupedArgs& a, GroupedKernel k, dim3 grid, hipStream_t s) {
    if (k == GroupedKernel::Split64) hipLaunchKernelGGL((grouped_gated_staged<DT, WT, 64, 4>), grid, dim3(1024), 0, s, a);
    else if (k == GroupedKernel::Staged64) hipLaunchKernelGGL((grouped_gated_staged<DT, WT, 64, 1>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((grouped_gated_staged<DT, WT, 128, 1>), grid, dim3(256), 0, s, a);
}

template <bool WT, GateKind KIND>
static void thin(const GroupedArgs& a, dim3 grid, hipStream_t s) {
    if constexpr (!WT) {   // (see grouped_thin_cols)
        if (grouped_thin_cols(a) == kThinCols) {
            hipLaunchKernelGGL((grouped_mm_thin<WT, Gate::Forward, KIND>), grid, dim3(256), 0, s, a);
            return;
        }
    }
    hipLaunchKernelGGL((grouped_mm_thin<WT, Gate::Forward, KIND, kThinCols / 2>), grid, dim3(256), 0, s, a);
}

template <int MODE, GateKind KIND>
static void big(const GroupedArgs& a, int tiles, hipStream_t s) {
    const dim3 grid(grouped_big_grid(tiles)), threads(512);
    if (a.p != nullptr) hipLaunchKernelGGL((grouped_big<MODE, Gate::Forward, true, KIND>), grid, threads, 0, s, a, tiles);
    else hipLaunchKernelGGL((grouped_big<MODE, Gate::Forward, false, KIND>), grid, threads, 0, s, a, tiles);
}

template <GateKind KIND>
static void aligned(const GroupedArgs& a, GroupedKernel k, int64_t tiles, hipStream_t s) {
    if (k == GroupedKernel::Thin) {
        if (a.nk) thin<true, KIND>(a, dim3((uint32_t)tiles), s);
        else thin<false, KIND>(a, dim3((uint32_t)tiles), s);
    } else {
        if (a.nk) big<1, KIND>(a, (int)tiles, s);
        else big<0, KIND>(a, (int)tiles, s);
    }
}

hipError_t launch_grouped_gated(const GroupedArgs& a, hipStream_t s) {
    const GroupedKernel k = grouped_mm_kernel(a);
    const int64_t tiles = grouped_mm_grid(a);
    const dim3 grid((uint32_t)tiles);
    if (k == GroupedKernel::Thin || k == GroupedKernel::Big) {
        if (a.kind == GateKind::Linear) aligned<GateKind::Linear>(a, k, tiles, s);
        else if (a.kind == GateKind::Cubic) aligned<GateKind::Cubic>(a, k, tiles, s);
        else if (a.kind == GateKind::Erf) aligned<GateKind::Erf>(a, k, tiles, s);
        else aligned<GateKind::Step>(a, k, tiles, s);
    } else if (a.dtype == 0) {
        if (a.nk) staged<0, true>(a, k, grid, s);
        else staged<0, false>(a, k, grid, s);
    } else {
        if (a.nk) staged<1, true>(a, k, grid, s);
        else staged<1, false>(a, k, grid, s);
    }
    return hipGetLastError();
}

}  // namespace himuon
