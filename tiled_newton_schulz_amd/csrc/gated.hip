// The gated experts' block on gfx950, forward and backward (grouped_tiles.h has the
// kernels): launches.

#include "grouped_tiles.h"

namespace himuon {

template <int DT, bool WT>
static void gated_staged(const GroupedArgs& a, GroupedKernel k, dim3 grid, hipStream_t s) {
    if (a.gate == Gate::Forward) {
        if (k == GroupedKernel::Split64) hipLaunchKernelGGL((grouped_gated_staged<DT, WT, 64, 4>), grid, dim3(1024), 0, s, a);
        else if (k == GroupedKernel::Staged64) hipLaunchKernelGGL((grouped_gated_staged<DT, WT, 64, 1>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((grouped_gated_staged<DT, WT, 128, 1>), grid, dim3(256), 0, s, a);
    } else {
        if (k == GroupedKernel::Split64) hipLaunchKernelGGL((grouped_gated_grad_staged<DT, WT, 64, 4>), grid, dim3(1024), 0, s, a);
        else if (k == GroupedKernel::Staged64) hipLaunchKernelGGL((grouped_gated_grad_staged<DT, WT, 64, 1>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((grouped_gated_grad_staged<DT, WT, 128, 1>), grid, dim3(256), 0, s, a);
    }
}

template <int MODE, bool ERF>
static void gated_big(const GroupedArgs& a, int tiles, hipStream_t s) {
    const dim3 grid(grouped_big_grid(tiles)), threads(512);
    if (a.gate == Gate::Grad) hipLaunchKernelGGL((grouped_big<MODE, Gate::Grad, false, ERF>), grid, threads, 0, s, a, tiles);
    else if (a.p != nullptr) hipLaunchKernelGGL((grouped_big<MODE, Gate::Forward, true, ERF>), grid, threads, 0, s, a, tiles);
    else hipLaunchKernelGGL((grouped_big<MODE, Gate::Forward, false, ERF>), grid, threads, 0, s, a, tiles);
}

template <bool WT, bool ERF>
static void gated_thin(const GroupedArgs& a, dim3 grid, hipStream_t s) {
    if (a.gate == Gate::Grad) hipLaunchKernelGGL((grouped_mm_thin<WT, Gate::Grad, ERF>), grid, dim3(256), 0, s, a);
    else if (grouped_thin_cols(a) == kThinCols) hipLaunchKernelGGL((grouped_mm_thin<WT, Gate::Forward, ERF>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((grouped_mm_thin<WT, Gate::Forward, ERF, kThinCols / 2>), grid, dim3(256), 0, s, a);
}

hipError_t launch_grouped_gated(const GroupedArgs& a, bool trans_w, hipStream_t s) {
    const GroupedKernel k = grouped_mm_kernel(a);
    const int64_t tiles = grouped_mm_grid(a);
    const dim3 grid((uint32_t)tiles);
    if (k == GroupedKernel::Thin) {
        if (trans_w) a.erf ? gated_thin<true, true>(a, grid, s) : gated_thin<true, false>(a, grid, s);
        else a.erf ? gated_thin<false, true>(a, grid, s) : gated_thin<false, false>(a, grid, s);
    } else if (k == GroupedKernel::Big) {
        if (trans_w) a.erf ? gated_big<1, true>(a, (int)tiles, s) : gated_big<1, false>(a, (int)tiles, s);
        else a.erf ? gated_big<0, true>(a, (int)tiles, s) : gated_big<0, false>(a, (int)tiles, s);
    } else if (a.dtype == 0) {
        if (trans_w) gated_staged<0, true>(a, k, grid, s);
        else gated_staged<0, false>(a, k, grid, s);
    } else {
        if (trans_w) gated_staged<1, true>(a, k, grid, s);
        else gated_staged<1, false>(a, k, grid, s);
    }
    return hipGetLastError();
}

}  // namespace himuon
