// Products of a mixture-of-experts layer on gfx950 (grouped_tiles.h has the
// kernels): which kernel a call takes, and its launches.

#include "grouped_tiles.h"

namespace himuon {
namespace {

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

int device_cus_or_256() {
    static const int cus = [] { const int c = device_cus(); return c >= 8 ? std::min(c, 512) : 256; }();
    return cus;
}

// Column tiles: in a gated block's forward pass half a tile's columns are the gate's.
int64_t col_tiles(const GroupedArgs& a, int edge) { return cdiv(a.ndim, a.gate == Gate::Forward ? edge / 2 : edge); }
int64_t mm_tiles(const GroupedArgs& a, int edge) {
    // every slot ends in at most one partial row tile
    return (a.rows / edge + a.n + 1) * col_tiles(a, edge);
}
int64_t wgrad_tiles(const GroupedArgs& a, int edge) { return cdiv(a.kdim, edge) * cdiv(a.ndim, edge) * a.n; }

// Tiles to expect: the host knows the rows and the experts, not which expert has
// how many; half a partial row tile each.  Of the whole call: where it takes more
// than one launch they all run the same kernel.  (The last launch of 256 experts
// holds one: planned by its share of the rows, calls of 1024 x 512 took 60 instead
// of 72 us at 32 rows an expert, but 148 instead of 132 us at 256, as its grid has
// to hold all rows and nearly all of it is empty.)
double mm_expect(const GroupedArgs& a, int edge) {
    return ((double)a.rows / edge + 0.5 * a.total) * (double)col_tiles(a, edge);
}

// Which kernel.  Measured in us, experts x rows x K x N (K x N stored, bf16):
//                           thin   256-tiles   staged 128   staged 64
//   64 x  16 x 4096 x 1408   134         148
//   64 x  17 x 4096 x 1408   160         147
//    1 x 512 x 1024 x 1024   8.7          25           11          11
//    8 x 128 x 2048 x 2048    46          39           36          27
//    8 x 512 x 4096 x 1024   140          78           65          65
//    2 x 2048 x 512 x 2048    78          21           21          25
// so: thin up to 16 rows an expert (32 where 256-tiles are too few), 256-tiles
// from three quarters of a tile a CU, else staged with tiles of 128 from one a
// CU.  Weight gradients alike: 1 x 1024 x 1024 x 1024 (16 tiles of 256) 30
// against 7 us staged, 1 x 256 x 4096 x 4096 (256 tiles) 19 against 27 us.
using Kernel = GroupedKernel;
bool enough_big(double tiles) { return tiles >= 0.75 * device_cus_or_256(); }
// Four parts of a workgroup share a tile's steps; one such workgroup fits a CU.
// In us without and with: weight gradients 2 x 4528 x 925 x 39 35 and 22, 1 x
// 1024 x 512 x 512 11.9 and 9.4, 16 x 8192 x 256 x 256 (8 steps) 9.3 and 8.8;
// products (rows of all experts) 4 x 300 x 4095 x 500 55 and 30, in fp32 129
// and 93, with K = 512 in fp32 19.6 and 17.4.
bool split(const GroupedArgs& a, double tiles, int64_t k) {
    return tiles <= device_cus_or_256() && k >= 8 * (a.dtype == 0 ? Io<0>::BK : Io<1>::BK);
}
}  // namespace

Kernel grouped_mm_kernel(const GroupedArgs& a) {
    if (a.dtype == 0 && a.vec) {
        const bool big = enough_big(mm_expect(a, kBig));
        if (a.rows <= (big ? 16 : 32) * (int64_t)a.total) return Kernel::Thin;
        if (big) return Kernel::Big;
    }
    if (mm_expect(a, 128) >= device_cus_or_256()) return Kernel::Staged128;
    return split(a, mm_expect(a, 64), a.kdim) ? Kernel::Split64 : Kernel::Staged64;
}
namespace {

Kernel wgrad_kernel(const GroupedArgs& a) {
    if (a.dtype == 0 && a.vec && enough_big((double)wgrad_tiles(a, kBig))) return Kernel::Big;
    if (wgrad_tiles(a, 128) >= device_cus_or_256()) return Kernel::Staged128;
    return split(a, (double)wgrad_tiles(a, 64), a.rows / a.total) ? Kernel::Split64 : Kernel::Staged64;
}
int edge_of(Kernel k) { return k == Kernel::Big ? kBig : k == Kernel::Staged128 ? 128 : 64; }

}  // namespace

// A gated block's forward pass reads K x N weights in pieces of 64 or 128 bytes of a row:
// 64 experts of 4096 x 2 x 1408, 96 rows, 234 against 216 us, so 64 columns of H where
// there are tiles enough; stored N x K the 32 take 252 and the 64 267 us (fewer tiles,
// one workgroup a CU), so 32 columns.
int grouped_thin_cols(const GroupedArgs& a) {
    if (a.gate != Gate::Forward) return kThinCols;
    return !a.nk && (double)a.total * (double)cdiv(a.ndim, kThinCols) >= device_cus_or_256() ? kThinCols : kThinCols / 2;
}

// Most tiles of a launch, whole rounds of the XCDs.
int64_t grouped_mm_grid(const GroupedArgs& a) {
    const Kernel k = grouped_mm_kernel(a);
    if (k == Kernel::Thin) return cdiv((a.rows / kThinRows + a.n + 1) * cdiv(a.ndim, grouped_thin_cols(a)), 8) * 8;
    return cdiv(mm_tiles(a, edge_of(k)), 8) * 8;
}

namespace {

int64_t grouped_wgrad_grid(const GroupedArgs& a) { return cdiv(wgrad_tiles(a, edge_of(wgrad_kernel(a))), 8) * 8; }

// A workgroup a tile, and at most 2^32 - 1 threads a launch; the 256-tiles have
// workgroups of their own number and count tiles in an int.
bool fits(Kernel k, int64_t tiles) {
    if (k == Kernel::Big) return tiles <= INT32_MAX / 2;
    return tiles <= UINT32_MAX / (k == Kernel::Split64 ? 1024 : 256);
}

}  // namespace

bool grouped_mm_fits(const GroupedArgs& a) { return fits(grouped_mm_kernel(a), grouped_mm_grid(a)); }
bool grouped_wgrad_fits(const GroupedArgs& a) { return fits(wgrad_kernel(a), grouped_wgrad_grid(a)); }

// Where the tiles split in a workgroup are few and the rows many, the rows are cut
// into the parts that should take the least time: rounds of one workgroup a CU, at
// 1.1 us (fp32: 2.6) for a workgroup's four steps, at least four times these a
// part; 5 us for the join, and its bytes.  In us without and with, 256 x 256: bf16
// 2048 rows 12.4 and 11.8 on the device and 12.6 and 15.6 with the host's calls
// (so not cut), 3000 rows 16.4 and 13.8, 8192 rows 37 and 13.5; fp32 1024 rows 25
// and 18, 4096 rows 85 and 20.  32768 x 512 x 512 in bf16: 160 and 50.
constexpr int64_t kMostParts = 1024;   // of all tiles: 16 MiB
int32_t grouped_wgrad_parts(const GroupedArgs& a) {
    if (wgrad_kernel(a) != Kernel::Split64) return 1;
    const int64_t steps = a.rows / a.total / (a.dtype == 0 ? Io<0>::BK : Io<1>::BK), tiles = wgrad_tiles(a, 64);
    int64_t best = 1;
    double least = 1e30;
    for (int64_t p = 1; p == 1 || (p <= steps / 16 && p * tiles <= kMostParts); ++p) {
        const double rounds = (double)cdiv(tiles * p, device_cus_or_256()) * (double)steps / (4.0 * (double)p);
        const double t = rounds * (a.dtype == 0 ? 1.1 : 2.6) + (p > 1 ? 5.0 + 0.0067 * (double)(p * tiles) : 0.0);
        if (t < least) {
            least = t;
            best = p;
        }
    }
    return (int32_t)best;
}
int64_t grouped_wgrad_part_bytes(const GroupedArgs& a) { return wgrad_tiles(a, 64) * 64 * 64 * 4; }

// Workgroups of the 256 x 256 kernel for at most `tiles` tiles: one fits a CU.
uint32_t grouped_big_grid(int64_t tiles) { return (uint32_t)std::min<int64_t>(tiles, device_cus_or_256() / 8 * 8); }

template <int DT, bool WT>
static void mm_staged(const GroupedArgs& a, Kernel k, dim3 grid, hipStream_t s) {
    if (k == Kernel::Split64) hipLaunchKernelGGL((grouped_mm_staged<DT, WT, 64, 4>), grid, dim3(1024), 0, s, a);
    else if (k == Kernel::Staged64) hipLaunchKernelGGL((grouped_mm_staged<DT, WT, 64, 1>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((grouped_mm_staged<DT, WT, 128, 1>), grid, dim3(256), 0, s, a);
}

hipError_t launch_grouped_mm(const GroupedArgs& a, bool trans_w, hipStream_t s) {
    const Kernel k = grouped_mm_kernel(a);
    const int64_t tiles = grouped_mm_grid(a);
    const dim3 grid((uint32_t)tiles);
    if (k == Kernel::Thin) {
        if (trans_w) hipLaunchKernelGGL((grouped_mm_thin<true>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((grouped_mm_thin<false>), grid, dim3(256), 0, s, a);
    } else if (k == Kernel::Big) {
        if (trans_w) hipLaunchKernelGGL((grouped_big<1>), dim3(grouped_big_grid(tiles)), dim3(512), 0, s, a, (int)tiles);
        else hipLaunchKernelGGL((grouped_big<0>), dim3(grouped_big_grid(tiles)), dim3(512), 0, s, a, (int)tiles);
    } else if (a.dtype == 0) {
        if (trans_w) mm_staged<0, true>(a, k, grid, s);
        else mm_staged<0, false>(a, k, grid, s);
    } else {
        if (trans_w) mm_staged<1, true>(a, k, grid, s);
        else mm_staged<1, false>(a, k, grid, s);
    }
    return hipGetLastError();
}

template <int DT>
static void wgrad_staged(const GroupedArgs& a, Kernel k, dim3 grid, hipStream_t s) {
    if (k == Kernel::Split64 && a.parts > 1) {
        const int64_t tiles = wgrad_tiles(a, 64);
        hipLaunchKernelGGL((grouped_wgrad_staged<DT, 64, 4, true>), dim3((uint32_t)(cdiv(tiles * a.parts, 8) * 8)),
                           dim3(1024), 0, s, a);
        hipLaunchKernelGGL((grouped_wgrad_join<DT>), dim3((uint32_t)tiles), dim3(256), 0, s, a);
    } else if (k == Kernel::Split64) {
        hipLaunchKernelGGL((grouped_wgrad_staged<DT, 64, 4, false>), grid, dim3(1024), 0, s, a);
    } else if (k == Kernel::Staged64) {
        hipLaunchKernelGGL((grouped_wgrad_staged<DT, 64, 1, false>), grid, dim3(256), 0, s, a);
    } else {
        hipLaunchKernelGGL((grouped_wgrad_staged<DT, 128, 1, false>), grid, dim3(256), 0, s, a);
    }
}

hipError_t launch_grouped_wgrad(const GroupedArgs& a, hipStream_t s) {
    const Kernel k = wgrad_kernel(a);
    const int64_t tiles = grouped_wgrad_grid(a);
    const dim3 grid((uint32_t)tiles);
    if (k == Kernel::Big)
        hipLaunchKernelGGL((grouped_big<2>), dim3(grouped_big_grid(tiles)), dim3(512), 0, s, a, (int)tiles);
    else if (a.dtype == 0) wgrad_staged<0>(a, k, grid, s);
    else wgrad_staged<1>(a, k, grid, s);
    return hipGetLastError();
}

}  // namespace himuon
