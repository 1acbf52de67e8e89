// Products of a mixture-of-experts layer on gfx950, grouped by expert with
// ragged sizes known only on the device:
//     product          Y[r, :] = X[r, :] W_e  (or W_e^T)   for the rows r of expert e
//     weight gradient  G_e = X_e^T D_e
//
// One launch covers up to 255 experts.  A workgroup takes its output tile from
// a linear id: every wave reads the experts' end rows (four slots a lane),
// counts the tiles of each expert with a prefix sum over the wave and finds
// the expert that holds the id, so no table has to be built on the host and
// the grid is only bounded there (ragged last tiles included).

#include <algorithm>

#include "device_util.h"
#include "grouped.h"

namespace himuon {
namespace {

struct GroupTile {
    int e;          // slot of the launch (a.n: the rows that belong to no expert)
    int row0;       // first row of the expert
    int rows;       // rows of the expert
    int mt, nt;     // tile of the expert's grid
};

// Rows [lo, hi) of slot i, clamped to the operand.
__device__ __forceinline__ void slot_rows(const GroupedArgs& a, int i, int& lo, int& hi) {
    const int g = a.e0 + i;
    lo = g > 0 ? min(max(a.ends[g - 1], 0), a.rows) : 0;
    hi = i < a.n ? min(max(a.ends[g], 0), a.rows) : a.rows;
}

// The tile of this workgroup in the product's launch; false if there is none.
// Tiles are counted expert by expert, the row tiles of one column tile next to
// each other (they share the weights' panel).  Consecutive tiles go to the
// workgroups of one XCD (workgroup ids go round the eight XCDs), so that the
// operands they share sit in one L2.
__device__ __forceinline__ bool find_tile(const GroupedArgs& a, int BM, int ntn, GroupTile& t) {
    const int lane = threadIdx.x & 63;
    const int slots = a.n + (a.last ? 1 : 0);
    int cnt[4], sum = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int i = lane * 4 + k;
        int lo = 0, hi = 0;
        if (i < slots) slot_rows(a, i, lo, hi);
        cnt[k] = hi > lo ? (hi - lo + BM - 1) / BM : 0;
        sum += cnt[k];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(incl, o, 64);
        if (lane >= o) incl += v;
    }
    const int64_t total = (int64_t)__shfl(incl, 63, 64) * ntn;
    const int64_t per = (total + 7) / 8;
    const int64_t id = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((int64_t)(blockIdx.x >> 3) >= per || id >= total) return false;
    int64_t excl = incl - sum;
    // the last lane whose first tile is at or before id
    const unsigned long long before = __ballot(excl * ntn <= id);
    const int src = 63 - __builtin_clzll(before);
    int64_t base = __shfl((int)excl, src, 64);
    int e = src * 4, c = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        c = __shfl(cnt[k], src, 64);
        e = src * 4 + k;
        if (id < (base + c) * ntn) break;
        base += c;
    }
    int lo, hi;
    slot_rows(a, e, lo, hi);
    t.e = e;
    t.row0 = lo;
    t.rows = hi - lo;
    const int64_t off = id - base * ntn;
    // always true where the end rows do not decrease; otherwise the tile is left out
    if (c <= 0 || off < 0 || off >= (int64_t)c * ntn) return false;
    t.mt = (int)(off % c);
    t.nt = (int)(off / c);
    return true;
}

template <int DT> struct Io;
template <> struct Io<0> {
    using T = unsigned short;
    static constexpr int BK = 32;
    __device__ static T cv(float f) { return f2bf(f); }
};
template <> struct Io<1> {
    using T = float;
    static constexpr int BK = 16;
    __device__ static T cv(float f) { return f; }
};

// C (64 x 64) += A (64 x k) B (k x 64) of one workgroup of four waves, each
// 32 x 32.  Element (i, k) of A sits at A[i * ai + k * ak], (k, j) of B at
// B[k * bk + j * bj]; elements past mi, kd or nj are zero.  Both panels are
// kept in LDS along k.
template <int DT>
__device__ __forceinline__ void tile64(const typename Io<DT>::T* A, int64_t ai, int64_t ak,
                                       const typename Io<DT>::T* B, int64_t bk, int64_t bj, int mi, int kd, int nj,
                                       f32x16& acc) {
    using T = typename Io<DT>::T;
    constexpr int BK = Io<DT>::BK;
    constexpr int LD = BK + (DT == 0 ? 8 : 1);
    __shared__ __attribute__((aligned(16))) T sA[64 * LD], sB[64 * LD];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int l32 = lane & 31, gl = lane >> 5, wm = wave >> 1, wn = wave & 1;
    for (int k0 = 0; k0 < kd; k0 += BK) {
        __syncthreads();
        for (int p = tid; p < 64 * BK; p += 256) {
            // consecutive threads along the operand's unit stride
            const int i = ak == 1 ? p / BK : p % 64, k = ak == 1 ? p % BK : p / 64;
            sA[i * LD + k] = (i < mi && k0 + k < kd) ? A[i * ai + (k0 + k) * ak] : T(0);
            const int j = bk == 1 ? p / BK : p % 64, kb = bk == 1 ? p % BK : p / 64;
            sB[j * LD + kb] = (j < nj && k0 + kb < kd) ? B[(k0 + kb) * bk + j * bj] : T(0);
        }
        __syncthreads();
        if constexpr (DT == 0) {
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk) {
                const u32x4 av = *reinterpret_cast<const u32x4*>(&sA[(wm * 32 + l32) * LD + kk * 16 + gl * 8]);
                const u32x4 bv = *reinterpret_cast<const u32x4*>(&sB[(wn * 32 + l32) * LD + kk * 16 + gl * 8]);
                acc = mfma32w(av, bv, acc);
            }
        } else {
#pragma unroll
            for (int kk = 0; kk < BK / 2; ++kk)
                acc = __builtin_amdgcn_mfma_f32_32x32x2f32(sA[(wm * 32 + l32) * LD + kk * 2 + gl],
                                                           sB[(wn * 32 + l32) * LD + kk * 2 + gl], acc, 0, 0, 0);
        }
    }
}

template <int DT>
__device__ __forceinline__ void store64(typename Io<DT>::T* C, int64_t ld, int mi, int nj, const f32x16& acc) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l32 = lane & 31, gl = lane >> 5, wm = wave >> 1, wn = wave & 1;
    const int j = wn * 32 + l32;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
        const int i = wm * 32 + (q >> 2) * 8 + gl * 4 + (q & 3);
        if (i < mi && j < nj) C[(int64_t)i * ld + j] = Io<DT>::cv(acc[q]);
    }
}

template <int DT, bool WT>
__global__ __launch_bounds__(256) void grouped_mm_kernel(const GroupedArgs a) {
    using T = typename Io<DT>::T;
    GroupTile t;
    if (!find_tile(a, 64, (a.ndim + 63) / 64, t)) return;
    const int m0 = t.row0 + t.mt * 64, n0 = t.nt * 64;
    const int mi = min(64, t.row0 + t.rows - m0), nj = min(64, a.ndim - n0);
    f32x16 acc{};
    if (t.e < a.n) {
        const T* W = reinterpret_cast<const T*>(a.w[t.e]);
        const int64_t ld = a.w_ld[t.e];
        tile64<DT>(reinterpret_cast<const T*>(a.x) + m0 * a.x_ld, a.x_ld, 1, WT ? W + n0 * ld : W + n0, WT ? 1 : ld,
                   WT ? ld : 1, mi, a.kdim, nj, acc);
    }
    store64<DT>(reinterpret_cast<T*>(a.y) + m0 * a.y_ld + n0, a.y_ld, mi, nj, acc);
}

template <int DT>
__global__ __launch_bounds__(256) void grouped_wgrad_kernel(const GroupedArgs a) {
    using T = typename Io<DT>::T;
    const int ntk = (a.kdim + 63) / 64, ntn = (a.ndim + 63) / 64;
    const int e = blockIdx.x / (ntk * ntn), b = blockIdx.x % (ntk * ntn);
    const int i0 = (b % ntk) * 64, j0 = (b / ntk) * 64;
    int lo, hi;
    slot_rows(a, e, lo, hi);
    const int mi = min(64, a.kdim - i0), nj = min(64, a.ndim - j0);
    f32x16 acc{};
    if (hi > lo)
        tile64<DT>(reinterpret_cast<const T*>(a.x) + lo * a.x_ld + i0, 1, a.x_ld,
                   reinterpret_cast<const T*>(a.d) + lo * a.d_ld + j0, a.d_ld, 1, mi, hi - lo, nj, acc);
    store64<DT>(reinterpret_cast<T*>(a.w[e]) + i0 * a.w_ld[e] + j0, a.w_ld[e], mi, nj, acc);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

int64_t grouped_mm_grid(const GroupedArgs& a) {
    // every slot ends in at most one partial row tile
    const int64_t row_tiles = a.rows / 64 + a.n + 1;
    return cdiv(row_tiles * cdiv(a.ndim, 64), 8) * 8;
}

int64_t grouped_wgrad_grid(const GroupedArgs& a) { return cdiv(a.kdim, 64) * cdiv(a.ndim, 64) * a.n; }

hipError_t launch_grouped_mm(const GroupedArgs& a, bool trans_w, hipStream_t s) {
    const dim3 grid((uint32_t)grouped_mm_grid(a));
    if (a.dtype == 0) {
        if (trans_w) hipLaunchKernelGGL((grouped_mm_kernel<0, true>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((grouped_mm_kernel<0, false>), grid, dim3(256), 0, s, a);
    } else {
        if (trans_w) hipLaunchKernelGGL((grouped_mm_kernel<1, true>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((grouped_mm_kernel<1, false>), grid, dim3(256), 0, s, a);
    }
    return hipGetLastError();
}

hipError_t launch_grouped_wgrad(const GroupedArgs& a, hipStream_t s) {
    const dim3 grid((uint32_t)grouped_wgrad_grid(a));
    if (a.dtype == 0) hipLaunchKernelGGL((grouped_wgrad_kernel<0>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((grouped_wgrad_kernel<1>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace himuon
