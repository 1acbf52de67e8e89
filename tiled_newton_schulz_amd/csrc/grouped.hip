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
    // the same in every lane: scalar registers
    t.e = __builtin_amdgcn_readfirstlane(e);
    t.row0 = __builtin_amdgcn_readfirstlane(lo);
    t.rows = __builtin_amdgcn_readfirstlane(hi - lo);
    const int64_t off = id - base * ntn;
    // always true where the end rows do not decrease; otherwise the tile is left out
    if (c <= 0 || off < 0 || off >= (int64_t)c * ntn) return false;
    t.mt = __builtin_amdgcn_readfirstlane((int)off % c);
    t.nt = __builtin_amdgcn_readfirstlane((int)off / c);
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
    if ((int)blockIdx.x >= a.n * ntk * ntn) return;
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

// ---------------------------------------------------------------------------
// bf16 operands of 16-byte chunks: 256 x 256 tiles, k in steps of 64, eight
// waves (2 along the rows, 4 along the columns), two LDS stages filled straight
// from global memory.
//
// Ragged tiles: the 32 x 32 blocks of a wave interleave with the other waves'
// (rows (2 i + wm) 32, columns (4 j + wn) 32), so a tile of r rows and c columns
// costs FM = ceil(r / 64) by FN = ceil(c / 128) blocks in every wave, and the
// loop is compiled for each FM and FN.
//
// An operand is stored in memory either along k (rows i of k) or along its
// other side (rows k of i), and its LDS stage keeps that order:
//   along k: 256 rows of 8 16-byte chunks, chunk c of row r at place c ^ (r & 7)
//   along i: two sub-panels of 64 k rows of 128 elements, chunk c of row k at
//            place c ^ (4 (k & 3)); read transposed (ds_read_tr16_b64)
// The products run with the operands exchanged (columns as the MFMA's rows), so
// that a lane ends with runs of four consecutive columns of one row.
// ---------------------------------------------------------------------------
constexpr int kBig = 256;             // tile edge
constexpr int kBK = 64;
constexpr int kStage = kBig * kBK;    // elements of one operand's stage
constexpr int kLdc = kBig + 8;        // row stride of the result in LDS

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Buffer descriptor of [p, p + bytes): loads past it give zeros.
__device__ __forceinline__ i32x4 rsrc_words(const void* p, uint32_t bytes) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    return i32x4{(int)(uint32_t)u, (int)(uint32_t)(u >> 32) & 0xffff, (int)bytes, 0x00020000};
}
// 64 lanes x 16 bytes from r + off to LDS byte address lds + 16 lane.  As
// inline assembly, since the compiler makes every transposed LDS read wait for
// all such loads it knows of; the waits are in stage_ready().  It has no
// register result, so nothing can be read or reused too early.
__device__ __forceinline__ void dma16(i32x4 r, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :: "s"(lds), "v"(off), "s"(r) : "memory");
}
// Every load of this wave has landed and its LDS reads are done; then the same
// of all waves.
__device__ __forceinline__ void stage_ready() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// One operand of a tile: up to 256 rows or columns (`side`) by k.
template <bool ALONG_K>
struct Panel {
    const unsigned short* p;   // element (0, 0) of the tile at k = 0
    int64_t ld;
    int side;                  // rows (or columns) of the tile inside the operand
    int kd;                    // length of k

    // instructions a wave issues for B blocks of 32 * (waves along the side)
    static constexpr int count(int units64) { return ALONG_K ? units64 : 2 * ((units64 + 1) / 2); }

    // byte offset of instruction j of this wave from the step's first byte
    __device__ __forceinline__ uint32_t offset(int j, int wave, int lane) const {
        const int pos = (j * 8 + wave) * 64 + lane;
        if (ALONG_K) {
            const int r = pos >> 3, c = (pos & 7) ^ (r & 7);
            // rows past the operand go past the buffer's end
            return r < side ? (uint32_t)(r * (uint32_t)ld * 2u) + c * 16u : 0xffffff00u;
        }
        const int sub = pos >> 10, k = (pos & 1023) >> 4, c = (pos & 15) ^ ((k & 3) * 4);
        const int i = sub * 128 + c * 8;
        return i < side ? (uint32_t)(k * (uint32_t)ld * 2u) + i * 2u : 0xffffff00u;
    }
    // first k element of the chunk (stored along k)
    static __device__ __forceinline__ int chunk_k(int j, int wave, int lane) {
        const int pos = (j * 8 + wave) * 64 + lane, r = pos >> 3;
        return ((pos & 7) ^ (r & 7)) * 8;
    }
    // the operand's bytes from step k0 on (the last row that counts ends them)
    __device__ __forceinline__ i32x4 rsrc(int k0) const {
        if (ALONG_K) return rsrc_words(p + k0, (uint32_t)(((side - 1) * ld + kd - k0) * 2));
        const int rows = min(kBK, kd - k0);
        return rsrc_words(p + k0 * ld, (uint32_t)(((rows - 1) * ld + side) * 2));
    }
    // MFMA operand of the 32-wide block at `first`, k sub-step kk
    static __device__ __forceinline__ bf16x8 read(const unsigned short* st, int first, int kk, int lane) {
        if (ALONG_K) {
            const int r = first + (lane & 31), c = (kk * 2 + (lane >> 5)) ^ (r & 7);
            return *reinterpret_cast<const bf16x8*>(&st[r * kBK + c * 8]);
        }
        const int i16 = lane & 15;
        const int col = first + 16 * ((lane >> 4) & 1) + 4 * (i16 & 3);
        const int k = kk * 16 + 8 * (lane >> 5) + (i16 >> 2);
        const int cl = col & 127;
        const unsigned short* q = &st[(col >> 7) * (kBK * 128) + k * 128 + (((cl >> 3) ^ ((k & 3) * 4)) * 8) + (cl & 7)];
        const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LDS_AS bf16x4*)(q));
        const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LDS_AS bf16x4*)(q + 4 * 128));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

template <bool AK, bool BK_, int FM, int FN>
__device__ __forceinline__ void big_tile(const Panel<AK>& A, const Panel<BK_>& B, unsigned short* sbuf,
                                         unsigned short* C, int64_t ldc) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    constexpr int NA = Panel<AK>::count(FM), NB = Panel<BK_>::count(2 * FN);
    uint32_t oa[NA], ob[NB];
#pragma unroll
    for (int j = 0; j < NA; ++j) oa[j] = A.offset(j, wave, lane);
#pragma unroll
    for (int j = 0; j < NB; ++j) ob[j] = B.offset(j, wave, lane);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(LDS_AS void*)sbuf;
    const int nk = (A.kd + kBK - 1) / kBK;

    auto issue = [&](int kt) __attribute__((always_inline)) {
        const int k0 = kt * kBK;
        const i32x4 ra = A.rsrc(k0), rb = B.rsrc(k0);
        const uint32_t la = lds0 + (kt & 1) * (2 * kStage * 2) + wave * 1024, lb = la + kStage * 2;
        // a last step that k does not fill: chunks past its end would read the
        // next row, so they go past the buffer's end too
        const int left = A.kd - k0;
#pragma unroll
        for (int j = 0; j < NA; ++j)
            dma16(ra, AK && left < kBK && Panel<AK>::chunk_k(j, wave, lane) >= left ? 0xffffff00u : oa[j], la + j * 8192);
#pragma unroll
        for (int j = 0; j < NB; ++j)
            dma16(rb, BK_ && left < kBK && Panel<BK_>::chunk_k(j, wave, lane) >= left ? 0xffffff00u : ob[j], lb + j * 8192);
    };

    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{};

    if (nk > 0) issue(0);
    for (int kt = 0; kt < nk; ++kt) {
        stage_ready();
        if (kt + 1 < nk) issue(kt + 1);
        const unsigned short* sa = sbuf + (kt & 1) * 2 * kStage;
        const unsigned short* sb = sa + kStage;
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk) {
            bf16x8 av[FM], bv[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i) av[i] = Panel<AK>::read(sa, (i * 2 + wm) * 32, kk, lane);
#pragma unroll
            for (int j = 0; j < FN; ++j) bv[j] = Panel<BK_>::read(sb, (j * 4 + wn) * 32, kk, lane);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bv[j], av[i], acc[i][j], 0, 0, 0);
        }
    }

    // result through LDS, then whole 16-byte chunks of rows
    __syncthreads();
    const int l32 = lane & 31, gl = lane >> 5;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const u32x2 v = {pack2(acc[i][j][4 * m], acc[i][j][4 * m + 1]),
                                 pack2(acc[i][j][4 * m + 2], acc[i][j][4 * m + 3])};
                *reinterpret_cast<u32x2*>(&sbuf[((i * 2 + wm) * 32 + l32) * kLdc + (j * 4 + wn) * 32 + m * 8 + gl * 4]) = v;
            }
    __syncthreads();
    constexpr int CH = FN * 16;   // chunks of a row
#pragma unroll
    for (int it = 0; it < FM * 64 * CH / 512; ++it) {
        const int id = it * 512 + tid, r = id / CH, c = (id % CH) * 8;
        if (r < A.side && c < B.side)
            *reinterpret_cast<u32x4*>(C + r * ldc + c) = *reinterpret_cast<const u32x4*>(&sbuf[r * kLdc + c]);
    }
}

template <bool AK, bool BK_>
__device__ __forceinline__ void big_dispatch(const Panel<AK>& A, const Panel<BK_>& B, unsigned short* sbuf,
                                             unsigned short* C, int64_t ldc) {
    const int fm = (A.side + 63) / 64;
    if (B.side > 128) {
        if (fm == 4) big_tile<AK, BK_, 4, 2>(A, B, sbuf, C, ldc);
        else if (fm == 3) big_tile<AK, BK_, 3, 2>(A, B, sbuf, C, ldc);
        else if (fm == 2) big_tile<AK, BK_, 2, 2>(A, B, sbuf, C, ldc);
        else big_tile<AK, BK_, 1, 2>(A, B, sbuf, C, ldc);
    } else {
        if (fm == 4) big_tile<AK, BK_, 4, 1>(A, B, sbuf, C, ldc);
        else if (fm == 3) big_tile<AK, BK_, 3, 1>(A, B, sbuf, C, ldc);
        else if (fm == 2) big_tile<AK, BK_, 2, 1>(A, B, sbuf, C, ldc);
        else big_tile<AK, BK_, 1, 1>(A, B, sbuf, C, ldc);
    }
}

template <bool WT>
__global__ __launch_bounds__(512) void grouped_mm_big(const GroupedArgs a) {
    __shared__ __attribute__((aligned(16))) unsigned short sbuf[kBig * kLdc];
    GroupTile t;
    if (!find_tile(a, kBig, (a.ndim + kBig - 1) / kBig, t)) return;
    const int64_t m0 = t.row0 + t.mt * kBig;
    const int n0 = t.nt * kBig;
    Panel<true> A{reinterpret_cast<const unsigned short*>(a.x) + m0 * a.x_ld, a.x_ld,
                  min(kBig, t.rows - t.mt * kBig), a.kdim};
    Panel<WT> B{nullptr, 0, min(kBig, a.ndim - n0), a.kdim};
    if (t.e < a.n) {
        B.ld = a.w_ld[t.e];
        B.p = reinterpret_cast<const unsigned short*>(a.w[t.e]) + (WT ? n0 * B.ld : n0);
    } else {
        A.kd = B.kd = 0;   // rows of no expert: zeros
    }
    big_dispatch<true, WT>(A, B, sbuf, reinterpret_cast<unsigned short*>(a.y) + m0 * a.y_ld + n0, a.y_ld);
}

__global__ __launch_bounds__(512) void grouped_wgrad_big(const GroupedArgs a) {
    __shared__ __attribute__((aligned(16))) unsigned short sbuf[kBig * kLdc];
    const int ntk = (a.kdim + kBig - 1) / kBig, ntn = (a.ndim + kBig - 1) / kBig;
    const int total = a.n * ntk * ntn, per = (total + 7) / 8;
    const int id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || id >= total) return;
    const int e = id / (ntk * ntn), b = id % (ntk * ntn);
    const int i0 = (b % ntk) * kBig, j0 = (b / ntk) * kBig;
    int lo, hi;
    slot_rows(a, e, lo, hi);
    lo = __builtin_amdgcn_readfirstlane(lo);
    const int kd = __builtin_amdgcn_readfirstlane(max(hi - lo, 0));
    const Panel<false> A{reinterpret_cast<const unsigned short*>(a.x) + lo * a.x_ld + i0, a.x_ld, min(kBig, a.kdim - i0), kd};
    const Panel<false> B{reinterpret_cast<const unsigned short*>(a.d) + lo * a.d_ld + j0, a.d_ld, min(kBig, a.ndim - j0), kd};
    big_dispatch<false, false>(A, B, sbuf, reinterpret_cast<unsigned short*>(a.w[e]) + i0 * a.w_ld[e] + j0, a.w_ld[e]);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

int tile_edge(const GroupedArgs& a) { return a.dtype == 0 && a.vec ? kBig : 64; }

}  // namespace

int64_t grouped_mm_grid(const GroupedArgs& a) {
    // every slot ends in at most one partial row tile
    const int edge = tile_edge(a);
    const int64_t row_tiles = a.rows / edge + a.n + 1;
    return cdiv(row_tiles * cdiv(a.ndim, edge), 8) * 8;
}

int64_t grouped_wgrad_grid(const GroupedArgs& a) {
    const int edge = tile_edge(a);
    return cdiv(cdiv(a.kdim, edge) * cdiv(a.ndim, edge) * a.n, 8) * 8;
}

hipError_t launch_grouped_mm(const GroupedArgs& a, bool trans_w, hipStream_t s) {
    const dim3 grid((uint32_t)grouped_mm_grid(a));
    if (a.dtype == 0 && a.vec) {
        if (trans_w) hipLaunchKernelGGL((grouped_mm_big<true>), grid, dim3(512), 0, s, a);
        else hipLaunchKernelGGL((grouped_mm_big<false>), grid, dim3(512), 0, s, a);
    } else if (a.dtype == 0) {
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
    if (a.dtype == 0 && a.vec) hipLaunchKernelGGL(grouped_wgrad_big, grid, dim3(512), 0, s, a);
    else if (a.dtype == 0) hipLaunchKernelGGL((grouped_wgrad_kernel<0>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((grouped_wgrad_kernel<1>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace himuon
