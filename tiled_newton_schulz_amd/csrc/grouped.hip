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
#include <type_traits>

#include "device_util.h"
#include "grouped.h"

namespace himuon {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

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
        cnt[k] = hi > lo ? (hi - lo - 1) / BM + 1 : 0;
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

// ---------------------------------------------------------------------------
// Any operand (fp32; bf16 rows and widths that are not whole 16-byte chunks):
// tiles of 128 x 128 (four waves of 64 x 64 each) or, where those would leave
// CUs idle, 64 x 64, k in steps of 64 (bf16) or 32 (fp32).  The next step's
// chunks are loaded into registers while the present one is multiplied from
// LDS, then stored in the other LDS buffer.  Loads and stores are 16 bytes wide
// at any alignment of the element.  A chunk that reaches past its row's end is
// loaded from as much further left and shifted (element by element, a load's
// latency each, the 39 columns of a 4528 x 925 x 39 gradient took 155 instead of
// 35 us, and 8 x 2048 x 2047 x 2045 386 instead of 258 us).  An operand stays in
// LDS in its own order, as below for the larger tiles; fp32 products take four k
// at a time (lane group g holds k = 4 g .. 4 g + 3 of eight, for both operands
// alike).
// Where even the 64 x 64 tiles are fewer than the CUs, four parts of the
// workgroup (SPLIT) take every fourth step each, and their sums are added in
// order at the end.
// ---------------------------------------------------------------------------
template <int DT> struct Io;
template <> struct Io<0> {
    using T = unsigned short;
    static constexpr int EPC = 8, BK = 64, KLD = 64, IPAD = 0;   // LDS row stride along k, padding along i
    __device__ static T cv(float f) { return f2bf(f); }
};
template <> struct Io<1> {
    using T = float;
    static constexpr int EPC = 4, BK = 32, KLD = 36, IPAD = 4;
    __device__ static T cv(float f) { return f; }
};
struct __attribute__((packed, aligned(2))) Loose16 { u32x4 v; };   // 16 bytes at an element's alignment

// One operand of a tile: `side` rows (or columns) of the tile by kd.
template <int DT, bool ALONG_K, int EDGE>
struct Staged {
    using T = typename Io<DT>::T;
    static constexpr int EPC = Io<DT>::EPC, BK = Io<DT>::BK;
    static constexpr int CPR = (ALONG_K ? BK : EDGE) / EPC;   // chunks of an LDS row
    static constexpr int ROWS = 256 / CPR;                    // LDS rows 256 threads fill at a time
    static constexpr int NCH = EDGE * BK / EPC / 256;         // chunks of a thread
    static constexpr int LD = ALONG_K ? Io<DT>::KLD : EDGE + Io<DT>::IPAD;
    static constexpr int SIZE = (ALONG_K ? EDGE : BK) * LD;   // elements of a buffer
    static_assert(ROWS * NCH == (ALONG_K ? EDGE : BK), "the chunks cover the panel");
    const T* p;
    int64_t ld;
    int side, kd;
    int before;   // elements of a row before p (along k: 0)

    // thread of its part of the workgroup
    __device__ __forceinline__ static int tid() { return threadIdx.x & 255; }
    // bf16 along i: place of chunk c of k row k is c ^ swap(k), so that the four
    // rows and 32 columns that are read together lie on different banks
    __device__ __forceinline__ static int swap(int k) { return EDGE == 128 ? 4 * (k & 3) : 2 * (k & 2); }
    // chunk j of this thread at k0: row and first column of the stored matrix
    // (a row of k elements, or a k row)
    __device__ __forceinline__ void load(int k0, u32x4 (&r)[NCH]) const {
        const int row0 = tid() / CPR, c = (tid() % CPR) * EPC;
        const int rows = ALONG_K ? side : kd - k0, cols = ALONG_K ? kd - k0 : side;
        const T* q = p + (ALONG_K ? (int64_t)k0 : k0 * ld) + c;
        // elements of the chunk past the row's end: it is loaded from as many
        // before its place where the row has them, see put()
        const int out = max(c + EPC - cols, 0);
        const bool wide = out < EPC && (ALONG_K ? k0 : before) + c >= out;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int row = row0 + j * ROWS;
            const T* at = q + row * ld;
            if (row < rows && wide) {
                r[j] = reinterpret_cast<const Loose16*>(at - out)->v;
                continue;
            }
            uint64_t w[2] = {0, 0};
            if (row < rows)
#pragma unroll 1
                for (int e = 0; e < cols - c; ++e) {   // a matrix narrower than a chunk
                    const uint64_t x = DT == 0 ? (uint64_t)reinterpret_cast<const unsigned short*>(at)[e]
                                               : (uint64_t)reinterpret_cast<const unsigned*>(at)[e];
                    const uint64_t y = x << (sizeof(T) * 8 * (e % (EPC / 2)));
                    if (e < EPC / 2) w[0] |= y;
                    else w[1] |= y;
                }
            r[j] = u32x4{(unsigned)w[0], (unsigned)(w[0] >> 32), (unsigned)w[1], (unsigned)(w[1] >> 32)};
        }
    }
    // stores the chunks that load(k0, r) has loaded
    __device__ __forceinline__ void put(int k0, T* s, u32x4 (&r)[NCH]) const {
        const int col = (tid() % CPR) * EPC, out = max(col + EPC - (ALONG_K ? kd - k0 : side), 0);
        if (out > 0 && out < EPC && (ALONG_K ? k0 : before) + col >= out) {
            const int by = out * (int)sizeof(T) * 8;   // 16 .. 112 bits
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
                const uint64_t lo = r[j][0] | (uint64_t)r[j][1] << 32, hi = r[j][2] | (uint64_t)r[j][3] << 32;
                const uint64_t a = by < 64 ? lo >> by | hi << (64 - by) : hi >> (by - 64), b = by < 64 ? hi >> by : 0;
                r[j] = u32x4{(unsigned)a, (unsigned)(a >> 32), (unsigned)b, (unsigned)(b >> 32)};
            }
        }
        const int row0 = tid() / CPR, ch = tid() % CPR;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            const int row = row0 + j * ROWS;
            int place = ch;
            if (DT == 0) place ^= ALONG_K ? (row >> 1) & 7 : swap(row);
            *reinterpret_cast<u32x4*>(&s[row * LD + place * EPC]) = r[j];
        }
    }
    // operand of the 32-wide block `first`: bf16 16 k from kk * 16, fp32 8 k from kk * 8
    __device__ __forceinline__ static u32x4 frag(const T* s, int first, int kk) {
        const int lane = threadIdx.x & 63, l32 = lane & 31, gl = lane >> 5;
        if constexpr (DT == 0 && ALONG_K) {
            const int r = first + l32;
            return *reinterpret_cast<const u32x4*>(&s[r * LD + (((kk * 2 + gl) ^ ((r >> 1) & 7)) * 8)]);
        } else if constexpr (DT == 0) {
            const int i16 = lane & 15, k = kk * 16 + 8 * gl + (i16 >> 2);
            const int col = first + 16 * ((lane >> 4) & 1) + 4 * (i16 & 3);
            const T* q = &s[k * LD + (((col >> 3) ^ swap(k)) * 8) + (col & 7)];
            const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LDS_AS bf16x4*)(q));
            const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LDS_AS bf16x4*)(q + 4 * LD));
            return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else if constexpr (ALONG_K) {
            return *reinterpret_cast<const u32x4*>(&s[(first + l32) * LD + kk * 8 + gl * 4]);
        } else {
            u32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __float_as_uint(s[(kk * 8 + gl * 4 + e) * LD + first + l32]);
            return v;
        }
    }
};

// Stores a wave's part of a tile: block (i, j) of rows and columns 32 i, 32 j
// from (r0, c0).  A lane holds runs of four columns of a row; through the wave's
// own 32 x 32 elements of LDS (chunk c of row r at c ^ (r / 2 & 3), fp32 c ^ (r &
// 7)) neighbouring lanes store whole rows of a block.  (Stored from registers in
// runs of four, the 0.13 GB of gradients of 4 rows over 15 experts of 1340 x 3339
// took 59 instead of 37 us.)
template <int DT, int F>
__device__ __forceinline__ void put_blocks(const f32x16 (&acc)[F][F], typename Io<DT>::T* scratch,
                                           typename Io<DT>::T* C, int64_t ldc, int rows, int cols, int r0, int c0) {
    using T = typename Io<DT>::T;
    constexpr int EPC = Io<DT>::EPC, CPR = 32 / EPC, RPP = 64 / CPR;   // chunks of a row, rows stored at a time
    const int lane = threadIdx.x & 63, l32 = lane & 31, gl = lane >> 5;
    auto at = [&](int r, int c) { return scratch + r * 32 + (c ^ ((DT == 0 ? r >> 1 : r) & (CPR - 1))) * EPC; };
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) {
            const int br = r0 + i * 32, bc = c0 + j * 32;
            if (br >= rows || bc >= cols) continue;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const auto& v = acc[i][j];
                if constexpr (DT == 0)
                    *reinterpret_cast<u32x2*>(at(l32, m) + 4 * gl) =
                        u32x2{pack2(v[4 * m], v[4 * m + 1]), pack2(v[4 * m + 2], v[4 * m + 3])};
                else
                    *reinterpret_cast<f32x4*>(at(l32, 2 * m + gl)) =
                        f32x4{v[4 * m], v[4 * m + 1], v[4 * m + 2], v[4 * m + 3]};
            }
#pragma unroll
            for (int p = 0; p < 32 / RPP; ++p) {
                const int r = p * RPP + lane / CPR, c = lane % CPR, col = bc + c * EPC;
                if (br + r >= rows || col >= cols) continue;
                const u32x4 v = *reinterpret_cast<const u32x4*>(at(r, c));
                T* to = C + (br + r) * ldc + col;
                if (col + EPC <= cols) {
                    *reinterpret_cast<Loose16*>(to) = Loose16{v};
                } else {
#pragma unroll
                    for (int e = 0; e < EPC - 1; ++e)
                        if (col + e < cols) {
                            if constexpr (DT == 0) to[e] = (unsigned short)(v[e >> 1] >> (16 * (e & 1)));
                            else to[e] = __uint_as_float(v[e]);
                        }
                }
            }
        }
}

// A B of one tile (operands exchanged in the MFMA, so that a lane holds runs of
// four columns of one row): done(sums, wave, its scratch) in each wave that ends
// with some.
template <int DT, bool AK, bool BKK, int EDGE, int SPLIT, typename Done>
__device__ __forceinline__ void staged_tile(const Staged<DT, AK, EDGE>& A, const Staged<DT, BKK, EDGE>& B, Done done) {
    using T = typename Io<DT>::T;
    constexpr int WE = EDGE / 2, F = WE / 32;   // edge of a wave's part, in 32-wide blocks
    constexpr int BK = Io<DT>::BK, SUB = DT == 0 ? 16 : 8;
    constexpr int SA = Staged<DT, AK, EDGE>::SIZE, SB = Staged<DT, BKK, EDGE>::SIZE;
    __shared__ __attribute__((aligned(16))) T buf_a[SPLIT][2][SA], buf_b[SPLIT][2][SB];
    const int lane = threadIdx.x & 63, id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wave = id & 3, part = SPLIT > 1 ? id >> 2 : 0;
    const int wm = wave >> 1, wn = wave & 1;
    T (&sa)[2][SA] = buf_a[part];
    T (&sb)[2][SB] = buf_b[part];
    const bool work = wm * WE < A.side && wn * WE < B.side;
    f32x16 acc[F][F];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) acc[i][j] = f32x16{};
    if (A.kd > 0) {
        u32x4 ra[Staged<DT, AK, EDGE>::NCH], rb[Staged<DT, BKK, EDGE>::NCH];
        A.load(part * BK, ra);   // past kd: zeros
        B.load(part * BK, rb);
        A.put(part * BK, sa[0], ra);
        B.put(part * BK, sb[0], rb);
        __syncthreads();
        for (int k0 = 0, cur = 0; k0 < A.kd; k0 += SPLIT * BK, cur ^= 1) {   // the same number of steps in every part
            const int next = k0 + (SPLIT + part) * BK;
            const bool more = next < A.kd;
            if (more) {
                A.load(next, ra);
                B.load(next, rb);
            }
            if (work && k0 + part * BK < A.kd) {
#pragma unroll
                for (int kk = 0; kk < BK / SUB; ++kk) {
                    u32x4 av[F], bv[F];
#pragma unroll
                    for (int i = 0; i < F; ++i) av[i] = Staged<DT, AK, EDGE>::frag(sa[cur], wm * WE + i * 32, kk);
#pragma unroll
                    for (int j = 0; j < F; ++j) bv[j] = Staged<DT, BKK, EDGE>::frag(sb[cur], wn * WE + j * 32, kk);
#pragma unroll
                    for (int i = 0; i < F; ++i)
#pragma unroll
                        for (int j = 0; j < F; ++j) {
                            if constexpr (DT == 0) {
                                acc[i][j] = mfma32w(bv[j], av[i], acc[i][j]);
                            } else {
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(
                                        __uint_as_float(bv[j][e]), __uint_as_float(av[i][e]), acc[i][j], 0, 0, 0);
                            }
                        }
                }
            }
            if (more) {
                A.put(next, sa[cur ^ 1], ra);
                B.put(next, sb[cur ^ 1], rb);
            }
            __syncthreads();
        }
    }
    if constexpr (SPLIT > 1) {
        static_assert(F == 1 && sizeof(buf_a) >= (SPLIT - 1) * 4 * 64 * 16 * sizeof(float), "the parts' sums fit");
        float* sums = reinterpret_cast<float*>(&buf_a[0][0][0]);   // no longer read (last barrier)
        if (part > 0)
#pragma unroll
            for (int e = 0; e < 16; ++e) sums[(((part - 1) * 4 + wave) * 16 + e) * 64 + lane] = acc[0][0][e];
        __syncthreads();
        if (part > 0) return;
#pragma unroll
        for (int o = 0; o < SPLIT - 1; ++o)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[0][0][e] += sums[((o * 4 + wave) * 16 + e) * 64 + lane];
    }
    // (buf_b is no longer read either)
    static_assert(sizeof(buf_b) >= 4 * 32 * 32 * sizeof(T), "the waves' scratch fits");
    done(acc, wave, &buf_b[0][0][0] + wave * (32 * 32));
}

template <int DT, bool WT, int EDGE, int SPLIT>
__global__ __launch_bounds__(256 * SPLIT) void grouped_mm_staged(const GroupedArgs a) {
    using T = typename Io<DT>::T;
    GroupTile t;
    if (!find_tile(a, EDGE, (a.ndim + EDGE - 1) / EDGE, t)) return;
    const int64_t m0 = (int64_t)t.row0 + t.mt * EDGE;
    const int n0 = t.nt * EDGE;
    Staged<DT, true, EDGE> A{reinterpret_cast<const T*>(a.x) + m0 * a.x_ld, a.x_ld,
                             min(EDGE, t.rows - t.mt * EDGE), a.kdim, 0};
    Staged<DT, WT, EDGE> B{nullptr, 0, min(EDGE, a.ndim - n0), a.kdim, n0};
    if (t.e < a.n) {
        B.ld = a.w_ld[t.e];
        B.p = reinterpret_cast<const T*>(a.w[t.e]) + (WT ? n0 * B.ld : n0);
    } else {
        A.kd = B.kd = 0;   // rows of no expert: zeros
    }
    staged_tile<DT, true, WT, EDGE, SPLIT>(A, B, [&](const auto& acc, int wave, T* scratch) __attribute__((always_inline)) {
        put_blocks<DT>(acc, scratch, reinterpret_cast<T*>(a.y) + m0 * a.y_ld + n0, a.y_ld, A.side, B.side,
                       (wave >> 1) * (EDGE / 2), (wave & 1) * (EDGE / 2));
    });
}

// PARTS: a workgroup takes one of the parts that an expert's rows are cut into,
// and leaves its sums for grouped_wgrad_join.
template <int DT, int EDGE, int SPLIT, bool PARTS>
__global__ __launch_bounds__(256 * SPLIT) void grouped_wgrad_staged(const GroupedArgs a) {
    using T = typename Io<DT>::T;
    constexpr int BK = Io<DT>::BK;
    const int ntk = (a.kdim + EDGE - 1) / EDGE, ntn = (a.ndim + EDGE - 1) / EDGE;
    const int tiles = a.n * ntk * ntn, total = PARTS ? tiles * a.parts : tiles, per = (total + 7) / 8;
    const int id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || id >= total) return;
    // the tiles of one part of an expert next to each other: they share its rows
    const int e = id / (PARTS ? ntk * ntn * a.parts : ntk * ntn), b = id % (ntk * ntn);
    const int i0 = (b % ntk) * EDGE, j0 = (b / ntk) * EDGE;
    int lo, hi;
    slot_rows(a, e, lo, hi);
    hi = max(lo, hi);
    const int part = id / (ntk * ntn) % (PARTS ? a.parts : 1);
    if (PARTS) {
        const int64_t steps = (hi - lo + BK - 1) / BK;   // the host leaves room for such roundings
        const int from = (int)(steps * part / a.parts) * BK, to = (int)(steps * (part + 1) / a.parts) * BK;
        hi = min(hi, lo + to);
        lo += from;
    }
    lo = __builtin_amdgcn_readfirstlane(lo);
    const int kd = __builtin_amdgcn_readfirstlane(hi - lo);
    const Staged<DT, false, EDGE> A{reinterpret_cast<const T*>(a.x) + lo * a.x_ld + i0, a.x_ld,
                                    min(EDGE, a.kdim - i0), kd, i0};
    const Staged<DT, false, EDGE> B{reinterpret_cast<const T*>(a.d) + lo * a.d_ld + j0, a.d_ld,
                                    min(EDGE, a.ndim - j0), kd, j0};
    staged_tile<DT, false, false, EDGE, SPLIT>(A, B, [&](const auto& acc, int wave, T* scratch) __attribute__((always_inline)) {
        if constexpr (PARTS) {
            f32x4* to = reinterpret_cast<f32x4*>(a.sums + ((int64_t)part * tiles + e * ntk * ntn + b) * (EDGE * EDGE)) +
                        wave * 256 + (threadIdx.x & 63);
#pragma unroll
            for (int m = 0; m < 4; ++m)
                to[m * 64] = f32x4{acc[0][0][4 * m], acc[0][0][4 * m + 1], acc[0][0][4 * m + 2], acc[0][0][4 * m + 3]};
        } else {
            put_blocks<DT>(acc, scratch, reinterpret_cast<T*>(a.w[e]) + i0 * a.w_ld[e] + j0, a.w_ld[e], A.side,
                           B.side, (wave >> 1) * (EDGE / 2), (wave & 1) * (EDGE / 2));
        }
    });
}

// Adds the parts' sums of one 64 x 64 tile, in order.
template <int DT>
__global__ __launch_bounds__(256) void grouped_wgrad_join(const GroupedArgs a) {
    using T = typename Io<DT>::T;
    const int ntk = (a.kdim + 63) / 64, ntn = (a.ndim + 63) / 64, tiles = a.n * ntk * ntn;
    const int id = blockIdx.x, e = id / (ntk * ntn), b = id % (ntk * ntn);
    const int i0 = (b % ntk) * 64, j0 = (b / ntk) * 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const f32x4* from = reinterpret_cast<const f32x4*>(a.sums + (int64_t)id * 4096) + wave * 256 + lane;
    f32x16 acc[1][1] = {};
#pragma unroll 4
    for (int p = 0; p < a.parts; ++p, from += (int64_t)tiles * 1024)
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const f32x4 v = from[m * 64];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[0][0][4 * m + i] += v[i];
        }
    __shared__ __attribute__((aligned(16))) T scratch[4][32 * 32];
    put_blocks<DT>(acc, scratch[wave], reinterpret_cast<T*>(a.w[e]) + i0 * a.w_ld[e] + j0, a.w_ld[e],
                   min(64, a.kdim - i0), min(64, a.ndim - j0), (wave >> 1) * 32, (wave & 1) * 32);
}

// ---------------------------------------------------------------------------
// bf16 operands of 16-byte chunks: 256 x 256 tiles, k in steps of 64, eight
// waves (2 along the rows, 4 along the columns).
//
// LDS holds two steps of both operands (A0 A1 B0 B1, each half a panel: 128 rows
// or columns by 64), filled straight from global memory.  The 32 x 32 blocks of
// a wave interleave with the other waves' (rows (2 i + wm) 32, columns
// (4 j + wn) 32), so every wave reads every half.  A step is four slots of a
// wave, with a barrier after each:
//     read     A0, B0, B1 into registers
//     multiply A0 B0, A0 B1 (16 MFMAs)
//     read     A1 into the registers of A0
//     multiply A1 B0, A1 B1
// Waves 4 - 7 run one slot behind waves 0 - 3, so that of the two waves on a
// SIMD one always multiplies while the other reads, stores a finished tile or
// starts the next one.  (With all waves in step, the reads between the products
// as in a usual pipeline, the matrix units idled a third of the time around the
// barriers.)  A half is free once both groups have read it; a wave loads its
// part of the successor in the next reading slot, a step before it has to be
// there.  (Loading between the products instead, one slot earlier, lost more in
// the multiplying group than it gained.)
// The loads run on into the next tile of the workgroup, and the result goes from
// registers to memory, so neither the pipeline's start nor a tile's end drains it.
//
// Ragged tiles: blocks of 64 rows or 128 columns outside the tile are not
// multiplied; their loads end past the buffer and give zeros.
//
// An operand is stored in memory either along k (rows i of k) or along its
// other side (rows k of i), and LDS keeps that order:
//   along k: 16-byte chunk c of row i at place c ^ ((i / 2) & 7)
//   along i: sub-panels of 128 elements; chunk c of row k at place
//            c ^ (4 (k & 3)); read transposed (ds_read_tr16_b64)
// Both leave the 16 lanes that read together on 64 different banks.
// The products run with the operands exchanged (columns as the MFMA's rows), so
// that a lane ends with runs of four consecutive columns of one row.
//
// Measured: 8 experts of 2048 x 4096 x 4096 420 us either way (1.3 PFLOP/s; a
// step takes 1.47 us, 82 % of the matrix rate at the clock the chip holds), their
// weight gradients 460 us.  64 experts with ragged shares, 4096 x 1408: products
// of 16384 rows 266 us, input gradients of 32768 rows 385 - 408 us, weight
// gradients 450 us (0.74 GB of results).
// ---------------------------------------------------------------------------
constexpr int kBig = 256;                  // tile edge
constexpr int kBK = 64;                    // k of a step
constexpr int kPanel = kBig * kBK;         // elements of one operand's step
constexpr uint32_t kNowhere = 0x80000000u; // byte offset past every buffer

typedef int i32x4 __attribute__((ext_vector_type(4)));

// A value that every lane holds, as a scalar.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ uint64_t uniform(uint64_t x) {
    return (uint32_t)uniform((int)(uint32_t)x) | (uint64_t)(uint32_t)uniform((int)(x >> 32)) << 32;
}

// The same for an operand of the assembly below: the compiler drops uniform()
// of a value it knows to be uniform, and may still keep it in a vector register.
__device__ __forceinline__ int scalar(int x) {
    int r;
    asm("v_readfirstlane_b32 %0, %1" : "=s"(r) : "v"(x));
    return r;
}

// Buffer descriptor of [p, p + bytes): loads past it give zeros, stores are dropped.
__device__ __forceinline__ i32x4 rsrc_words(const void* p, int64_t bytes) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    const int n = bytes < 0 ? 0 : bytes > 0x7fffff00 ? 0x7fffff00 : (int)bytes;
    return i32x4{(int)(uint32_t)u, (int)((uint32_t)(u >> 32) & 0xffffu), n, 0x00020000};
}
// 64 lanes x 16 bytes from r + off to LDS byte address lds + 16 lane.  As
// inline assembly, since the compiler makes every transposed LDS read wait for
// all such loads it knows of; the waits are in phase_gate().  It has no
// register result, so nothing can be read or reused too early.
__device__ __forceinline__ void dma16(i32x4 r, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :: "s"(lds), "v"(off), "s"(r) : "m0", "memory");
}
// Ends a reading slot: all but this wave's newest loads have landed and its LDS
// reads are done; then the same of all waves.  The half that the next reading
// slot needs was loaded one step before; four halves (8 loads of the wave) are
// newer, and near a tile's end so are the stores of its result (8 for each half
// of the rows, always issued; see put_result): MORE of them when `more` is set.
template <int MORE>
__device__ __forceinline__ void end_read(int more) {
    asm volatile("s_cmp_lg_u32 %0, 0\n\ts_cbranch_scc1 .Lmore%=\n\ts_waitcnt vmcnt(8)\n"
                 ".Lmore%=:\n\ts_waitcnt vmcnt(%1) lgkmcnt(0)\n\ts_barrier"
                 :: "s"(scalar(more)), "n"(8 + MORE) : "memory", "scc");
    __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0) again, for the compiler's own count
    __builtin_amdgcn_sched_barrier(0);
}
// Ends a multiplying slot: nothing to wait for but the other waves (waits and
// tests here, behind the products, cost a tenth of the kernel's time).
__device__ __forceinline__ void end_multiply() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// The loads of one operand, step by step.  An instruction of the workgroup
// fills 64 rows of 128 bytes (along k) or 32 rows of 256 bytes (along i); a half
// takes two.
template <bool ALONG_K>
struct Feed {
    uint64_t at;        // first byte of the step
    int64_t rest;       // bytes from there to the operand's end (the end of the last row that counts)
    int64_t move;       // bytes to the next step
    int left;           // k from the step on
    uint32_t v, first;  // this lane's byte offset in an instruction; first k element of its chunk
    uint32_t off[2][2]; // byte offset of instruction j of half h

    // p: element (0, 0) of the tile at k = 0; side: its rows (or columns) inside
    // the operand; kd: length of k (0: all zeros)
    __device__ __forceinline__ void start(uint64_t p, int64_t ld, int side, int kd, int wave, int lane) {
        const uint32_t ld2 = 2u * (uint32_t)ld;
        at = p;
        left = kd;
        if constexpr (ALONG_K) {
            const uint32_t c = (lane & 7) ^ (4 * (wave & 1) + (lane >> 4));
            rest = 2 * ((side - 1) * ld + kd);
            move = 2 * kBK;
            v = (uint32_t)(8 * wave + (lane >> 3)) * ld2 + c * 16u;
            first = c * 8;
        } else {
            rest = 2 * ((kd - 1) * ld + side);
            move = (int64_t)kBK * ld2;
            v = (uint32_t)(4 * wave + (lane >> 4)) * ld2 + (((lane & 15) ^ ((lane >> 4) * 4)) * 16u);
            first = 0;
        }
        // rows past the operand start past its end; columns are left out by half
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                off[h][j] = ALONG_K ? (h * 128 + j * 64) * ld2
                                    : h * 128 < side ? h * 256 + j * 32 * ld2 : kNowhere;
    }
    __device__ __forceinline__ void next() {
        at += move;
        rest -= move;
        left -= kBK;
    }
    // half h into LDS byte address lds (this wave's part)
    __device__ __forceinline__ void load(int h, uint32_t lds) const {
        const i32x4 r = rsrc_words(reinterpret_cast<const void*>(at), left > 0 ? rest : 0);
        // a last step that k does not fill: chunks along k past its end would
        // read the next row
        const uint32_t u = ALONG_K && (int)first >= left ? kNowhere : v;
#pragma unroll
        for (int j = 0; j < 2; ++j) dma16(r, u + off[h][j], lds + (h * 2 + j) * 8192);
    }
};

// LDS addresses of a wave's operand fragments.
template <bool ALONG_K>
struct Frag {
    // along k: one address for each k sub-step; along i: rows 0 - 63 and
    // 64 - 127 of a sub-panel (they differ in one bit of the swizzled chunk)
    uint32_t at[ALONG_K ? 4 : 2];
    // panel: LDS byte address; first: the wave's first row or column (along i:
    // below 64 where 64-wide blocks are read, else below 128)
    __device__ __forceinline__ Frag(uint32_t panel, int first, int lane) {
        if constexpr (ALONG_K) {
            const int r = first + (lane & 31);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                at[kk] = panel + r * 128 + (((kk * 2 + (lane >> 5)) ^ ((r >> 1) & 7)) * 16);
        } else {
            const int i16 = lane & 15, k = 8 * (lane >> 5) + (i16 >> 2);
            const int col = first + 16 * ((lane >> 4) & 1) + 4 * (i16 & 3);
            at[0] = panel + k * 256 + (((col >> 3) ^ ((k & 3) * 4)) * 16) + (col & 7) * 2;
            at[1] = at[0] ^ 128;
        }
    }
    // from the step of parity p to the other one of the two in LDS
    __device__ __forceinline__ void flip(int p) {
#pragma unroll
        for (uint32_t& x : at) x += p ? -(kPanel * 2) : kPanel * 2;
    }
    // MFMA operand of the 32-wide block `off` past `first`, k sub-step kk
    __device__ __forceinline__ bf16x8 read(int off, int kk) const {
        if constexpr (ALONG_K) {
            return *(const LDS_AS bf16x8*)(uintptr_t)(at[kk] + off * 128);
        } else {
            const uint32_t b = at[(off >> 6) & 1] + (off >> 7) * (kBK * 256) + kk * 16 * 256;
            const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LDS_AS bf16x4*)(uintptr_t)b);
            const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LDS_AS bf16x4*)(uintptr_t)(b + 4 * 256));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
};

// Half h of the result tile (rows 128 h ..): C[r][c] with r = (2 i + wm) 32 + l32
// and c = (4 j + wn) 32 + 8 m + 4 gl + e is acc[i][j][4 m + e] of lane
// 32 gl + l32.  Each 32 x 32 block goes through the wave's own LDS scratch, so
// that four neighbouring lanes store 64 bytes of a row: stored from registers
// in 16-byte pieces, the weight gradient's 0.8 GB of results cost 130 us more
// than no stores at all (64 experts of 512 x 4096 x 1536).
// All 8 stores are issued whatever the tile's size (those outside are dropped
// by the buffer's bounds): end_read counts them.
constexpr int kScratchLd = 40;                   // elements (80 bytes) a row
constexpr int kScratch = 32 * kScratchLd;        // elements of a wave
template <int AM, int FN>
__device__ __forceinline__ void put_result(const f32x16 (&acc)[AM][FN], int h, unsigned short* scratch, uint64_t C,
                                           int ldc, int rows, int cols, int wm, int wn, int lane) {
    const int l32 = lane & 31, gl = lane >> 5;
    const int r0 = wm * 32 + (lane >> 2), c0 = wn * 32 + (lane & 3) * 8;
    const uint32_t v0 = (uint32_t)r0 * (uint32_t)ldc * 2u + c0 * 2u, half = (uint32_t)ldc * 32u;
#pragma unroll
    for (int i = 2 * h; i < 2 * h + 2; ++i) {
        const int64_t at = (int64_t)i * 64 * ldc;
        const int64_t bytes = i * 64 < rows ? 2 * ((int64_t)(rows - 1) * ldc + cols - at) : 0;
        const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
            reinterpret_cast<void*>(C + 2 * at), (short)0, (int)min(bytes, (int64_t)0x7fffff00), 0x00020000);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (i >= AM || j >= FN) {
                // nothing there: two stores that are dropped (as assembly, so
                // that neither is removed)
                const i32x4 none = {0, 0, 0, 0x00020000};
                asm volatile("buffer_store_dword %0, %0, %1, 0 offen\n\tbuffer_store_dword %0, %0, %1, 0 offen"
                             :: "v"(kNowhere), "s"(none) : "memory");
                continue;
            }
            const auto& v = acc[i < AM ? i : 0][j < FN ? j : 0];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const u32x2 w = {pack2(v[4 * m], v[4 * m + 1]), pack2(v[4 * m + 2], v[4 * m + 3])};
                *reinterpret_cast<u32x2*>(&scratch[l32 * kScratchLd + m * 8 + gl * 4]) = w;
            }
            const uint32_t at_j = j * 128 + c0 < cols ? v0 + j * 256u : kNowhere;
#pragma unroll
            for (int s = 0; s < 2; ++s)
                __builtin_amdgcn_raw_buffer_store_b128(
                    *reinterpret_cast<const u32x4*>(&scratch[(s * 16 + (lane >> 2)) * kScratchLd + (lane & 3) * 8]), rb,
                    at_j + s * half, 0, 0);
        }
    }
}

// One output tile.
struct Job {
    uint64_t a, b, c;    // element (0, 0) of its operands (at k = 0) and result
    int w_ld;            // row stride of the expert's matrix
    int rows, cols;      // size of the tile
    int kd;              // length of k (0: the result is zero)
};
constexpr int kJobs = 128;   // tiles of a workgroup planned at a time

// The launch's slots (experts, and the rows of none).
struct GroupTable {
    int lo[kExperts + 1];      // first row
    int rows[kExperts + 1];
    int first[kExperts + 2];   // tiles before the slot
    float cost[kExperts + 2];  // cost of all tiles before the slot
};

// Tiles of the launch: an expert has a grid of row tiles (product: of its rows;
// weight gradient: of the K rows of G) by column tiles, counted column by column
// in bands of row tiles: the 32 workgroups of an XCD then work on about 8 x 4
// tiles at a time, which read the least through its L2 (2 experts of 8192 x 4096
// x 4096: 443 us without bands, 411 with; weight gradient of 64 experts of 512 x
// 4096 x 1408: 450 and 434).
constexpr int kBand = 8;
template <int MODE>
struct Grid {
    const GroupedArgs& a;
    int ntn;   // column tiles
    __device__ __forceinline__ explicit Grid(const GroupedArgs& x) : a(x), ntn((x.ndim - 1) / kBig + 1) {}
    __device__ __forceinline__ int row_tiles(int rows) const {
        const int h = MODE == 2 ? a.kdim : rows;
        return h > 0 ? (h - 1) / kBig + 1 : 0;
    }
    // Time of a slot's tiles, to share them out: a step of a tile takes about
    // 1.0 us and 0.12 us for each block of 64 rows, a tile about 4 us (measured
    // on the experts' products with ragged rows).
    __device__ __forceinline__ float cost(int rows) const {
        const int h = MODE == 2 ? a.kdim : rows, steps = ((MODE == 2 ? rows : a.kdim) + kBK - 1) / kBK;
        return ntn * (row_tiles(rows) * (steps * 1.0f + 4.0f) + (float)((h + 63) / 64) * steps * 0.12f);
    }
    __device__ __forceinline__ Job job(const GroupTable& t, int id) const {
        // the last slot whose first tile is at or before id
        int e = 0;
#pragma unroll
        for (int s = 128; s > 0; s >>= 1)
            if (e + s <= kExperts && t.first[e + s] <= id) e += s;
        const int R = row_tiles(t.rows[e]), off = id - t.first[e];
        // bands of eight row tiles, column by column
        const int band = off / (kBand * ntn), in = off - band * kBand * ntn, high = min(kBand, R - band * kBand);
        const int m = (band * kBand + in % high) * kBig, n0 = in / high * kBig;
        Job j;
        const unsigned short* x = reinterpret_cast<const unsigned short*>(a.x);
        j.cols = min(kBig, a.ndim - n0);
        if constexpr (MODE == 2) {
            j.a = reinterpret_cast<uint64_t>(x + t.lo[e] * a.x_ld + m);
            j.b = reinterpret_cast<uint64_t>(reinterpret_cast<const unsigned short*>(a.d) + t.lo[e] * a.d_ld + n0);
            j.w_ld = (int)a.w_ld[e];
            j.c = reinterpret_cast<uint64_t>(reinterpret_cast<unsigned short*>(a.w[e]) + m * a.w_ld[e] + n0);
            j.rows = min(kBig, a.kdim - m);
            j.kd = t.rows[e];
        } else {
            const int64_t m0 = (int64_t)t.lo[e] + m;
            j.a = reinterpret_cast<uint64_t>(x + m0 * a.x_ld);
            j.c = reinterpret_cast<uint64_t>(reinterpret_cast<unsigned short*>(a.y) + m0 * a.y_ld + n0);
            j.rows = min(kBig, t.rows[e] - m);
            j.b = 0;
            j.w_ld = 0;
            j.kd = 0;
            if (e < a.n) {   // else rows of no expert
                j.w_ld = (int)a.w_ld[e];
                j.kd = a.kdim;
                j.b = reinterpret_cast<uint64_t>(reinterpret_cast<const unsigned short*>(a.w[e]) +
                                                 (MODE == 1 ? n0 * a.w_ld[e] : n0));
            }
        }
        return j;
    }
};

// Fills the table (one wave).  `most`: the tiles the launch was made for (end
// rows that decrease could count more; those are cut off).
template <int MODE>
__device__ __forceinline__ void fill_table(const GroupedArgs& a, const Grid<MODE>& g, GroupTable& t, int most) {
    const int lane = threadIdx.x, slots = a.n + (MODE != 2 && a.last ? 1 : 0);
    float c[4], csum = 0.f;
    int n[4], nsum = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int i = lane * 4 + k;
        int lo = 0, hi = 0;
        if (i < slots) slot_rows(a, i, lo, hi);
        const int rows = max(hi - lo, 0);
        t.lo[i] = lo;
        t.rows[i] = rows;
        n[k] = i < slots ? g.row_tiles(rows) * g.ntn : 0;
        c[k] = i < slots ? g.cost(rows) : 0.f;
        nsum = min(nsum + n[k], most);
        csum += c[k];
    }
    int nincl = nsum;
    float cincl = csum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int nv = __shfl_up(nincl, o, 64);
        const float cv = __shfl_up(cincl, o, 64);
        if (lane >= o) {
            nincl = min(nincl + nv, most);
            cincl += cv;
        }
    }
    int nat = __shfl_up(nincl, 1, 64);
    float cat = __shfl_up(cincl, 1, 64);
    if (lane == 0) {
        nat = 0;
        cat = 0.f;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        t.first[lane * 4 + k] = nat;
        t.cost[lane * 4 + k] = cat;
        nat = min(nat + n[k], most);
        cat += c[k];
    }
    if (lane == 63) {
        t.first[256] = nat;
        t.cost[256] = cat;
    }
}

// First tile of share x of eight, of about equal cost.
__device__ __forceinline__ int share(const GroupTable& t, int x) {
    if (x == 8) return t.first[256];
    const float at = t.cost[256] * ((float)x / 8.f);
    int e = 0;
#pragma unroll
    for (int s = 128; s > 0; s >>= 1)
        if (e + s <= kExperts && t.cost[e + s] <= at) e += s;
    const float c = t.cost[e + 1] - t.cost[e];
    const int n = t.first[e + 1] - t.first[e];
    return t.first[e] + (c > 0.f ? max(0, min(n, (int)((at - t.cost[e]) / c * n))) : 0);
}

template <int MODE>
__global__ __launch_bounds__(512) void grouped_big(const GroupedArgs a, const int most) {
    constexpr bool AK = MODE != 2, BKK = MODE == 1;   // operands stored along k
    __shared__ __attribute__((aligned(1024))) unsigned short sbuf[4 * kPanel];
    __shared__ __attribute__((aligned(16))) unsigned short scratch[8 * kScratch];
    __shared__ __attribute__((aligned(16))) Job jobs[kJobs];
    __shared__ GroupTable table;
    const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
    const int wm = wave >> 2, wn = wave & 3;

    // ---- this workgroup's tiles.  Each XCD (workgroup ids go round the eight)
    //      takes a run of tiles, so that what they share sits in one L2, and
    //      deals them out to its workgroups in turn
    const Grid<MODE> grid(a);
    if (wave == 0) fill_table<MODE>(a, grid, table, most);
    __syncthreads();
    const int stride = gridDim.x >> 3;
    const int end = uniform(share(table, (blockIdx.x & 7) + 1));
    int id = uniform(share(table, blockIdx.x & 7)) + (blockIdx.x >> 3);

  for (; id < end; id += kJobs * stride) {   // kJobs of them at a time (nearly always all)
    const int count = min((end - id + stride - 1) / stride, kJobs);
    for (int m = threadIdx.x; m < count; m += 512) jobs[m] = grid.job(table, id + m * stride);
    __syncthreads();

    const uint32_t lds = (uint32_t)(uintptr_t)(LDS_AS void*)sbuf;
    const uint32_t ldsA = lds + wave * 1024, ldsB = ldsA + 4 * kPanel;
    Frag<AK> fa(lds, wm * 32, lane);
    Frag<BKK> fb(lds + 4 * kPanel, wn * 32, lane);

    // ---- loads, ahead of the products: tile `in` ----
    Feed<AK> feed_a;
    Feed<BKK> feed_b;
    int in = 0;
    auto start_feed = [&]() __attribute__((always_inline)) {
        const Job j = jobs[min(in, count - 1)];
        const int kd = in < count ? uniform(j.kd) : 0;   // past the last tile: zeros
        const int64_t w_ld = uniform(j.w_ld);
        feed_a.start(uniform(j.a), a.x_ld, uniform(j.rows), kd, wave, lane);
        feed_b.start(uniform(j.b), MODE == 2 ? a.d_ld : w_ld, uniform(j.cols), kd, wave, lane);
    };
    auto advance = [&]() __attribute__((always_inline)) {
        feed_a.next();
        feed_b.next();
        if (feed_a.left > 0) return;
        ++in;
        start_feed();
    };

    // ---- products: tile `out` ----
    int out = 0, rows, cols, kd, ldc;
    uint64_t C;
    auto start_tile = [&]() __attribute__((always_inline)) {
        const Job j = jobs[out];
        rows = uniform(j.rows);
        cols = uniform(j.cols);
        kd = uniform(j.kd);
        ldc = MODE == 2 ? uniform(j.w_ld) : (int)a.y_ld;
        C = uniform(j.c);
    };
    // loads: A1 of the feeds' step, and A0, B0, B1 of the step after it (q: its
    // parity)
    int q = 0;
    auto load_a1 = [&]() __attribute__((always_inline)) { feed_a.load(1, ldsA + q * (2 * kPanel)); };
    auto load_rest = [&]() __attribute__((always_inline)) {
        advance();
        q ^= 1;
        feed_a.load(0, ldsA + q * (2 * kPanel));
        feed_b.load(0, ldsB + q * (2 * kPanel));
        feed_b.load(1, ldsB + q * (2 * kPanel));
    };
    int after = 0;   // the tile's first step comes after another tile's
    int p = 0;       // parity of the step
    // the steps of one tile of AM blocks of 64 rows and FN of 128 columns
    auto run = [&](auto am, auto fn) __attribute__((always_inline)) {
        constexpr int AM = decltype(am)::value, FN = decltype(fn)::value;
        f32x16 acc[AM][FN];
#pragma unroll
        for (int i = 0; i < AM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = f32x16{};
        bf16x8 av[2][4], bv[2][4];
        auto read_a = [&](int h) __attribute__((always_inline)) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                for (int i = 0; i < 2; ++i) av[i][kk] = fa.read((h * 2 + i) * 64, kk);
        };
        auto read_b = [&](int j) __attribute__((always_inline)) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) bv[j][kk] = fb.read(j * 128, kk);
        };
        auto multiply = [&](int h) __attribute__((always_inline)) {
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (2 * h + i < AM) {
                            f32x16& c = acc[2 * h + i < AM ? 2 * h + i : 0][j];
                            c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bv[j][kk], av[i][kk], c, 0, 0, 0);
                        }
            __builtin_amdgcn_s_setprio(0);
        };
        for (int k = 0;; ++k) {
            const int last = (k + 1) * kBK >= kd;
            read_a(0);
            read_b(0);
            if (FN > 1) read_b(1);
            load_a1();
            end_read<16>(after);
            multiply(0);
            end_multiply();
            if (AM > 2) read_a(1);
            if (last) put_result(acc, 0, scratch + wave * kScratch, C, ldc, rows, cols, wm, wn, lane);
            load_rest();
            fa.flip(p);
            fb.flip(p);
            end_read<8>(after | last);
            if (AM > 2) multiply(1);
            end_multiply();
            p ^= 1;
            after = 0;
            if (last) break;
        }
        put_result(acc, 1, scratch + wave * kScratch, C, ldc, rows, cols, wm, wn, lane);
    };

    // the first step, and the second but for A1
    start_feed();
    feed_a.load(0, ldsA);
    feed_b.load(0, ldsB);
    feed_b.load(1, ldsB);
    load_a1();
    load_rest();
    start_tile();
    asm volatile("s_waitcnt vmcnt(8)\n\ts_barrier" ::: "memory");
    if (wm == 1) end_multiply();   // one slot behind

    for (;;) {
        const int am = (rows + 63) >> 6;
        constexpr std::integral_constant<int, 1> c1{};
        constexpr std::integral_constant<int, 2> c2{};
        constexpr std::integral_constant<int, 3> c3{};
        constexpr std::integral_constant<int, 4> c4{};
        if (cols > 128) {
            if (am == 4) run(c4, c2);
            else if (am == 3) run(c3, c2);
            else if (am == 2) run(c2, c2);
            else run(c1, c2);
        } else {
            if (am == 4) run(c4, c1);
            else if (am == 3) run(c3, c1);
            else if (am == 2) run(c2, c1);
            else run(c1, c1);
        }
        if (++out == count) break;
        start_tile();
        after = 1;
    }
    if (wm == 0) end_multiply();   // as many barriers as the others
    // the loads past the last tile still write (zeros) into this workgroup's LDS
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Few rows an expert (tokens being decoded; bf16, 16-byte chunks): a stream of
// the weights, HBM bound.  Tiles of 16 rows by 64 columns; the four waves of a
// workgroup take a quarter of k each, with no barrier until their sums are
// joined.  A wave keeps a ring of kRing stages of 32 k in LDS (16 rows of X and 64
// columns of W, 5 KB), loaded straight from global memory: two workgroups hold
// 120 KB a CU in flight, which covers the memory's latency.  In a larger tile
// the same weights would wait for a pipeline's start and end at every tile.
// 96 rows over 64 experts of 4096 x 1408: 107 us, 5.7 TB/s.
//   along k: rows of four 16-byte chunks, chunk c of row r at c ^ ((r / 4) & 3)
//   along i: 32 k rows of eight chunks, chunk c of row k at c ^ (2 (k & 2))
// ---------------------------------------------------------------------------
constexpr int kThinRows = 16, kThinCols = 64, kRing = 4, kThinK = 32;
constexpr int kThinStage = (kThinRows + kThinCols) * kThinK;   // elements

template <bool WT>
__global__ __launch_bounds__(256) void grouped_mm_thin(const GroupedArgs a) {
    __shared__ __attribute__((aligned(1024))) unsigned short ring[4 * kRing * kThinStage];
    constexpr int kSumLd = kThinCols + 4;
    static_assert(4 * kThinRows * kSumLd * 4 <= (int)sizeof(ring), "the sums are joined in the ring's memory");
    GroupTile t;
    if (!find_tile(a, kThinRows, (a.ndim + kThinCols - 1) / kThinCols, t)) return;
    const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
    const int64_t m0 = (int64_t)t.row0 + t.mt * kThinRows;
    const int n0 = t.nt * kThinCols;
    const int rows = min(kThinRows, t.rows - t.mt * kThinRows), cols = min(kThinCols, a.ndim - n0);
    // this wave's k
    const int kw = (a.kdim + 4 * kThinK - 1) / (4 * kThinK) * kThinK;
    const int kb = min(a.kdim, wave * kw);
    int left = t.e < a.n ? min(kw, a.kdim - kb) : 0;   // none: rows of no expert
    const int64_t ldw = t.e < a.n ? a.w_ld[t.e] : 0;

    // ---- loads ----
    const uint32_t ldx2 = 2u * (uint32_t)a.x_ld, ldw2 = 2u * (uint32_t)ldw;
    const int r4 = lane >> 2, c4 = (lane & 3) ^ ((r4 >> 2) & 3);   // along k
    const int k8 = lane >> 3, c8 = (lane & 7) ^ (2 * (k8 & 2));    // along i
    uint64_t px = reinterpret_cast<uint64_t>(a.x) + 2 * (m0 * a.x_ld + kb), pw = 0;
    int64_t rest_x = 2 * ((int64_t)(rows - 1) * a.x_ld + left), rest_w = 0;
    if (t.e < a.n) {
        pw = reinterpret_cast<uint64_t>(a.w[t.e]) + 2 * (WT ? n0 * ldw + kb : kb * ldw + n0);
        rest_w = WT ? 2 * ((int64_t)(cols - 1) * ldw + left) : 2 * ((int64_t)(left - 1) * ldw + cols);
    }
    const uint32_t vx = r4 * ldx2 + c4 * 16u;
    const uint32_t vw = WT ? r4 * ldw2 + c4 * 16u : c8 * 8 < cols ? k8 * ldw2 + c8 * 16u : kNowhere;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(LDS_AS void*)ring + wave * (kRing * kThinStage * 2);
    auto load = [&](int slot) __attribute__((always_inline)) {
        const uint32_t lds = lds0 + slot * (kThinStage * 2);
        const i32x4 rx = rsrc_words(reinterpret_cast<const void*>(px), left > 0 ? rest_x : 0);
        const i32x4 rw = rsrc_words(reinterpret_cast<const void*>(pw), left > 0 ? rest_w : 0);
        const bool past = c4 * 8 >= left;   // chunks along k past the wave's end
        dma16(rx, past ? kNowhere : vx, lds);
        const uint32_t v = WT && past ? kNowhere : vw;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            dma16(rw, v == kNowhere ? v : v + j * (WT ? 16 : 8) * ldw2, lds + (kThinRows * kThinK * 2) + j * 1024);
        px += 2 * kThinK;
        rest_x -= 2 * kThinK;
        const int64_t move = WT ? 2 * kThinK : (int64_t)kThinK * ldw2;
        pw += move;
        rest_w -= move;
        left -= kThinK;
    };

    // ---- products: columns as the MFMA's rows ----
    f32x4 acc[4] = {};
    const int steps = (left + kThinK - 1) / kThinK;
    const int i16 = lane & 15, g = lane >> 4;
    const int at_x = i16 * kThinK + ((g ^ ((i16 >> 2) & 3)) * 8);
    const int kr = 8 * g + (i16 >> 2), sw = 2 * (kr & 2);
#pragma unroll
    for (int s = 0; s < kRing; ++s) load(s);
    for (int s = 0, slot = 0; s < steps; ++s, slot = (slot + 1) % kRing) {
        // all but the newest three stages have landed
        asm volatile("s_waitcnt vmcnt(15)" ::: "memory");
        const unsigned short* st = ring + (wave * kRing + slot) * kThinStage;
        const unsigned short* sw_ = st + kThinRows * kThinK;
        const bf16x8 xv = *reinterpret_cast<const bf16x8*>(&st[at_x]);
        bf16x8 wv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (WT) {
                wv[j] = *reinterpret_cast<const bf16x8*>(&sw_[j * 16 * kThinK + at_x]);
            } else {
                const unsigned short* q = &sw_[kr * kThinCols + (((j * 2 + ((i16 & 3) >> 1)) ^ sw) * 8) + 4 * (i16 & 1)];
                const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LDS_AS bf16x4*)(q));
                const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LDS_AS bf16x4*)(q + 4 * kThinCols));
                wv[j] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            }
        }
        // in registers: the stage can be filled again
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0xc07f);   // (the same, for the compiler's own count)
        load(slot);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[j], xv, acc[j], 0, 0, 0);
    }
    static_assert(kRing == 4, "the wait above counts five loads for each of three stages");

    // ---- the four waves' sums, in order ----
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    float* sums = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<f32x4*>(&sums[(wave * kThinRows + i16) * kSumLd + j * 16 + g * 4]) = acc[j];
    __syncthreads();
    const int r = threadIdx.x >> 4, c = (threadIdx.x & 15) * 4;
    f32x4 v = *reinterpret_cast<const f32x4*>(&sums[r * kSumLd + c]);
#pragma unroll
    for (int w = 1; w < 4; ++w) v += *reinterpret_cast<const f32x4*>(&sums[(w * kThinRows + r) * kSumLd + c]);
    if (r < rows && c < cols) {
        const u32x2 o = {pack2(v[0], v[1]), pack2(v[2], v[3])};
        *reinterpret_cast<u32x2*>(reinterpret_cast<unsigned short*>(a.y) + (m0 + r) * a.y_ld + n0 + c) = o;
    }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

int device_cus_or_256() {
    static const int cus = [] { const int c = device_cus(); return c >= 8 ? std::min(c, 512) : 256; }();
    return cus;
}

int64_t mm_tiles(const GroupedArgs& a, int edge) {
    // every slot ends in at most one partial row tile
    return (a.rows / edge + a.n + 1) * cdiv(a.ndim, edge);
}
int64_t wgrad_tiles(const GroupedArgs& a, int edge) { return cdiv(a.kdim, edge) * cdiv(a.ndim, edge) * a.n; }

// Tiles to expect: the host knows the rows and the experts, not which expert has
// how many; half a partial row tile each.  Of the whole call: where it takes more
// than one launch they all run the same kernel.  (The last launch of 256 experts
// holds one: planned by its share of the rows, calls of 1024 x 512 took 60 instead
// of 72 us at 32 rows an expert, but 148 instead of 132 us at 256, as its grid has
// to hold all rows and nearly all of it is empty.)
double mm_expect(const GroupedArgs& a, int edge) {
    return ((double)a.rows / edge + 0.5 * a.total) * (double)cdiv(a.ndim, edge);
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
enum class Kernel { Thin, Big, Staged128, Staged64, Split64 };
bool enough_big(double tiles) { return tiles >= 0.75 * device_cus_or_256(); }
// Four parts of a workgroup share a tile's steps; one such workgroup fits a CU.
// In us without and with: weight gradients 2 x 4528 x 925 x 39 35 and 22, 1 x
// 1024 x 512 x 512 11.9 and 9.4, 16 x 8192 x 256 x 256 (8 steps) 9.3 and 8.8;
// products (rows of all experts) 4 x 300 x 4095 x 500 55 and 30, in fp32 129
// and 93, with K = 512 in fp32 19.6 and 17.4.
bool split(const GroupedArgs& a, double tiles, int64_t k) {
    return tiles <= device_cus_or_256() && k >= 8 * (a.dtype == 0 ? Io<0>::BK : Io<1>::BK);
}
Kernel mm_kernel(const GroupedArgs& a) {
    if (a.dtype == 0 && a.vec) {
        const bool big = enough_big(mm_expect(a, kBig));
        if (a.rows <= (big ? 16 : 32) * (int64_t)a.total) return Kernel::Thin;
        if (big) return Kernel::Big;
    }
    if (mm_expect(a, 128) >= device_cus_or_256()) return Kernel::Staged128;
    return split(a, mm_expect(a, 64), a.kdim) ? Kernel::Split64 : Kernel::Staged64;
}
Kernel wgrad_kernel(const GroupedArgs& a) {
    if (a.dtype == 0 && a.vec && enough_big((double)wgrad_tiles(a, kBig))) return Kernel::Big;
    if (wgrad_tiles(a, 128) >= device_cus_or_256()) return Kernel::Staged128;
    return split(a, (double)wgrad_tiles(a, 64), a.rows / a.total) ? Kernel::Split64 : Kernel::Staged64;
}
int edge_of(Kernel k) { return k == Kernel::Big ? kBig : k == Kernel::Staged128 ? 128 : 64; }

// Most tiles of a launch, whole rounds of the XCDs.
int64_t grouped_mm_grid(const GroupedArgs& a) {
    const Kernel k = mm_kernel(a);
    if (k == Kernel::Thin) return cdiv((a.rows / kThinRows + a.n + 1) * cdiv(a.ndim, kThinCols), 8) * 8;
    return cdiv(mm_tiles(a, edge_of(k)), 8) * 8;
}
int64_t grouped_wgrad_grid(const GroupedArgs& a) { return cdiv(wgrad_tiles(a, edge_of(wgrad_kernel(a))), 8) * 8; }

// A workgroup a tile, and at most 2^32 - 1 threads a launch; the 256-tiles have
// workgroups of their own number and count tiles in an int.
bool fits(Kernel k, int64_t tiles) {
    if (k == Kernel::Big) return tiles <= INT32_MAX / 2;
    return tiles <= UINT32_MAX / (k == Kernel::Split64 ? 1024 : 256);
}

}  // namespace

bool grouped_mm_fits(const GroupedArgs& a) { return fits(mm_kernel(a), grouped_mm_grid(a)); }
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
static uint32_t big_grid(int64_t tiles) { return (uint32_t)std::min<int64_t>(tiles, device_cus_or_256() / 8 * 8); }

template <int DT, bool WT>
static void mm_staged(const GroupedArgs& a, Kernel k, dim3 grid, hipStream_t s) {
    if (k == Kernel::Split64) hipLaunchKernelGGL((grouped_mm_staged<DT, WT, 64, 4>), grid, dim3(1024), 0, s, a);
    else if (k == Kernel::Staged64) hipLaunchKernelGGL((grouped_mm_staged<DT, WT, 64, 1>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((grouped_mm_staged<DT, WT, 128, 1>), grid, dim3(256), 0, s, a);
}

hipError_t launch_grouped_mm(const GroupedArgs& a, bool trans_w, hipStream_t s) {
    const Kernel k = mm_kernel(a);
    const int64_t tiles = grouped_mm_grid(a);
    const dim3 grid((uint32_t)tiles);
    if (k == Kernel::Thin) {
        if (trans_w) hipLaunchKernelGGL((grouped_mm_thin<true>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((grouped_mm_thin<false>), grid, dim3(256), 0, s, a);
    } else if (k == Kernel::Big) {
        if (trans_w) hipLaunchKernelGGL((grouped_big<1>), dim3(big_grid(tiles)), dim3(512), 0, s, a, (int)tiles);
        else hipLaunchKernelGGL((grouped_big<0>), dim3(big_grid(tiles)), dim3(512), 0, s, a, (int)tiles);
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
        hipLaunchKernelGGL((grouped_big<2>), dim3(big_grid(tiles)), dim3(512), 0, s, a, (int)tiles);
    else if (a.dtype == 0) wgrad_staged<0>(a, k, grid, s);
    else wgrad_staged<1>(a, k, grid, s);
    return hipGetLastError();
}

}  // namespace himuon
