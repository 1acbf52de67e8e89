// Layer normalisation of rows on gfx950, forward and backward.
//     y  = (x - mean) r w + b,                  r = 1 / sqrt(var + eps)
//     dx = r (dy w - mean(dy w) - xh mean(dy w xh)),   xh = (x - mean) r
//     dw = sum over rows of dy xh,   db = sum over rows of dy
// A stream over the rows (HBM bound: one read and one write forward, two reads
// and one write backward), so a row is read once and held packed in registers by
// L threads (4 to 1024) in up to eight 16-byte chunks each; mean and variance are
// taken in two passes over the registers, in fp32: the second, over the differences to
// the mean, also corrects it in fp32, so a large mean costs y nothing (uncorrected, rows
// of 12000 values of 3e6 +- 1.5 came out wrong by up to 0.7; the time is the same).
// Rows may start at any alignment: chunks count from the row's first element.
//
// The sums over rows stay in the registers of the threads that own the columns: a
// workgroup goes through its rows and leaves 2 D fp32 sums, which a second launch
// adds in order (no atomics: the same inputs give the same bits).
//
// Measured, 16384 x 4096 in bf16, inputs from HBM: forward 59 us (4.6 TB/s; 47 on the same
// rows again, half of them still in the cache behind the L2), gradients 85 us, 4.5 of them
// the second launch (4.8 TB/s of the 0.40 GB; a large copy reaches 4.9).  fp32, on the
// same rows again: forward 98 us, gradients 152.

#include <algorithm>
#include <type_traits>

#include "device_util.h"
#include "norm.h"

namespace himuon {
namespace {

template <int DT> struct Elem;
template <> struct Elem<0> {
    using T = unsigned short;
    static constexpr int EPC = 8;
    __device__ static float get(const u32x4& c, int e) { return (e & 1) ? hi_f(c[e >> 1]) : lo_f(c[e >> 1]); }
    __device__ static float up(T x) { return bf2f(x); }
    __device__ static T down(float f) { return f2bf(f); }
};
template <> struct Elem<1> {
    using T = float;
    static constexpr int EPC = 4;
    __device__ static float get(const u32x4& c, int e) { return __uint_as_float(c[e]); }
    __device__ static float up(T x) { return x; }
    __device__ static T down(float f) { return f; }
};
struct __attribute__((packed, aligned(2))) Loose16 { u32x4 v; };   // 16 bytes at an element's alignment

// `by` bits (less than 128) out of the low end.
__device__ __forceinline__ u32x4 shift_down(const u32x4& v, int by) {
    const uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
    const uint64_t a = by == 0 ? lo : by < 64 ? lo >> by | hi << (64 - by) : hi >> (by - 64), b = by < 64 ? hi >> by : 0;
    return u32x4{(unsigned)a, (unsigned)(a >> 32), (unsigned)b, (unsigned)(b >> 32)};
}

// A row's chunk at element `at` (zeros from `cols` on).  WHOLE: rows of whole chunks.  A
// chunk that the row's end cuts is loaded from as much further left and shifted.
template <int DT, bool WHOLE>
__device__ __forceinline__ u32x4 load_chunk(const typename Elem<DT>::T* row, int at, int cols) {
    constexpr int EPC = Elem<DT>::EPC;
    if (at >= cols) return u32x4{0, 0, 0, 0};
    const int over = WHOLE ? 0 : max(at + EPC - cols, 0);
    if (WHOLE || cols >= EPC) {
        const u32x4 v = reinterpret_cast<const Loose16*>(row + at - over)->v;
        return over > 0 ? shift_down(v, over * (128 / EPC)) : v;
    }
    uint64_t w[2] = {0, 0};
#pragma unroll 1
    for (int e = 0; e < cols; ++e) {   // a row narrower than a chunk
        uint64_t x;
        if constexpr (DT == 0) x = row[e];
        else x = __float_as_uint(row[e]);
        w[e / (EPC / 2)] |= x << (128 / EPC * (e % (EPC / 2)));
    }
    return u32x4{(unsigned)w[0], (unsigned)(w[0] >> 32), (unsigned)w[1], (unsigned)(w[1] >> 32)};
}
template <int DT, bool WHOLE>
__device__ __forceinline__ void store_chunk(typename Elem<DT>::T* row, int at, int cols,
                                            const float (&f)[Elem<DT>::EPC]) {
    constexpr int EPC = Elem<DT>::EPC;
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = DT == 0 ? pack2(f[(2 * i) % EPC], f[(2 * i + 1) % EPC]) : __float_as_uint(f[i]);
    if (WHOLE || at + EPC <= cols) {
        reinterpret_cast<Loose16*>(row + at)->v = v;
        return;
    }
#pragma unroll 1
    for (int e = 0; at + e < cols; ++e) {
        const u32x4 x = shift_down(v, e * (128 / EPC));
        if constexpr (DT == 0) row[at + e] = (unsigned short)x[0];
        else row[at + e] = __uint_as_float(x[0]);
    }
}
// Values that are unpacked again where they are used next (unpacked once, the rows would
// take twice the registers).
template <int N>
__device__ __forceinline__ void stay_packed(u32x4 (&v)[N]) {
#pragma unroll
    for (int c = 0; c < N; ++c) asm volatile("" : "+v"(v[c]));
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// Sum over the aligned group of L lanes, the same in each of them.
template <int L>
__device__ __forceinline__ float lane_sum(float v) {
    v += dpp<0xB1>(v);                   // neighbours
    v += dpp<0x4E>(v);                   // pairs of a quad
    if (L >= 8) v += dpp<0x141>(v);      // quads of eight lanes (mirrored)
    if (L >= 16) v += dpp<0x140>(v);     // eights of sixteen lanes (mirrored)
    if (L >= 32) v += __shfl_xor(v, 16, 64);
    if (L >= 64) v += __shfl_xor(v, 32, 64);
    return v;
}
// Sums of a and b over the L threads of a row.  slots: LDS of the workgroup, two
// sets used in turn, so that one barrier a call is enough.
template <int L>
__device__ __forceinline__ void row_sum2(float& a, float& b, float2 (*slots)[16], int& turn) {
    a = lane_sum<(L < 64 ? L : 64)>(a);
    b = lane_sum<(L < 64 ? L : 64)>(b);
    if constexpr (L > 64) {
        constexpr int W = L / 64;
        float2* s = slots[turn] + threadIdx.x / L * W;   // of the row's waves
        turn ^= 1;
        if ((threadIdx.x & 63) == 0) s[threadIdx.x % L >> 6] = make_float2(a, b);
        __syncthreads();
        a = s[0].x;
        b = s[0].y;
#pragma unroll
        for (int w = 1; w < W; ++w) {
            a += s[w].x;
            b += s[w].y;
        }
    }
}

// Threads of a forward pass's workgroup that holds rows with L threads each.
template <int L> constexpr int kGroup = L > 256 ? L : 256;

template <int DT, int L, int CH, bool WHOLE>
__global__ __launch_bounds__(kGroup<L>) void norm_forward(const NormArgs a) {
    using T = typename Elem<DT>::T;
    constexpr int EPC = Elem<DT>::EPC, G = kGroup<L> / L;
    // (bf16 rows with a mean far above their spread lie in two binades: their sums are exact)
    constexpr bool CORRECT = DT == 1;
    __shared__ float2 slots[2][16];
    int turn = 0;
    const int l = threadIdx.x % L;
    const float n = (float)a.cols;
    const int64_t step = (int64_t)gridDim.x * G;
    for (int64_t first = (int64_t)blockIdx.x * G; first < a.rows; first += step) {   // the same in all threads
        const int64_t row = first + threadIdx.x / L;
        const bool live = row < a.rows;
        const T* x = reinterpret_cast<const T*>(a.x) + (live ? row * a.x_ld : 0);
        const int cols = live ? a.cols : 0;
        u32x4 v[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) v[c] = load_chunk<DT, WHOLE>(x, (c * L + l) * EPC, cols);
        float sum = 0.f, none = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int e = 0; e < EPC; ++e) sum += Elem<DT>::get(v[c], e);
        stay_packed(v);
        row_sum2<L>(sum, none, slots, turn);
        const float about = sum / n;
        float var = 0.f, rest = 0.f;   // sums of squares and of differences
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int in = cols - (c * L + l) * EPC;
            if (in <= 0) continue;
#pragma unroll
            for (int e = 0; e < EPC; ++e) {
                const float d = Elem<DT>::get(v[c], e) - about;
                if (CORRECT) rest += WHOLE || e < in ? d : 0.f;
                var += WHOLE || e < in ? d * d : 0.f;
            }
        }
        stay_packed(v);
        row_sum2<L>(var, CORRECT ? rest : none, slots, turn);
        var /= n;
        if constexpr (CORRECT) {
            // `about` is off by its sum's roundings, the more the larger the mean; the mean of the
            // differences is that error, to their own roundings.  (Where all values are equal, so are the
            // differences, and all of this is exact: 0.)  Where the squares are infinite, rstd is 0, and
            // their sum may be infinite or NaN too.
            rest = var < __uint_as_float(0x7f800000u) ? rest / n : 0.f;
            var = fmaf(-rest, rest, var);
            var = var < 0.f ? 0.f : var;   // (NaN stays)
        }
        const float r = 1.f / sqrtf(var + a.eps);
        if (!live) continue;   // (no barrier below)
        if (l == 0 && a.stats != nullptr)
            *reinterpret_cast<float2*>(a.stats + 2 * row) = make_float2(CORRECT ? about + rest : about, r);
        T* y = reinterpret_cast<T*>(a.y) + row * a.y_ld;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int at = (c * L + l) * EPC;
            if (at >= cols) continue;
            float f[EPC];
#pragma unroll
            for (int e = 0; e < EPC; ++e) {
                const float d = Elem<DT>::get(v[c], e) - about;
                f[e] = (CORRECT ? d - rest : d) * r;
            }
            if (a.weight != nullptr) {
                const u32x4 w = load_chunk<DT, WHOLE>(reinterpret_cast<const T*>(a.weight), at, cols);
#pragma unroll
                for (int e = 0; e < EPC; ++e) f[e] *= Elem<DT>::get(w, e);
            }
            if (a.bias != nullptr) {
                const u32x4 b = load_chunk<DT, WHOLE>(reinterpret_cast<const T*>(a.bias), at, cols);
#pragma unroll
                for (int e = 0; e < EPC; ++e) f[e] += Elem<DT>::get(b, e);
            }
            store_chunk<DT, WHOLE>(y, at, cols, f);
        }
    }
}

// A workgroup of 1024 threads goes through 1024 / L rows at a time, the next ones loaded
// while those are worked on (AHEAD; not where the registers would not hold both).  Rows
// of more than two chunks a thread leave no room for their sums (SUMS = false): those
// are norm_columns' (2048 x 32768 in bf16 with the sums here 325 us).
constexpr int kBackward = 1024;
template <int DT, int L, int CH, bool WHOLE>
__global__ __launch_bounds__(kBackward) void norm_backward(const NormArgs a) {
    using T = typename Elem<DT>::T;
    constexpr int EPC = Elem<DT>::EPC, G = kBackward / L;
    constexpr bool AHEAD = CH * EPC <= 8, SUMS = CH <= 2;
    __shared__ float2 slots[2][16];
    int turn = 0;
    const int l = threadIdx.x % L;
    const float inv = 1.f / (float)a.cols;
    float dw[SUMS ? CH : 1][EPC], db[SUMS ? CH : 1][EPC];
    u32x4 wv[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        constexpr unsigned kOne = DT == 0 ? 0x3f803f80u : 0x3f800000u;
        wv[c] = a.weight != nullptr ? load_chunk<DT, WHOLE>(reinterpret_cast<const T*>(a.weight), (c * L + l) * EPC, a.cols)
                                    : u32x4{kOne, kOne, kOne, kOne};
        if (SUMS)
#pragma unroll
            for (int e = 0; e < EPC; ++e) dw[c][e] = db[c][e] = 0.f;
    }
    struct Rows {
        u32x4 x[CH], g[CH];
        float2 st;
    };
    const auto load = [&](int64_t row, Rows& p) __attribute__((always_inline)) {
        const bool live = row < a.rows;
        const T* x = reinterpret_cast<const T*>(a.x) + (live ? row * a.x_ld : 0);
        const T* dy = reinterpret_cast<const T*>(a.dy) + (live ? row * a.dy_ld : 0);
        p.st = live ? *reinterpret_cast<const float2*>(a.stats + 2 * row) : make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            p.x[c] = load_chunk<DT, WHOLE>(x, (c * L + l) * EPC, live ? a.cols : 0);
            p.g[c] = load_chunk<DT, WHOLE>(dy, (c * L + l) * EPC, live ? a.cols : 0);
        }
    };
    const int64_t step = (int64_t)gridDim.x * G, mine = threadIdx.x / L;
    Rows p;
    load((int64_t)blockIdx.x * G + mine, p);
    for (int64_t first = (int64_t)blockIdx.x * G; first < a.rows; first += step) {   // the same in all threads
        const int64_t row = first + mine;
        Rows q;
        if (AHEAD) load(row + step, q);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            // past the row's end x_hat is 0: there x is 0, and where -mean rstd is infinite its product
            // with g, 0 there too, would be NaN
            const int in = a.cols - (c * L + l) * EPC;
            const float mean = in > 0 ? p.st.x : 0.f;
#pragma unroll
            for (int e = 0; e < EPC; ++e) {
                const float d = Elem<DT>::get(p.x[c], e) - mean;
                const float g = Elem<DT>::get(p.g[c], e), xh = (WHOLE || e < in ? d : 0.f) * p.st.y;
                if (SUMS) {
                    db[c][e] += g;
                    dw[c][e] += g * xh;   // (past the row's end g is 0)
                }
                const float gw = g * Elem<DT>::get(wv[c], e);
                s1 += gw;
                s2 += gw * xh;
            }
        }
        stay_packed(p.x);
        stay_packed(p.g);
        stay_packed(wv);
        if (a.dx != nullptr) {
            row_sum2<L>(s1, s2, slots, turn);
            s1 *= inv;
            s2 *= inv;
            T* dx = reinterpret_cast<T*>(a.dx) + row * a.dx_ld;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int at = (c * L + l) * EPC;
                if (row >= a.rows || at >= a.cols) continue;
                float f[EPC];
#pragma unroll
                for (int e = 0; e < EPC; ++e) {
                    const float g = Elem<DT>::get(p.g[c], e), xh = (Elem<DT>::get(p.x[c], e) - p.st.x) * p.st.y;
                    f[e] = p.st.y * (g * Elem<DT>::get(wv[c], e) - s1 - xh * s2);
                }
                store_chunk<DT, WHOLE>(dx, at, a.cols, f);
            }
        }
        if (AHEAD) p = q;
        else if (first + step < a.rows) load(row + step, p);
    }
    if (a.part == nullptr) return;
    // ---- the workgroup's sums: its groups of threads in order, dw then db
    float* to = a.part + (int64_t)blockIdx.x * 2 * a.cols;
    if constexpr (!SUMS) {
    } else if constexpr (G == 1) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int e = 0; e < EPC; ++e) {
                const int at = (c * L + l) * EPC + e;
                if (at < a.cols) {
                    to[at] = dw[c][e];
                    to[a.cols + at] = db[c][e];
                }
            }
    } else {
        __shared__ float sums[G][CH * L * EPC];
        const int group = threadIdx.x / L;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k) __syncthreads();
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int e = 0; e < EPC; ++e) sums[group][(c * L + l) * EPC + e] = k ? db[c][e] : dw[c][e];
            __syncthreads();
            for (int i = threadIdx.x; i < a.cols; i += kBackward) {
                float s = sums[0][i];
                for (int g = 1; g < G; ++g) s += sums[g][i];
                to[k * a.cols + i] = s;
            }
        }
    }
}

// The sums over rows alone, of 256 chunks of columns (blockIdx.x) and one of gridDim.y
// parts of the rows, the next rows loaded while kRows are added.
template <int DT, bool WHOLE>
__global__ __launch_bounds__(256) void norm_columns(const NormArgs a) {
    using T = typename Elem<DT>::T;
    constexpr int EPC = Elem<DT>::EPC, kRows = 4;
    const int at = (int)(blockIdx.x * 256 + threadIdx.x) * EPC;
    const int64_t from = (int64_t)a.rows * blockIdx.y / gridDim.y, to = (int64_t)a.rows * (blockIdx.y + 1) / gridDim.y;
    float dw[EPC], db[EPC];
#pragma unroll
    for (int e = 0; e < EPC; ++e) dw[e] = db[e] = 0.f;
    struct Rows {
        u32x4 x[kRows], g[kRows];
        float2 st[kRows];
    };
    const auto load = [&](int64_t row, Rows& p) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const bool live = row + k < to;
            const int64_t r = live ? row + k : 0;
            p.x[k] = load_chunk<DT, WHOLE>(reinterpret_cast<const T*>(a.x) + r * a.x_ld, at, live ? a.cols : 0);
            p.g[k] = load_chunk<DT, WHOLE>(reinterpret_cast<const T*>(a.dy) + r * a.dy_ld, at, live ? a.cols : 0);
            p.st[k] = live ? *reinterpret_cast<const float2*>(a.stats + 2 * r) : make_float2(0.f, 0.f);
        }
    };
    Rows p;
    load(from, p);
    for (int64_t row = from; row < to; row += kRows) {
        Rows q;
        load(row + kRows, q);
#pragma unroll
        for (int k = 0; k < kRows; ++k)
#pragma unroll
            for (int e = 0; e < EPC; ++e) {
                const float g = Elem<DT>::get(p.g[k], e);
                db[e] += g;
                dw[e] += g * ((Elem<DT>::get(p.x[k], e) - p.st[k].x) * p.st[k].y);
            }
        p = q;
    }
    float* out = a.part + (int64_t)blockIdx.y * 2 * a.cols;
#pragma unroll
    for (int e = 0; e < EPC; ++e)
        if (at + e < a.cols) {
            out[at + e] = dw[e];
            out[a.cols + at + e] = db[e];
        }
}

// Adds the workgroups' sums in order: 64 of the 2 D columns by 16 runs of
// workgroups, whose sums are added in order too.
template <int DT>
__global__ __launch_bounds__(1024) void norm_join(const NormArgs a, const int parts) {
    using T = typename Elem<DT>::T;
    __shared__ float sums[16][64];
    const int i = threadIdx.x & 63, run = threadIdx.x >> 6;
    const int64_t col = (int64_t)blockIdx.x * 64 + i;
    const int64_t width = 2 * (int64_t)a.cols;
    const int from = (int)((int64_t)parts * run / 16), to = (int)((int64_t)parts * (run + 1) / 16);
    float s = 0.f;
    if (col < width) {
        const float* p = a.part + from * width + col;
#pragma unroll 8
        for (int k = from; k < to; ++k, p += width) s += *p;
    }
    sums[run][i] = s;
    __syncthreads();
    if (run != 0 || col >= width) return;
#pragma unroll
    for (int k = 1; k < 16; ++k) s += sums[k][i];
    T* out = reinterpret_cast<T*>(col < a.cols ? a.dw : a.db);
    if (out != nullptr) out[col < a.cols ? col : col - a.cols] = Elem<DT>::down(s);
}

int cus_or_256() {
    static const int cus = [] { const int c = device_cus(); return c >= 8 ? std::min(c, 512) : 256; }();
    return cus;
}
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How rows are held: L threads of CH chunks.
struct Shape { int l, ch; };
// Few rows take more threads each (4 x 4096 in bf16 with 64 threads a row 6.2 us, with
// 256 3.8).
Shape forward_shape(int32_t rows, int32_t cols, int32_t dtype) {
    const int64_t c = cdiv(cols, dtype == 0 ? 8 : 4);   // chunks of a row
    if (rows <= 4 * cus_or_256() && c > 64 && c <= 512) return {256, c <= 256 ? 1 : 2};
    if (c <= 4) return {4, 1};
    if (c <= 16) return {16, 1};
    if (c <= 64) return {64, 1};
    if (c <= 128) return {64, 2};
    if (c <= 256) return {64, 4};
    if (c <= 512) return {64, 8};
    if (c <= 1024) return {256, 4};
    if (c <= 2048) return {256, 8};
    if (c <= 4096) return {1024, 4};
    return {1024, 8};
}
// (One chunk a thread as far as 1024 threads reach: with two in bf16 and the next rows
// ahead, the sums spilled.  Two, above 8192 columns, fetch no rows ahead there; odd widths
// still spill 20 registers.  Four, without the sums: none, and at odd widths 48 in bf16
// and 24 in fp32.  Eight, fp32 rows above 16384 columns: 101, at odd widths 309; 2048 x
// 32768 take 500 us, x 32767 835.)
Shape backward_shape(int32_t cols, int32_t dtype) {
    const int64_t c = cdiv(cols, dtype == 0 ? 8 : 4);
    int l = 4;
    while (l < c && l < kBackward) l *= 2;
    int ch = 1;
    while ((int64_t)l * ch < c) ch *= 2;
    return {l, ch};
}

// Whether the sums over rows are a launch of their own.
bool apart(const Shape& s) { return s.ch > 2; }
// Workgroups of a gradient: one on a CU, and no more than have rows (apart: parts of the
// rows, of which there are four workgroups on a CU with the slabs of columns).
int64_t backward_groups(int32_t rows, const Shape& s) {
    if (apart(s)) return std::max<int64_t>(1, std::min<int64_t>(cdiv(rows, 4), cus_or_256() / s.ch));
    return std::max<int64_t>(1, std::min<int64_t>(cdiv(rows, kBackward / s.l), cus_or_256()));
}

template <int DT, int L, int CH>
hipError_t forward_of(const NormArgs& a, hipStream_t s) {
    constexpr int G = kGroup<L> / L;
    const dim3 grid((uint32_t)std::min<int64_t>(cdiv(a.rows, G), (int64_t)cus_or_256() * 64)), threads(kGroup<L>);
    if (a.cols % Elem<DT>::EPC == 0) hipLaunchKernelGGL((norm_forward<DT, L, CH, true>), grid, threads, 0, s, a);
    else hipLaunchKernelGGL((norm_forward<DT, L, CH, false>), grid, threads, 0, s, a);
    return hipGetLastError();
}
template <int DT>
hipError_t forward(const NormArgs& a, hipStream_t s) {
    const Shape sh = forward_shape(a.rows, a.cols, DT);
    switch (sh.l * 16 + sh.ch) {
        case 4 * 16 + 1: return forward_of<DT, 4, 1>(a, s);
        case 16 * 16 + 1: return forward_of<DT, 16, 1>(a, s);
        case 64 * 16 + 1: return forward_of<DT, 64, 1>(a, s);
        case 64 * 16 + 2: return forward_of<DT, 64, 2>(a, s);
        case 64 * 16 + 4: return forward_of<DT, 64, 4>(a, s);
        case 64 * 16 + 8: return forward_of<DT, 64, 8>(a, s);
        case 256 * 16 + 1: return forward_of<DT, 256, 1>(a, s);
        case 256 * 16 + 2: return forward_of<DT, 256, 2>(a, s);
        case 256 * 16 + 4: return forward_of<DT, 256, 4>(a, s);
        case 256 * 16 + 8: return forward_of<DT, 256, 8>(a, s);
        case 1024 * 16 + 4: return forward_of<DT, 1024, 4>(a, s);
    }
    if constexpr (DT == 1) return forward_of<DT, 1024, 8>(a, s);
    return hipErrorInvalidValue;
}

template <int DT, int L, int CH>
hipError_t backward_of(const NormArgs& a, uint32_t groups, hipStream_t s) {
    if (a.cols % Elem<DT>::EPC == 0) hipLaunchKernelGGL((norm_backward<DT, L, CH, true>), dim3(groups), dim3(kBackward), 0, s, a);
    else hipLaunchKernelGGL((norm_backward<DT, L, CH, false>), dim3(groups), dim3(kBackward), 0, s, a);
    return hipGetLastError();
}
template <int DT>
hipError_t backward_rows(const NormArgs& a, const Shape& sh, uint32_t g, hipStream_t s) {
    if (sh.ch == 1) {
        switch (sh.l) {
            case 4: return backward_of<DT, 4, 1>(a, g, s);
            case 8: return backward_of<DT, 8, 1>(a, g, s);
            case 16: return backward_of<DT, 16, 1>(a, g, s);
            case 32: return backward_of<DT, 32, 1>(a, g, s);
            case 64: return backward_of<DT, 64, 1>(a, g, s);
            case 128: return backward_of<DT, 128, 1>(a, g, s);
            case 256: return backward_of<DT, 256, 1>(a, g, s);
            case 512: return backward_of<DT, 512, 1>(a, g, s);
            default: return backward_of<DT, 1024, 1>(a, g, s);
        }
    }
    if (sh.ch == 2) return backward_of<DT, 1024, 2>(a, g, s);
    if (sh.ch == 4) return backward_of<DT, 1024, 4>(a, g, s);
    if constexpr (DT == 1) return backward_of<DT, 1024, 8>(a, g, s);
    return hipErrorInvalidValue;
}
template <int DT>
hipError_t backward(const NormArgs& a, hipStream_t s) {
    const Shape sh = backward_shape(a.cols, DT);
    const uint32_t groups = (uint32_t)backward_groups(a.rows, sh);
    if (!apart(sh)) {
        const hipError_t e = backward_rows<DT>(a, sh, groups, s);
        if (e != hipSuccess || a.part == nullptr) return e;
    } else {
        if (a.part != nullptr) {   // first, as dx may be written over dy or x
            const dim3 grid((uint32_t)cdiv(a.cols, 256 * Elem<DT>::EPC), groups);
            if (a.cols % Elem<DT>::EPC == 0) hipLaunchKernelGGL((norm_columns<DT, true>), grid, dim3(256), 0, s, a);
            else hipLaunchKernelGGL((norm_columns<DT, false>), grid, dim3(256), 0, s, a);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        if (a.dx != nullptr && a.rows > 0) {
            const hipError_t e = backward_rows<DT>(a, sh, (uint32_t)std::min<int64_t>(a.rows, 2 * cus_or_256()), s);
            if (e != hipSuccess || a.part == nullptr) return e;
        }
    }
    hipLaunchKernelGGL((norm_join<DT>), dim3((uint32_t)cdiv(2 * (int64_t)a.cols, 64)), dim3(1024), 0, s, a, (int)groups);
    return hipGetLastError();
}

}  // namespace

int64_t norm_grad_bytes(int32_t rows, int32_t cols, int32_t dtype) {
    return backward_groups(rows, backward_shape(cols, dtype)) * 2 * cols * (int64_t)sizeof(float);
}

hipError_t launch_layer_norm(const NormArgs& a, hipStream_t s) { return a.dtype == 0 ? forward<0>(a, s) : forward<1>(a, s); }
hipError_t launch_layer_norm_grad(const NormArgs& a, hipStream_t s) {
    return a.dtype == 0 ? backward<0>(a, s) : backward<1>(a, s);
}

}  // namespace himuon
