// Layer normalisation of rows on gfx950, forward and backward.
//     y  = (x - mean) r w + b,                  r = 1 / sqrt(var + eps)
//     dx = r (dy w - mean(dy w) - xh mean(dy w xh)),   xh = (x - mean) r
//     dw = sum over rows of dy xh,   db = sum over rows of dy
// A stream over the rows (HBM bound: one read and one write forward, two reads
// and one write backward), so a row is read once and held packed in registers by
// L threads (4 to 1024) in up to eight 16-byte chunks each; mean and variance are
// taken in two passes over the registers, in fp32, so a large mean costs nothing.
// Rows may start at any alignment: chunks count from the row's first element.
//
// The sums over rows stay in the registers of the threads that own the columns: a
// workgroup goes through its rows and leaves 2 D fp32 sums, which a second launch
// adds in order (no atomics: the same inputs give the same bits).

#include <algorithm>

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

// A row's chunk at element `at` (zeros from `cols` on).
template <int DT>
__device__ __forceinline__ u32x4 load_chunk(const typename Elem<DT>::T* row, int at, int cols) {
    constexpr int EPC = Elem<DT>::EPC;
    if (at + EPC <= cols) return reinterpret_cast<const Loose16*>(row + at)->v;
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < EPC - 1; ++e)
        if (at + e < cols) {
            if constexpr (DT == 0) v[e >> 1] |= (unsigned)row[at + e] << (16 * (e & 1));
            else v[e] = __float_as_uint(row[at + e]);
        }
    return v;
}
template <int DT>
__device__ __forceinline__ void store_chunk(typename Elem<DT>::T* row, int at, int cols,
                                            const float (&f)[Elem<DT>::EPC]) {
    constexpr int EPC = Elem<DT>::EPC;
    if (at + EPC <= cols) {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = DT == 0 ? pack2(f[(2 * i) % EPC], f[(2 * i + 1) % EPC]) : __float_as_uint(f[i]);
        reinterpret_cast<Loose16*>(row + at)->v = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < EPC - 1; ++e)
        if (at + e < cols) row[at + e] = Elem<DT>::down(f[e]);
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
    if (L >= 16) {
        v += dpp<0x141>(v);              // quads of eight lanes (mirrored)
        v += dpp<0x140>(v);              // eights of sixteen lanes (mirrored)
    }
    if (L >= 64) {
        v += __shfl_xor(v, 16, 64);
        v += __shfl_xor(v, 32, 64);
    }
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
        float2* s = slots[turn];
        turn ^= 1;
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) s[wave] = make_float2(a, b);
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

// Threads of a workgroup that holds rows with L threads each.
template <int L> constexpr int kGroup = L > 256 ? L : 256;

template <int DT, int L, int CH>
__global__ __launch_bounds__(kGroup<L>) void norm_forward(const NormArgs a) {
    using T = typename Elem<DT>::T;
    constexpr int EPC = Elem<DT>::EPC, G = kGroup<L> / L;
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
        for (int c = 0; c < CH; ++c) v[c] = load_chunk<DT>(x, (c * L + l) * EPC, cols);
        float sum = 0.f, none = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int e = 0; e < EPC; ++e) sum += Elem<DT>::get(v[c], e);
        row_sum2<L>(sum, none, slots, turn);
        const float mean = sum / n;   // (exact where all values are equal)
        float var = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int at = (c * L + l) * EPC;
#pragma unroll
            for (int e = 0; e < EPC; ++e) {
                const float d = Elem<DT>::get(v[c], e) - mean;
                var += at + e < cols ? d * d : 0.f;
            }
        }
        row_sum2<L>(var, none, slots, turn);
        const float r = 1.f / sqrtf(var / n + a.eps);
        if (!live) continue;   // (no barrier below)
        if (l == 0 && a.stats != nullptr) *reinterpret_cast<float2*>(a.stats + 2 * row) = make_float2(mean, r);
        T* y = reinterpret_cast<T*>(a.y) + row * a.y_ld;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int at = (c * L + l) * EPC;
            if (at >= cols) continue;
            float f[EPC];
#pragma unroll
            for (int e = 0; e < EPC; ++e) f[e] = (Elem<DT>::get(v[c], e) - mean) * r;
            if (a.weight != nullptr) {
                const u32x4 w = load_chunk<DT>(reinterpret_cast<const T*>(a.weight), at, cols);
#pragma unroll
                for (int e = 0; e < EPC; ++e) f[e] *= Elem<DT>::get(w, e);
            }
            if (a.bias != nullptr) {
                const u32x4 b = load_chunk<DT>(reinterpret_cast<const T*>(a.bias), at, cols);
#pragma unroll
                for (int e = 0; e < EPC; ++e) f[e] += Elem<DT>::get(b, e);
            }
            store_chunk<DT>(y, at, cols, f);
        }
    }
}

template <int DT, int L, int CH>
__global__ __launch_bounds__(kGroup<L>) void norm_backward(const NormArgs a) {
    using T = typename Elem<DT>::T;
    constexpr int EPC = Elem<DT>::EPC, G = kGroup<L> / L;
    __shared__ float2 slots[2][16];
    int turn = 0;
    const int l = threadIdx.x % L;
    const float inv = 1.f / (float)a.cols;
    float dw[CH][EPC], db[CH][EPC];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e = 0; e < EPC; ++e) dw[c][e] = db[c][e] = 0.f;
    const int64_t step = (int64_t)gridDim.x * G;
    for (int64_t first = (int64_t)blockIdx.x * G; first < a.rows; first += step) {
        const int64_t row = first + threadIdx.x / L;
        const bool live = row < a.rows;
        const T* x = reinterpret_cast<const T*>(a.x) + (live ? row * a.x_ld : 0);
        const T* dy = reinterpret_cast<const T*>(a.dy) + (live ? row * a.dy_ld : 0);
        const int cols = live ? a.cols : 0;
        const float2 st = live ? *reinterpret_cast<const float2*>(a.stats + 2 * row) : make_float2(0.f, 0.f);
        u32x4 xv[CH], gv[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            xv[c] = load_chunk<DT>(x, (c * L + l) * EPC, cols);
            gv[c] = load_chunk<DT>(dy, (c * L + l) * EPC, cols);
        }
        float s1 = 0.f, s2 = 0.f;
        u32x4 wv[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if (a.weight != nullptr) wv[c] = load_chunk<DT>(reinterpret_cast<const T*>(a.weight), (c * L + l) * EPC, cols);
#pragma unroll
            for (int e = 0; e < EPC; ++e) {
                const float g = Elem<DT>::get(gv[c], e), xh = (Elem<DT>::get(xv[c], e) - st.x) * st.y;
                db[c][e] += g;
                dw[c][e] += g * xh;   // (past the row's end g is 0)
                const float gw = a.weight != nullptr ? g * Elem<DT>::get(wv[c], e) : g;
                s1 += gw;
                s2 += gw * xh;
            }
        }
        if (a.dx == nullptr) continue;
        row_sum2<L>(s1, s2, slots, turn);
        s1 *= inv;
        s2 *= inv;
        if (!live) continue;   // (no barrier below)
        T* dx = reinterpret_cast<T*>(a.dx) + row * a.dx_ld;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int at = (c * L + l) * EPC;
            if (at >= cols) continue;
            float f[EPC];
#pragma unroll
            for (int e = 0; e < EPC; ++e) {
                const float g = Elem<DT>::get(gv[c], e), xh = (Elem<DT>::get(xv[c], e) - st.x) * st.y;
                const float gw = a.weight != nullptr ? g * Elem<DT>::get(wv[c], e) : g;
                f[e] = st.y * (gw - s1 - xh * s2);
            }
            store_chunk<DT>(dx, at, cols, f);
        }
    }
    if (a.part == nullptr) return;
    // ---- the workgroup's sums: its groups of threads in order, dw then db
    float* to = a.part + (int64_t)blockIdx.x * 2 * a.cols;
    if constexpr (G == 1) {
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
            for (int i = threadIdx.x; i < a.cols; i += kGroup<L>) {
                float s = sums[0][i];
#pragma unroll
                for (int g = 1; g < G; ++g) s += sums[g][i];
                to[k * a.cols + i] = s;
            }
        }
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
Shape shape_of(int32_t cols, int32_t dtype) {
    const int64_t c = cdiv(cols, dtype == 0 ? 8 : 4);   // chunks of a row
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

// Workgroups of a gradient: two on a CU, and no more than have rows.
int64_t backward_groups(int32_t rows, const Shape& s) {
    const int64_t g = s.l > 256 ? 1 : 256 / s.l;
    return std::max<int64_t>(1, std::min<int64_t>(cdiv(rows, g), 2 * cus_or_256()));
}

template <int DT, typename F>
hipError_t with_shape(const Shape& s, F f) {
#define HIMUON_SHAPE(L, CH) \
    if (s.l == L && s.ch == CH) return f(std::integral_constant<int, L>{}, std::integral_constant<int, CH>{})
    HIMUON_SHAPE(4, 1);
    HIMUON_SHAPE(16, 1);
    HIMUON_SHAPE(64, 1);
    HIMUON_SHAPE(64, 2);
    HIMUON_SHAPE(64, 4);
    HIMUON_SHAPE(64, 8);
    HIMUON_SHAPE(256, 4);
    HIMUON_SHAPE(256, 8);
    HIMUON_SHAPE(1024, 4);
    if constexpr (DT == 1) HIMUON_SHAPE(1024, 8);
#undef HIMUON_SHAPE
    return hipErrorInvalidValue;
}

template <int DT>
hipError_t forward(const NormArgs& a, hipStream_t s) {
    return with_shape<DT>(shape_of(a.cols, DT), [&](auto l, auto ch) {
        constexpr int L = decltype(l)::value, CH = decltype(ch)::value, G = kGroup<L> / L;
        const int64_t groups = std::min<int64_t>(cdiv(a.rows, G), (int64_t)cus_or_256() * 64);
        hipLaunchKernelGGL((norm_forward<DT, L, CH>), dim3((uint32_t)groups), dim3(kGroup<L>), 0, s, a);
        return hipGetLastError();
    });
}

template <int DT>
hipError_t backward(const NormArgs& a, hipStream_t s) {
    const Shape sh = shape_of(a.cols, DT);
    const int64_t groups = backward_groups(a.rows, sh);
    const hipError_t e = with_shape<DT>(sh, [&](auto l, auto ch) {
        constexpr int L = decltype(l)::value, CH = decltype(ch)::value;
        hipLaunchKernelGGL((norm_backward<DT, L, CH>), dim3((uint32_t)groups), dim3(kGroup<L>), 0, s, a);
        return hipGetLastError();
    });
    if (e != hipSuccess || a.part == nullptr) return e;
    hipLaunchKernelGGL((norm_join<DT>), dim3((uint32_t)cdiv(2 * (int64_t)a.cols, 64)), dim3(1024), 0, s, a, (int)groups);
    return hipGetLastError();
}

}  // namespace

int64_t norm_grad_bytes(int32_t rows, int32_t cols, int32_t dtype) {
    return backward_groups(rows, shape_of(cols, dtype)) * 2 * cols * (int64_t)sizeof(float);
}

hipError_t launch_layer_norm(const NormArgs& a, hipStream_t s) { return a.dtype == 0 ? forward<0>(a, s) : forward<1>(a, s); }
hipError_t launch_layer_norm_grad(const NormArgs& a, hipStream_t s) {
    return a.dtype == 0 ? backward<0>(a, s) : backward<1>(a, s);
}

}  // namespace himuon
