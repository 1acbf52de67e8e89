// AdamW over many tensors at once on gfx950, element by element:
//     m <- beta1 m + (1 - beta1) g,   v <- beta2 v + (1 - beta2) g^2
//     w <- (1 - lr decay) w - lr m / (1 - beta1^t) / (sqrt(v / (1 - beta2^t)) + eps)
// with the states m and v in fp32, or in 8 bits: codes of m and of r = sqrt(v) in
// e4m3 (4 exponent and 3 mantissa bits), times an fp32 scale for each block of 256
// elements of a tensor, chosen so that the block's largest is 448.  r rather than v
// is held since the update divides by it: 17 binades of r are 34 of v.
//
// Codes are rounded up or down by 16 random bits an element (a hash of the step and
// the element's index in its tensor): a moving average whose relative change in a
// step is below half a code step (beta2 = 0.999: 0.05 % of r against 6 %) would
// never move if it were rounded to nearest.  What is not zero in r is never rounded
// to zero, as the update divides by it.
//
// A stream (HBM bound: 16 + 2 size(w) + size(g) bytes an element, in 8 bits 4.06 +
// 2 size(w) + size(g)).  One launch takes 256 tensors: a workgroup takes units of
// 4096 elements and finds a unit's tensor in the table of the kernel arguments.
// Measured: 262 M bf16 weights with 8-bit states 566 to 590 us (4.6 TB/s; about 65 vector
// instructions an element, near the rate's share of them), with 32-bit states 1128 us
// (5.1 TB/s); 96 tensors of 2048 fp32 weights 5.5 us one launch after the other, 7.5 to 8
// alone.

#include <algorithm>

#include "adamw.h"
#include "device_util.h"

namespace himuon {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
struct __attribute__((packed, aligned(2))) Loose16 { u32x4 v; };   // at an element's alignment
struct __attribute__((packed, aligned(1))) Loose8 { u32x2 v; };

template <int DT> struct Elem;
template <> struct Elem<0> {
    using T = unsigned short;
    __device__ static float up(T x) { return bf2f(x); }
    __device__ static T down(float f) { return f2bf(f); }
};
template <> struct Elem<1> {
    using T = float;
    __device__ static float up(T x) { return x; }
    __device__ static T down(float f) { return f; }
};

template <int DT>
__device__ __forceinline__ void load8(const typename Elem<DT>::T* p, float (&f)[8]) {
    if constexpr (DT == 0) {
        const u32x4 c = reinterpret_cast<const Loose16*>(p)->v;
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = (e & 1) ? hi_f(c[e >> 1]) : lo_f(c[e >> 1]);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const u32x4 c = reinterpret_cast<const Loose16*>(p + 4 * h)->v;
#pragma unroll
            for (int e = 0; e < 4; ++e) f[4 * h + e] = __uint_as_float(c[e]);
        }
    }
}
template <int DT>
__device__ __forceinline__ void store8(typename Elem<DT>::T* p, const float (&f)[8]) {
    if constexpr (DT == 0) {
        reinterpret_cast<Loose16*>(p)->v = u32x4{pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])};
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            reinterpret_cast<Loose16*>(p + 4 * h)->v = u32x4{__float_as_uint(f[4 * h]), __float_as_uint(f[4 * h + 1]),
                                                             __float_as_uint(f[4 * h + 2]), __float_as_uint(f[4 * h + 3])};
    }
}

// Eight elements of a tensor from flat index `at`, `here` of them (0 to 8) inside.
// WHOLE: all of the unit's are, in one run of memory.
template <bool WHOLE>
struct Place {
    int64_t at;
    int here;
    int64_t row, col;   // where the rows have gaps
    __device__ __forceinline__ Place(const AdamwTensor& t, int64_t base, int in) : at(base + in), here(8), row(0), col(0) {
        if (WHOLE) return;
        here = (int)max((int64_t)0, min((int64_t)8, t.numel - at));
        if (t.cols != 0) {
            row = at / t.cols;
            col = at - row * t.cols;
        }
    }
    // in one run of memory: the offset of its first element
    __device__ __forceinline__ bool run(const AdamwTensor& t) const {
        return WHOLE || (here == 8 && (t.cols == 0 || col + 8 <= t.cols));
    }
    __device__ __forceinline__ int64_t offset(const AdamwTensor& t, int64_t ld) const {
        return WHOLE || t.cols == 0 ? at : row * ld + col;
    }
    __device__ __forceinline__ int64_t offset(const AdamwTensor& t, int64_t ld, int e) const {
        if (t.cols == 0) return at + e;
        int64_t r = row, c = col + e;
        while (c >= t.cols) {
            c -= t.cols;
            ++r;
        }
        return r * ld + c;
    }
};
template <int DT, bool WHOLE>
__device__ __forceinline__ void load_part(const AdamwTensor& t, const void* base, int64_t ld, const Place<WHOLE>& p,
                                          float (&f)[8]) {
    using T = typename Elem<DT>::T;
    const T* q = reinterpret_cast<const T*>(base);
    if (p.run(t)) {
        load8<DT>(q + p.offset(t, ld), f);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = e < p.here ? Elem<DT>::up(q[p.offset(t, ld, e)]) : 0.f;
}
template <int DT, bool WHOLE>
__device__ __forceinline__ void store_part(const AdamwTensor& t, void* base, int64_t ld, const Place<WHOLE>& p,
                                           const float (&f)[8]) {
    using T = typename Elem<DT>::T;
    T* q = reinterpret_cast<T*>(base);
    if (p.run(t)) {
        store8<DT>(q + p.offset(t, ld), f);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < p.here) q[p.offset(t, ld, e)] = Elem<DT>::down(f[e]);
}

template <bool WHOLE>
__device__ __forceinline__ u32x2 load_codes(const void* base, const Place<WHOLE>& p) {
    const unsigned char* q = reinterpret_cast<const unsigned char*>(base) + p.at;
    if (p.here == 8) return reinterpret_cast<const Loose8*>(q)->v;
    u32x2 c = {0, 0};
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < p.here) c[e >> 2] |= (unsigned)q[e] << (8 * (e & 3));
    return c;
}
template <bool WHOLE>
__device__ __forceinline__ void store_codes(void* base, const Place<WHOLE>& p, u32x2 c) {
    unsigned char* q = reinterpret_cast<unsigned char*>(base) + p.at;
    if (p.here == 8) {
        reinterpret_cast<Loose8*>(q)->v = c;
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < p.here) q[e] = (unsigned char)(c[e >> 2] >> (8 * (e & 3)));
}
__device__ __forceinline__ void decode8(u32x2 c, float scale, float (&f)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[h], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[h], true);
        f[4 * h] = a[0] * scale;
        f[4 * h + 1] = a[1] * scale;
        f[4 * h + 2] = b[0] * scale;
        f[4 * h + 3] = b[1] * scale;
    }
}
// e4m3 code of y, 0 to 448 (and at most 2^-21 of that more): the value at or below y +
// u / 65536 of the step between codes there.  Below 2^-6 codes are 2^-9 apart, as they
// are from 2^-6 to 2^-5, to where such a y is moved.
__device__ __forceinline__ unsigned encode(float y, unsigned u) {
    const bool small = y < 0.015625f;
    const float z = small ? y + 0.015625f : y;
    return ((__float_as_uint(z) + (u << 4)) >> 20) - (small ? 968u : 960u);
}
// Largest over 32 lanes (a block's), the same in each of them.
template <int CTRL>
__device__ __forceinline__ unsigned dpp(unsigned v) {
    return (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
__device__ __forceinline__ unsigned block_max(unsigned v) {
    v = max(v, dpp<0xB1>(v));
    v = max(v, dpp<0x4E>(v));
    v = max(v, dpp<0x141>(v));
    v = max(v, dpp<0x140>(v));
    return max(v, (unsigned)__shfl_xor((int)v, 16, 64));
}
// A float without its sign, as a number: these compare as the floats do, infinity and
// NaN above the finite ones.
__device__ __forceinline__ unsigned magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }
constexpr unsigned kInfinity = 0x7f800000u, kLeast = 0x0da24260u;   // of 1e-30

// A block's largest finite magnitude, at least 1e-30; `odd`: the block holds others too.
__device__ __forceinline__ float largest(const float (&x)[8], bool& odd) {
    unsigned most = kLeast;
#pragma unroll
    for (int e = 0; e < 8; ++e) most = max(most, magnitude(x[e]));
    most = block_max(most);
    odd = most >= kInfinity;
    if (odd) {
        asm volatile("");   // (a branch that is hardly ever taken, not selects that always run)
        most = kLeast;
#pragma unroll
        for (int e = 0; e < 8; ++e) most = max(most, magnitude(x[e]) < kInfinity ? magnitude(x[e]) : 0u);
        most = block_max(most);
    }
    return __uint_as_float(most);
}

// sqrt(v): the hardware's reciprocal root and a Newton step, which leaves nearly every
// result rounded correctly at two thirds of sqrtf's instructions (arithmetic bounds the
// step in 8 bits; with the hardware's root alone more codes fell on the wrong side).
// For v from 2^-96 on: the hardware takes a subnormal v for 0, and further down v - r^2
// has no bits left.
__device__ __forceinline__ float root(float v) {
    const float s = __builtin_amdgcn_rsqf(v), r = v * s;
    return fmaf(fmaf(-r, r, v), 0.5f * s, r);
}
// The same for any v, 0 among them, through a multiple of v.  Infinite where v is (its
// update is then 0), and where it is NaN: of a NaN gradient m is NaN too, and else NaN is
// how codes hold infinity.
__device__ __forceinline__ float root_any(float v) {
    const bool small = v < 0x1p-96f;
    const float x = small ? v * 0x1p64f : v, s = fminf(__builtin_amdgcn_rsqf(x), 1e30f), r = x * s;
    const float q = fmaf(fmaf(-r, r, x), 0.5f * s, r) * (small ? 0x1p-32f : 1.f);
    return v < __uint_as_float(kInfinity) ? q : __uint_as_float(kInfinity);
}
// r = sqrt(v) of a thread's eight.  A second moment below 2^-96 is rare, but for zeros
// (weights that no gradient has met), and so is an infinite one, so the way for any v is
// behind a branch; an element's result is the same bits on either.
__device__ __forceinline__ void roots(const float (&v)[8], float (&r)[8]) {
    unsigned least = __float_as_uint(v[0]), most = least;
#pragma unroll
    for (int e = 1; e < 8; ++e) {
        least = min(least, __float_as_uint(v[e]));
        most = max(most, __float_as_uint(v[e]));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = root(v[e]);
    if (least < 0x0f800000u || most >= kInfinity) {   // (2^-96)
        asm volatile("");   // (not selects that always run)
        if (most == 0u) {   // 262 M weights from zero states without gradients: 597 us without this, 590 with
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] = 0.f;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] = root_any(v[e]);
        }
    }
}

// 448 / x likewise, for x from 1e-30 on (through x / 8: above 8.5e37 the reciprocal of x
// itself would be subnormal, which the hardware's is not).
__device__ __forceinline__ float codes_per(float x) {
    x *= 0.125f;
    const float s = __builtin_amdgcn_rcpf(x);
    return fmaf(fmaf(-x, s, 1.f), s, s) * 56.f;
}
__device__ __forceinline__ unsigned at_most_1(unsigned x) {   // (the compiler makes a test and a select of min)
    unsigned r;
    asm("v_min_u32 %0, 1, %1" : "=v"(r) : "v"(x));
    return r;
}

// One unit of a tensor, from element `base`.
template <int WT, int GT, int BITS, bool WHOLE>
__device__ __forceinline__ void step_unit(const AdamwArgs& a, const AdamwTensor& t, int64_t base, float gs) {
#pragma clang fp contract(off)
    // (the states are rounded after every operation, as the codes' rounding is a
    // function of their last bits)
    constexpr int U = (int)(kAdamwUnit / (256 * 8));
    float w[U][8], g[U][8], m[U][8], v[U][8];
    u32x2 mc[U], vc[U];
    float ms[U], vs[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Place<WHOLE> p(t, base, u * 2048 + (int)threadIdx.x * 8);
        load_part<WT>(t, t.w, t.w_ld, p, w[u]);
        load_part<GT>(t, t.g, t.g_ld, p, g[u]);
        if constexpr (BITS == 32) {
            if (p.here == 8) {
                load8<1>(reinterpret_cast<const float*>(t.m) + p.at, m[u]);
                load8<1>(reinterpret_cast<const float*>(t.v) + p.at, v[u]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    m[u][e] = e < p.here ? reinterpret_cast<const float*>(t.m)[p.at + e] : 0.f;
                    v[u][e] = e < p.here ? reinterpret_cast<const float*>(t.v)[p.at + e] : 0.f;
                }
            }
        } else {
            mc[u] = load_codes(t.m, p);
            vc[u] = load_codes(t.v, p);
            const int64_t block = p.at / kAdamwBlock;
            const bool there = WHOLE || block * kAdamwBlock < t.numel;
            ms[u] = there ? t.m_scale[block] : 0.f;
            vs[u] = there ? t.v_scale[block] : 0.f;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Place<WHOLE> p(t, base, u * 2048 + (int)threadIdx.x * 8);
        if constexpr (BITS == 8) {
            decode8(mc[u], ms[u], m[u]);
            decode8(vc[u], vs[u], v[u]);
        }
        float r[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = g[u][e] * gs;
            if constexpr (BITS == 8) v[u][e] = v[u][e] * v[u][e];
            m[u][e] = m[u][e] * a.beta1 + x * a.rest1;
            v[u][e] = v[u][e] * a.beta2 + (x * x) * a.rest2;
        }
        if constexpr (BITS == 8) roots(v[u], r);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (BITS == 32) r[e] = sqrtf(v[u][e]);
            const float up = m[u][e] * __builtin_amdgcn_rcpf(fmaf(r[e], a.root, a.eps));
            w[u][e] = fmaf(-a.rate, up, w[u][e] * a.keep);
        }
        store_part<WT>(t, t.w, t.w_ld, p, w[u]);
        if constexpr (BITS == 32) {
            if (p.here == 8) {
                store8<1>(reinterpret_cast<float*>(t.m) + p.at, m[u]);
                store8<1>(reinterpret_cast<float*>(t.v) + p.at, v[u]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < p.here) {
                        reinterpret_cast<float*>(t.m)[p.at + e] = m[u][e];
                        reinterpret_cast<float*>(t.v)[p.at + e] = v[u][e];
                    }
            }
        } else {
            bool m_odd, r_odd;
            const float m_max = largest(m[u], m_odd), r_max = largest(r, r_odd);
            const float mi = codes_per(m_max), ri = codes_per(r_max);
            unsigned cm[8], cv[8];
            const unsigned first = (uint32_t)(p.at >> 1) * 0xB890E049u + a.key;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                unsigned h = first + (unsigned)k * 0xB890E049u;   // of elements 2 k and 2 k + 1
                h = (h ^ (h >> 15)) * 0xB4A1B41Du;
                h = (h ^ (h >> 13)) * 0xF5BBB081u;
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    const int e = 2 * k + o;
                    const unsigned uv = o ? h >> 16 : h & 0xffffu;
                    const unsigned um = __builtin_amdgcn_perm(0u, uv, 0x0c0c0001u);   // its two bytes exchanged
                    cm[e] = encode(fabsf(m[u][e]) * mi, um) | ((__float_as_uint(m[u][e]) >> 24) & 128u);
                    cv[e] = max(encode(r[e] * ri, uv), at_most_1(__float_as_uint(r[e])));   // not 0 where r is not
                }
            }
            if (m_odd || r_odd) {
                asm volatile("");   // (as above)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (magnitude(m[u][e]) >= kInfinity) cm[e] = 127u;
                    if (magnitude(r[e]) >= kInfinity) cv[e] = 127u;
                }
            }
            u32x2 mo, vo;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                mo[k] = cm[4 * k] | cm[4 * k + 1] << 8 | cm[4 * k + 2] << 16 | cm[4 * k + 3] << 24;
                vo[k] = cv[4 * k] | cv[4 * k + 1] << 8 | cv[4 * k + 2] << 16 | cv[4 * k + 3] << 24;
            }
            store_codes(t.m, p, mo);
            store_codes(t.v, p, vo);
            if (p.here > 0 && (threadIdx.x & 31) == 0) {
                const int64_t block = p.at / kAdamwBlock;
                t.m_scale[block] = m_max * (1.f / 448.f);
                t.v_scale[block] = r_max * (1.f / 448.f);
            }
        }
    }
}

template <int WT, int GT, int BITS>
__global__ __launch_bounds__(256) void adamw_kernel(const AdamwArgs a) {
    const float gs = a.grad_scale != nullptr ? *a.grad_scale : 1.f;
    int id = 0;
    for (uint32_t unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
        // the last tensor whose first unit is at or before this one
        if (id + 1 < a.n && a.t[id + 1].first <= unit) {
            int lo = id + 1, hi = a.n;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (a.t[mid].first <= unit) lo = mid;
                else hi = mid;
            }
            id = lo;
        }
        id = __builtin_amdgcn_readfirstlane(id);
        const AdamwTensor& t = a.t[id];
        const int64_t base = (int64_t)(unit - t.first) * kAdamwUnit;
        if (t.cols == 0 && base + kAdamwUnit <= t.numel) step_unit<WT, GT, BITS, true>(a, t, base, gs);
        else step_unit<WT, GT, BITS, false>(a, t, base, gs);
    }
}

template <int WT, int GT>
void launch(const AdamwArgs& a, dim3 grid, hipStream_t s) {
    if (a.bits == 8) hipLaunchKernelGGL((adamw_kernel<WT, GT, 8>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((adamw_kernel<WT, GT, 32>), grid, dim3(256), 0, s, a);
}

}  // namespace

hipError_t launch_adamw(const AdamwArgs& a, hipStream_t s) {
    static const int cus = [] { const int c = device_cus(); return c >= 8 ? std::min(c, 512) : 256; }();
    const dim3 grid(std::min<uint32_t>(a.units, (uint32_t)cus * 16));
    if (a.w_dtype == 0) {
        if (a.g_dtype == 0) launch<0, 0>(a, grid, s);
        else launch<0, 1>(a, grid, s);
    } else {
        if (a.g_dtype == 0) launch<1, 0>(a, grid, s);
        else launch<1, 1>(a, grid, s);
    }
    return hipGetLastError();
}

}  // namespace himuon
