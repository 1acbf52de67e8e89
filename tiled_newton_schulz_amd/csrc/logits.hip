// Losses over rows of logits on gfx950: distillation from a teacher's top
// logits and log probabilities of given tokens (include/himuon.h has the
// formulas).  With s = z / temperature and m = max s, a row needs
//     S = sum exp(s - m),  lse = m + log S,  E = sum exp(s - m) (s - m),
//     entropy = log S - E / S,
// all in fp32.  One workgroup per row: a pass for m, one for the sums.

#include "device_util.h"
#include "logits.h"

namespace himuon {
namespace {

constexpr int kThreads = 256;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float load_z(const LogitsArgs& a, int64_t row, int64_t col) {
    const int64_t o = row * a.z_ld + col;
    return a.dtype == 0 ? bf2f(reinterpret_cast<const unsigned short*>(a.z)[o])
                        : reinterpret_cast<const float*>(a.z)[o];
}
__device__ __forceinline__ void store_dz(const LogitsArgs& a, int64_t row, int64_t col, float v) {
    const int64_t o = row * a.dz_ld + col;
    if (a.dtype == 0) reinterpret_cast<unsigned short*>(a.dz)[o] = f2bf(v);
    else reinterpret_cast<float*>(a.dz)[o] = v;
}
// Id i of an array, -1 if it lies outside [0, V).
__device__ __forceinline__ int load_id(const void* p, int idx64, int64_t i, int cols) {
    const int64_t v = idx64 ? reinterpret_cast<const int64_t*>(p)[i] : reinterpret_cast<const int32_t*>(p)[i];
    return v >= 0 && v < cols ? (int)v : -1;
}


template <typename F>
__device__ __forceinline__ float block_reduce(float v, float* red, F f) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v = f(v, __shfl_xor(v, o, 64));
    __syncthreads();   // red may still be read from the last use
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float r = red[0];
    for (int i = 1; i < (int)(blockDim.x >> 6); ++i) r = f(r, red[i]);
    return r;
}
__device__ __forceinline__ float block_sum(float v, float* red) {
    return block_reduce(v, red, [](float x, float y) { return x + y; });
}
__device__ __forceinline__ float block_max(float v, float* red) {
    return block_reduce(v, red, [](float x, float y) { return fmaxf(x, y); });
}

// log sum exp of a row as hi + lo: hi is its fp32 value and lo what that
// rounding lost, which counts where |m| is large (a row masked by the lowest
// value would lose log S altogether).
struct Lse {
    float hi, lo;
};
__device__ __forceinline__ Lse make_lse(float m, float S) {
    if (S == 0.f) return {kNegInf, 0.f};   // -inf only
    const float l = __logf(S), hi = m + l;
    // |m| >= |l| or not: the exact rest of the sum either way
    const float lo = fabsf(m) >= fabsf(l) ? (m - hi) + l : (l - hi) + m;
    return {hi, lo};
}
__device__ __forceinline__ float log_q_of(float s, Lse l) {
    if (s == kNegInf && l.hi == l.hi) return kNegInf;
    return (s - l.hi) - l.lo;
}

struct RowStats {
    Lse lse;
    float entropy;
};

__device__ __forceinline__ void put_lse(const LogitsArgs& a, int64_t row, Lse l) {
    a.lse[2 * row] = l.hi;
    a.lse[2 * row + 1] = l.lo;
}
__device__ __forceinline__ Lse get_lse(const LogitsArgs& a, int64_t row) { return {a.lse[2 * row], a.lse[2 * row + 1]}; }

// lse and entropy of a row.  NaN: fmaxf passes over it, the sum takes it in.
// A maximum of +inf gives inf - inf = NaN in the sum, one of -inf leaves
// nothing (lse -inf, entropy 0).
__device__ __forceinline__ RowStats row_stats(const LogitsArgs& a, int64_t row, float* red) {
    float m = kNegInf;
    for (int v = threadIdx.x; v < a.cols; v += kThreads) m = fmaxf(m, load_z(a, row, v) * a.inv_temp);
    m = block_max(m, red);
    float s = 0.f, e = 0.f;
    for (int v = threadIdx.x; v < a.cols; v += kThreads) {
        const float z = load_z(a, row, v) * a.inv_temp;
        if (z == kNegInf) continue;
        const float d = z - m, x = __expf(d);
        s += x;
        e += x > 0.f ? x * d : 0.f;
    }
    s = block_sum(s, red);
    e = block_sum(e, red);
    return {make_lse(m, s), s == 0.f ? 0.f : __logf(s) - e / s};
}

// ---- distillation ------------------------------------------------------------

// The teacher's entries of a row: ids (-1: absent) and probabilities in LDS.
struct Teacher {
    int* id;
    float* p;
    float P;       // their sum
    float plogp;   // sum p log p
    bool live;     // some entry has p > 0 (or is NaN)
};

__device__ __forceinline__ Teacher load_teacher(const LogitsArgs& a, int64_t row, int* id, float* p, float* red) {
    const float it = a.normalize ? a.inv_temp : 1.f;
    float m = kNegInf, some = 0.f;
    for (int j = threadIdx.x; j < a.k; j += kThreads) {
        id[j] = load_id(a.idx, a.idx64, row * a.k + j, a.cols);
        const float t = id[j] >= 0 ? a.t[row * a.t_ld + j] * it : kNegInf;
        p[j] = t;
        m = fmaxf(m, t);
        if (!(t == kNegInf)) some = 1.f;
    }
    Teacher r{id, p, 0.f, 0.f, block_max(some, red) > 0.f};
    if (!r.live) return r;
    m = a.normalize ? block_max(m, red) : 0.f;
    float S = 0.f;
    for (int j = threadIdx.x; j < a.k; j += kThreads) S += p[j] == kNegInf ? 0.f : __expf(p[j] - m);
    S = block_sum(S, red);
    const float l = a.normalize ? m + __logf(S) : 0.f;
    float sum = 0.f, plogp = 0.f;
    for (int j = threadIdx.x; j < a.k; j += kThreads) {
        const float lp = p[j] - l;
        const float q = p[j] == kNegInf ? 0.f : __expf(lp);
        sum += q;
        plogp += q == 0.f ? 0.f : q * lp;
        p[j] = q;
    }
    r.P = block_sum(sum, red);
    r.plogp = block_sum(plogp, red);   // its barriers also publish id and p
    return r;
}

__device__ __forceinline__ void zero_row(const LogitsArgs& a, int64_t row) {
    for (int v = threadIdx.x; v < a.cols; v += kThreads) store_dz(a, row, v, 0.f);
}

// Teacher probability of the row's entries that hold the same id as entry j
// (usually entry j alone), in the entries' order.
__device__ __forceinline__ float mass_at(const Teacher& t, int k, int j) {
    float sum = 0.f;
    for (int i = 0; i < k; ++i) sum += t.id[i] == t.id[j] ? t.p[i] : 0.f;
    return sum;
}

// dz = c (P q - p), q from lse.  The ids of entries are written after the
// others, from logits taken before any gradient is stored (dz may be z); equal
// ids write the same value.
__device__ __forceinline__ void distill_grad_row(const LogitsArgs& a, int64_t row, const Teacher& t, Lse lse, float w) {
    const float c = w * a.inv_temp;
    float fix[kMaxEntries / kThreads];
    auto q_of = [&](int64_t v) { return __expf(log_q_of(load_z(a, row, v) * a.inv_temp, lse)); };
#pragma unroll
    for (int u = 0; u < kMaxEntries / kThreads; ++u) {
        const int j = u * kThreads + threadIdx.x;
        fix[u] = j < a.k && t.id[j] >= 0 ? c * (t.P * q_of(t.id[j]) - mass_at(t, a.k, j)) : 0.f;
    }
    __syncthreads();
    for (int v = threadIdx.x; v < a.cols; v += kThreads) store_dz(a, row, v, c * (t.P * q_of(v)));
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMaxEntries / kThreads; ++u) {
        const int j = u * kThreads + threadIdx.x;
        if (j < a.k && t.id[j] >= 0) store_dz(a, row, t.id[j], fix[u]);
    }
}

__global__ __launch_bounds__(kThreads) void distill_kernel(const LogitsArgs a) {
    __shared__ float red[kThreads / 64];
    __shared__ int id[kMaxEntries];
    __shared__ float p[kMaxEntries];
    const int64_t row = blockIdx.x;
    const float w = a.weight ? a.weight[row] : 1.f;
    Teacher t{};
    if (w != 0.f) t = load_teacher(a, row, id, p, red);
    if (!t.live) {
        if (threadIdx.x == 0) {
            a.loss[row] = 0.f;
            if (a.lse) put_lse(a, row, {0.f, 0.f});
        }
        if (a.dz) zero_row(a, row);
        return;
    }
    const RowStats r = row_stats(a, row, red);
    float cross = 0.f;
    for (int j = threadIdx.x; j < a.k; j += kThreads) {
        if (t.p[j] == 0.f) continue;
        cross += t.p[j] * log_q_of(load_z(a, row, t.id[j]) * a.inv_temp, r.lse);
    }
    cross = block_sum(cross, red);
    if (threadIdx.x == 0) {
        a.loss[row] = w * (t.plogp - cross);
        if (a.lse) put_lse(a, row, r.lse);
    }
    if (a.dz) distill_grad_row(a, row, t, r.lse, w);
}

__global__ __launch_bounds__(kThreads) void distill_grad_kernel(const LogitsArgs a) {
    __shared__ float red[kThreads / 64];
    __shared__ int id[kMaxEntries];
    __shared__ float p[kMaxEntries];
    const int64_t row = blockIdx.x;
    const float w = a.weight[row];
    Teacher t{};
    if (w != 0.f) t = load_teacher(a, row, id, p, red);
    if (t.live) distill_grad_row(a, row, t, get_lse(a, row), w);
    else zero_row(a, row);
}

// ---- log probabilities of given tokens -----------------------------------------

// Order of the alternatives: larger logit first (NaN as -inf), equal ones by
// the lower id.  0 is below every key of an element.
__device__ __forceinline__ uint64_t rank_key(float z, int id) {
    z = z != z ? kNegInf : z + 0.f;   // -0 as +0
    const uint32_t u = __float_as_uint(z);
    const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return ((uint64_t)o << 32) | (uint32_t)~id;
}

__device__ __forceinline__ uint64_t block_max_key(uint64_t v, uint64_t* red) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
        const uint64_t w = __shfl_xor((unsigned long long)v, o, 64);
        v = v > w ? v : w;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    uint64_t r = red[0];
    for (int i = 1; i < kThreads / 64; ++i) r = r > red[i] ? r : red[i];
    return r;
}

__global__ __launch_bounds__(kThreads) void logprobs_kernel(const LogitsArgs a) {
    __shared__ float red[kThreads / 64];
    __shared__ uint64_t redk[kThreads / 64];
    const int64_t row = blockIdx.x;
    const int tok = a.tokens ? load_id(a.tokens, a.idx64, row, a.cols) : 0;
    if (tok < 0) {
        if (threadIdx.x == 0) {
            if (a.logp) a.logp[row] = 0.f;
            if (a.entropy) a.entropy[row] = 0.f;
            if (a.lse) put_lse(a, row, {0.f, 0.f});
        }
        for (int j = threadIdx.x; j < a.top; j += kThreads) {
            a.top_idx[row * a.top + j] = -1;
            a.top_logp[row * a.top + j] = kNegInf;
        }
        return;
    }
    const RowStats r = row_stats(a, row, red);
    auto log_q = [&](int v) { return log_q_of(load_z(a, row, v) * a.inv_temp, r.lse); };
    if (threadIdx.x == 0) {
        if (a.logp) a.logp[row] = log_q(tok);
        if (a.entropy) a.entropy[row] = r.entropy;
        if (a.lse) put_lse(a, row, r.lse);
    }
    uint64_t below = ~0ull;
    for (int j = 0; j < a.top; ++j) {   // the largest key below the last one taken
        uint64_t best = 0;
        for (int v = threadIdx.x; v < a.cols; v += kThreads) {
            const uint64_t key = rank_key(load_z(a, row, v), v);
            if (key < below && key > best) best = key;
        }
        below = block_max_key(best, redk);
        if (threadIdx.x == 0) {
            const int v = (int)~(uint32_t)below;
            a.top_idx[row * a.top + j] = v;
            a.top_logp[row * a.top + j] = log_q(v);
        }
    }
}

__global__ __launch_bounds__(kThreads) void logprobs_grad_kernel(const LogitsArgs a) {
    const int64_t row = blockIdx.x;
    const int tok = a.tokens ? load_id(a.tokens, a.idx64, row, a.cols) : -1;
    float gl = a.g_logp ? a.g_logp[row] * a.inv_temp : 0.f;
    float gh = a.g_entropy ? a.g_entropy[row] * a.inv_temp : 0.f;
    if (a.tokens && tok < 0) gl = gh = 0.f;
    if (gl == 0.f && gh == 0.f) {
        zero_row(a, row);
        return;
    }
    const Lse lse = get_lse(a, row);
    const float H = gh != 0.f ? a.entropy[row] : 0.f;
    for (int v = threadIdx.x; v < a.cols; v += kThreads) {
        const float lq = log_q_of(load_z(a, row, v) * a.inv_temp, lse), q = __expf(lq);
        float g = v == tok ? gl * (1.f - q) : -gl * q;
        if (gh != 0.f && q != 0.f) g -= gh * (q * (lq + H));
        store_dz(a, row, v, g);
    }
}

}  // namespace

hipError_t launch_distill(const LogitsArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(distill_kernel, dim3(a.rows), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}
hipError_t launch_distill_grad(const LogitsArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(distill_grad_kernel, dim3(a.rows), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}
hipError_t launch_logprobs(const LogitsArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(logprobs_kernel, dim3(a.rows), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}
hipError_t launch_logprobs_grad(const LogitsArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(logprobs_grad_kernel, dim3(a.rows), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace himuon
