// Losses over rows of logits on gfx950: distillation from a teacher's top
// logits and log probabilities of given tokens (include/himuon.h has the
// formulas).  With s = z / temperature and m = max z, a row needs
//     S = sum exp(s - s_m),  E = sum exp(s - s_m) (z - m),
//     lse = s_m + log S,     entropy = log S - E / (S temperature),
// all in fp32.  The differences are taken before they are scaled, so a row
// masked by the type's lowest value loses nothing; a gradient from a known lse
// takes s rounded as the lse has it, and the differences after (Softmax).
//
// The work is a stream over the logits (HBM bound, a read for a forward pass, a
// read and a write for a gradient), so rows move in 16-byte chunks and stay
// packed in registers between the maximum and the sums:
// - forward passes cut a row into segments of up to 256 x 8 chunks, one
//   workgroup each (few rows: smaller segments, so that the chip is filled), and
//   a second launch joins them; a row of one segment ends in the first;
// - the distillation loss with its gradient keeps the whole row in the
//   registers of one workgroup: one read and one write in all;
// - gradients from a known lse are element-wise, in segments.
// Rows may start at any alignment: a row's chunks are those of the 16-byte grid,
// and the elements of its first and last chunk are moved one by one.

#include <algorithm>
#include <type_traits>

#include "device_util.h"
#include "logits.h"

namespace himuon {
namespace {

constexpr int kThreads = 256;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float ln_hw(float x) { return __builtin_amdgcn_logf(x) * kLn2; }

// ---- rows in 16-byte chunks ------------------------------------------------
template <int DT> constexpr int kEpc = DT == 0 ? 8 : 4;   // elements of a chunk
// A chunk past every row: with at most 2^29 columns, neither its first column
// nor the one after its last overflows an int.
constexpr int kNoChunk = (1 << 27) + 8;
static_assert(int64_t(kNoChunk) * 4 > (1 << 29) + 4 && int64_t(kNoChunk + 1) * 8 < INT32_MAX, "kNoChunk");

// Element e of a chunk.
template <int DT>
__device__ __forceinline__ float elem(const u32x4& c, int e) {
    if constexpr (DT == 0) return (e & 1) ? hi_f(c[e >> 1]) : lo_f(c[e >> 1]);
    else return __uint_as_float(c[e]);
}
template <int DT>
__device__ __forceinline__ u32x4 pack(const float (&v)[kEpc<DT>]) {
    u32x4 c;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = DT == 0 ? pack2(v[(2 * i) % kEpc<DT>], v[(2 * i + 1) % kEpc<DT>]) : __float_as_uint(v[i]);
    return c;
}

// FLUSH: the caller's rows all start and end on the grid.
template <int DT, bool FLUSH>
struct Row {
    static constexpr int EPC = kEpc<DT>, ES = 16 / EPC;
    char* base;    // 16-byte aligned, at or before the row's first element
    int mis;       // elements from there to it
    int cols;
    __device__ __forceinline__ Row(const void* p, int64_t ld, int64_t row, int n) : cols(n) {
        const uint64_t at = reinterpret_cast<uint64_t>(p) + (uint64_t)(row * ld) * ES;
        mis = FLUSH ? 0 : (int)(at & 15) / ES;
        base = reinterpret_cast<char*>(at & ~uint64_t(15));
    }
    __device__ __forceinline__ int chunks() const { return (mis + cols + EPC - 1) / EPC; }
    __device__ __forceinline__ int first(int c) const { return c * EPC - mis; }   // column of element 0
    __device__ __forceinline__ bool whole(int c) const {
        return FLUSH ? c * EPC < cols : first(c) >= 0 && first(c) + EPC <= cols;
    }
    // byte offsets fit 32 bits (the host allows 2^29 columns)
    __device__ __forceinline__ char* at(int c) const { return base + (uint32_t)c * 16u; }
    // Chunk c; what lies outside the row is -inf.  (The element loops of this
    // and of store() are kept rolled: they run for a row's two ends only.)
    __device__ __forceinline__ u32x4 load(int c) const {
        if (whole(c)) return *reinterpret_cast<const u32x4*>(at(c));
        constexpr uint64_t kFill = DT == 0 ? 0xff80ff80ff80ff80ull : 0xff800000ff800000ull;
        uint64_t w[2] = {kFill, kFill};
        const int v0 = first(c);
        if (!FLUSH && v0 < cols) {
#pragma unroll 1
            for (int e = max(0, -v0); e < min(EPC, cols - v0); ++e) {
                const char* p = base + ((int64_t)c * EPC + e) * ES;
                const uint64_t x = DT == 0 ? *reinterpret_cast<const unsigned short*>(p)
                                           : *reinterpret_cast<const unsigned*>(p);
                const int at = 8 * ES * (e % (EPC / 2));
                const uint64_t keep = ~((DT == 0 ? 0xffffull : 0xffffffffull) << at);
                if (e < EPC / 2) w[0] = (w[0] & keep) | x << at;
                else w[1] = (w[1] & keep) | x << at;
            }
        }
        return u32x4{(unsigned)w[0], (unsigned)(w[0] >> 32), (unsigned)w[1], (unsigned)(w[1] >> 32)};
    }
    __device__ __forceinline__ void store_elem(int col, float v) const {
        char* p = base + ((int64_t)mis + col) * ES;
        if constexpr (DT == 0) *reinterpret_cast<unsigned short*>(p) = f2bf(v);
        else *reinterpret_cast<float*>(p) = v;
    }
    __device__ __forceinline__ float load_elem(int col) const {
        const char* p = base + ((int64_t)mis + col) * ES;
        if constexpr (DT == 0) return bf2f(*reinterpret_cast<const unsigned short*>(p));
        else return *reinterpret_cast<const float*>(p);
    }
    // Elements of chunk c of a row that starts `from` elements into its chunk
    // grid (the row the values were read from; the same grid when equal).
    __device__ __forceinline__ void store(int c, const u32x4& v, int from) const {
        const int v0 = c * EPC - from;
        if (mis == from && whole(c)) {
            *reinterpret_cast<u32x4*>(at(c)) = v;
            return;
        }
        if (FLUSH) return;
        const uint64_t w0 = v[0] | (uint64_t)v[1] << 32, w1 = v[2] | (uint64_t)v[3] << 32;
#pragma unroll 1
        for (int e = max(0, -v0); e < min(EPC, cols - v0); ++e) {
            const uint64_t x = (e < EPC / 2 ? w0 : w1) >> (8 * ES * (e % (EPC / 2)));
            char* p = base + ((int64_t)mis + v0 + e) * ES;
            if constexpr (DT == 0) *reinterpret_cast<unsigned short*>(p) = (unsigned short)x;
            else *reinterpret_cast<unsigned*>(p) = (unsigned)x;
        }
    }
};

// Makes chunks opaque to the optimiser, which would otherwise keep them unpacked
// in registers from one pass over them to the next.
template <int U>
__device__ __forceinline__ void stay_packed(u32x4 (&r)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) asm volatile("" : "+v"(r[u]));
}

// Id i of an array, -1 if it lies outside [0, V).
__device__ __forceinline__ int load_id(const void* p, int idx64, int64_t i, int cols) {
    const int64_t v = idx64 ? reinterpret_cast<const int64_t*>(p)[i] : reinterpret_cast<const int32_t*>(p)[i];
    return v >= 0 && v < cols ? (int)v : -1;
}

// ---- reductions ----------------------------------------------------------------
// Over a wave, in a fixed order (lanes without a source take `none`).
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float none, float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(none), __float_as_int(v), CTRL, ROWS, 0xf, false));
}
template <typename F>
__device__ __forceinline__ float wave_reduce(float v, float none, F f) {
    v = f(v, dpp<0x111, 0xf>(none, v));   // row_shr 1, 2, 4, 8
    v = f(v, dpp<0x112, 0xf>(none, v));
    v = f(v, dpp<0x114, 0xf>(none, v));
    v = f(v, dpp<0x118, 0xf>(none, v));
    v = f(v, dpp<0x142, 0xa>(none, v));   // row_bcast 15, 31
    v = f(v, dpp<0x143, 0xc>(none, v));
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ float wsum(float v) {
    return wave_reduce(v, 0.f, [](float x, float y) { return x + y; });
}
__device__ __forceinline__ float wmax(float v) {
    return wave_reduce(v, kNegInf, [](float x, float y) { return fmaxf(x, y); });
}

// ---- statistics of a set of logits --------------------------------------------
struct Stats {
    float m, s, e;   // largest logit (NaN passed over), S and E relative to it
};
constexpr Stats kEmpty = {kNegInf, 0.f, 0.f};
// c: log2(e) / temperature.  A NaN reaches s and with it every result of the
// row, and so does +inf (inf - inf); sets of -inf only have s = e = 0.
__device__ __forceinline__ Stats join(Stats a, Stats b, float c) {
    const float m = fmaxf(a.m, b.m);
    if (m == kNegInf) return {m, a.s + b.s, 0.f};
    const float da = a.m - m, db = b.m - m;
    const float ea = exp2_hw(da * c), eb = exp2_hw(db * c);
    Stats r;
    r.m = m;
    r.s = a.s * ea + b.s * eb;
    r.e = ea * (a.e + fmaxf(da, -1e30f) * a.s) + eb * (b.e + fmaxf(db, -1e30f) * b.s);
    return r;
}

// log sum exp of a row as hi + lo: hi is its fp32 value and lo what that
// rounding lost, which counts where it is large (a row masked by the lowest
// value would lose log S altogether).  The largest s enters as the rounded
// product, held to fp32's range: where it reaches +-kFltMax, hi does not say
// which logit was the largest (Softmax::far).
constexpr float kFltMax = 3.40282346638528859812e38f;
struct Lse {
    float hi, lo;
};
__device__ __forceinline__ Lse make_lse(const Stats& st, float inv_temp) {
#pragma clang fp contract(off)
    if (st.s == 0.f) return {kNegInf, 0.f};   // -inf only
    const float m = fminf(fmaxf(st.m * inv_temp, -kFltMax), kFltMax), l = ln_hw(st.s), hi = m + l;
    const float lo = fabsf(m) >= fabsf(l) ? (m - hi) + l : (l - hi) + m;
    return {hi, lo};
}
__device__ __forceinline__ float entropy_of(const Stats& st, float inv_temp) {
    return st.s == 0.f ? 0.f : ln_hw(st.s) - inv_temp * (st.e / st.s);
}
// log q of a logit of a row with these statistics.
__device__ __forceinline__ float log_q(float z, float inv_temp, const Stats& st) {
    if (z == kNegInf && st.s == st.s) return kNegInf;
    return (z - st.m) * inv_temp - ln_hw(st.s);
}
// q and log q of the logits of a row from its lse alone:
//     d = z mul - sub,   log q = slope d - lo,   q = exp2(d k - lo log2 e).
// With mul = inv_temp, sub = hi the product is rounded before hi is taken off, as
// make_lse rounds the largest one (unrounded it would be off from it by half a
// unit of s, 32 where |s| is 1e9, whatever the logits' differences are).  A far
// row takes m, its largest logit, in hi's place: mul = 1, sub = m.  A row of -inf
// only takes sub = 0 and has q = 0.
struct Softmax {
    float mul, sub, slope, k, lo, neg_lo2;
    __device__ __forceinline__ static bool far(Lse l) { return fabsf(l.hi) == kFltMax; }
    __device__ __forceinline__ Softmax(float inv_temp, Lse l)
        : mul(inv_temp), sub(l.hi == kNegInf ? 0.f : l.hi), slope(1.f), k(kLog2e), lo(l.lo), neg_lo2(-l.lo * kLog2e) {}
    __device__ __forceinline__ void set_far(float inv_temp, float m) {
        mul = 1.f;
        sub = m;
        slope = inv_temp;
        k = inv_temp * kLog2e;
    }
    __device__ __forceinline__ float diff(float z) const {
#pragma clang fp contract(off)
        return z * mul - sub;
    }
    __device__ __forceinline__ float at(float d) const { return exp2_hw(__builtin_fmaf(d, k, neg_lo2)); }
    __device__ __forceinline__ float operator()(float z) const { return at(diff(z)); }
};

__device__ __forceinline__ void put_lse(const LogitsArgs& a, int64_t row, Lse l) {
    if (a.lse == nullptr) return;
    a.lse[2 * row] = l.hi;
    a.lse[2 * row + 1] = l.lo;
}
__device__ __forceinline__ Lse get_lse(const LogitsArgs& a, int64_t row) {
    return {a.lse[2 * row], a.lse[2 * row + 1]};
}

// Largest element of each chunk, and of all.
template <int DT, int U>
__device__ __forceinline__ float chunk_max(u32x4 (&r)[U], float (&cm)[U]) {
    float m = kNegInf;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        cm[u] = kNegInf;
#pragma unroll
        for (int e = 0; e < kEpc<DT>; ++e) cm[u] = fmaxf(cm[u], elem<DT>(r[u], e));
        m = fmaxf(m, cm[u]);
    }
    stay_packed(r);
    return m;
}
// Statistics of the chunks a wave holds, m their largest element.
template <int DT, int U>
__device__ __forceinline__ Stats wave_stats(u32x4 (&r)[U], float m, float c, bool want_e) {
    const float ref = m == kNegInf ? 0.f : m;
    float s = 0.f, t = 0.f;
    if (want_e) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < kEpc<DT>; ++e) {
                const float d = elem<DT>(r[u], e) - ref, x = exp2_hw(d * c);
                s += x;
                t = __builtin_fmaf(x, fmaxf(d, -1e30f), t);
            }
        t = wsum(t);
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < kEpc<DT>; ++e) s += exp2_hw((elem<DT>(r[u], e) - ref) * c);
    }
    stay_packed(r);
    return {m, wsum(s), t};
}

// ---- the teacher's entries ---------------------------------------------------------
// Sums over the entries of a row, with u_j = t_j / temperature (normalize) or
// t_j, M the largest u (normalize) or 0, e_j = exp(u_j - M), and b_j the log
// probability of the id under the student up to a constant B:
//     S = sum e,  E = sum e (u - M),  G = sum e b.
// Then P = 1 or S, p_j = e_j / S or e_j, and
//     loss = sum p log p - sum p log q = (E / S - log S - G / S) - P B   (or E - G - P B).
struct Entry {
    int id;      // -1: absent
    float u;
    float z;     // the student's logit at the id
};
template <int DT, bool FL>
__device__ __forceinline__ Entry load_entry(const LogitsArgs& a, const Row<DT, FL>& z, int64_t row, int j) {
    Entry x = {-1, kNegInf, 0.f};
    if (j >= a.k) return x;
    x.id = load_id(a.idx, a.idx64, row * a.k + j, a.cols);
    if (x.id < 0) return x;
    const float t = a.t[row * a.t_ld + j];
    x.u = a.normalize ? t * a.inv_temp : t;
    // no probability in fp32: as if it were -inf (a row of such entries counts nothing)
    if (!a.normalize && exp2_hw(t * kLog2e) == 0.f) x.u = kNegInf;
    x.z = z.load_elem(x.id);
    return x;
}

struct TeacherSums {
    float P, scale, loss;   // p_j = e_j scale; loss without P B
};
__device__ __forceinline__ TeacherSums teacher_sums(const LogitsArgs& a, float S, float E, float G) {
    if (a.normalize) {
        const float r = 1.f / S;
        return {1.f, r, E * r - ln_hw(S) - G * r};
    }
    return {S, 1.f, E - G};
}

// Teacher probability of the row's entries that hold entry j's id (usually j
// alone), in the entries' order.
__device__ __forceinline__ float mass_at(const int* id, const float* p, int k, int mine) {
    float sum = 0.f;
    for (int i = 0; i < k; ++i) sum += id[i] == mine ? p[i] : 0.f;
    return sum;
}

// Joins the waves' values of several reductions of a workgroup of NT threads in
// one go (v[i] holds the wave's; afterwards all threads hold the workgroup's).
template <int NT, int N, typename F>
__device__ __forceinline__ void block_join(float (&v)[N], float (*red)[N], float none, F f) {
    __syncthreads();   // red may still be read from the last use
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) red[threadIdx.x >> 6][i] = v[i];
    __syncthreads();
    const int w = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_reduce(w < NT / 64 ? red[w][i] : none, none, f);
}
struct Max {
    __device__ __forceinline__ float operator()(float x, float y) const { return fmaxf(x, y); }
};
struct Sum {
    __device__ __forceinline__ float operator()(float x, float y) const { return x + y; }
};

// Loss of a row whose statistics are known.  NT 256: a workgroup; 64: a wave (k <= 64).
template <int DT, bool FL, int NT>
__device__ __forceinline__ void distill_loss(const LogitsArgs& a, int64_t row, const Stats& st, Lse l) {
    constexpr int KE = NT == 64 ? 1 : kMaxEntries / NT;
    const int tid = threadIdx.x % NT;
    const Row<DT, FL> z(a.z, a.z_ld, row, a.cols);
    Entry x[KE];
    float mx[2] = {kNegInf, 0.f};
#pragma unroll
    for (int i = 0; i < KE; ++i) {
        x[i] = load_entry<DT, FL>(a, z, row, i * NT + tid);
        mx[0] = fmaxf(mx[0], x[i].u);
        if (!(x[i].u == kNegInf)) mx[1] = 1.f;
    }
    mx[0] = wmax(mx[0]);
    mx[1] = wmax(mx[1]);
    if constexpr (NT != 64) {
        __shared__ float red[NT / 64][2];
        block_join<NT>(mx, red, kNegInf, Max());
    }
    if (mx[1] == 0.f) {   // no entry counts
        if (tid == 0) {
            a.loss[row] = 0.f;
            put_lse(a, row, {0.f, 0.f});
        }
        return;
    }
    const float M = a.normalize ? mx[0] : 0.f;
    float sum[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < KE; ++i) {
        if (x[i].u == kNegInf) continue;
        const float e = exp2_hw((x[i].u - M) * kLog2e);
        if (e == 0.f) continue;   // adds nothing, whatever the student has there
        sum[0] += e;
        sum[1] += e * (x[i].u - M);
        sum[2] += e * log_q(x[i].z, a.inv_temp, st);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) sum[i] = wsum(sum[i]);
    if constexpr (NT != 64) {
        __shared__ float red[NT / 64][3];
        block_join<NT>(sum, red, 0.f, Sum());
    }
    if (tid == 0) {
        a.loss[row] = (a.weight ? a.weight[row] : 1.f) * teacher_sums(a, sum[0], sum[1], sum[2]).loss;
        put_lse(a, row, l);
    }
}

// ---- alternatives -----------------------------------------------------------------
// Order: larger logit first (NaN as -inf), equal ones by the lower id.  0 is
// below every key of an element.
__device__ __forceinline__ uint64_t rank_key(float z, int id) {
    z = z != z ? kNegInf : z + 0.f;   // -0 as +0
    const uint32_t u = __float_as_uint(z);
    const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return ((uint64_t)o << 32) | (uint32_t)~id;
}
__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ int key_id(uint64_t key) { return (int)~(uint32_t)key; }

constexpr int kCand = 1024, kChunkCand = 512;
struct TopShared {
    uint64_t cand[kCand];
    uint64_t best[4];
    int chunk[kChunkCand];
    float low[4];
    int ties[4];
    int count, chunks;
};

// Ranks the n candidates among each other; emit(rank, key) for the first `top`.
template <typename Emit>
__device__ __forceinline__ void rank_candidates(const TopShared& sh, int n, int top, Emit emit) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t key = sh.cand[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += sh.cand[j] > key ? 1 : 0;
        if (rank < top) emit(rank, key);
    }
}
// Searches each rank in turn: the largest key below the last one.  all(f) calls
// f(key) on every element of this thread.  Slow, and rare: in bf16, 1024 rows of
// 65536 that ascend take 1.5 ms with 20 alternatives and 4.6 ms with 64, against
// 58 and 62 us of rows in any order (fp32: 0.5 ms either way, against 66 and 87).
template <typename All, typename Emit>
__device__ __forceinline__ void search_ranks(TopShared& sh, int top, All all, Emit emit) {
    uint64_t below = ~0ull;
    for (int j = 0; j < top; ++j) {
        uint64_t best = 0;
        all([&](uint64_t key) {
            if (key < below && key > best) best = key;
        });
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) {
            const uint64_t w = __shfl_xor((unsigned long long)best, o, 64);
            best = best > w ? best : w;
        }
        __syncthreads();
        if ((threadIdx.x & 63) == 0) sh.best[threadIdx.x >> 6] = best;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) best = best > sh.best[i] ? best : sh.best[i];
        if (threadIdx.x == 0) emit(j, best);
        below = best;
    }
}

// The `top` largest elements of a segment (cn chunks from c0 on, chunk
// u * 256 + thread in this thread, cm its largest element): emit(rank, key).
//
// A bound first: every full wave takes the m-th largest of its lanes' maxima,
// m = ceil(top / full waves), and at least `top` elements reach the smallest of
// these.  The elements above it are few: the chunks that hold any are read
// again, an element a thread (looking through the registers' chunks took 190
// registers), and ranked against each other.  If they are fewer than `top`, the
// rest equals the bound and follows in the order of the ids, which is the order
// of the chunks (constant rows, rows masked but for a few ids).  Where too many
// lie above the bound, each rank is searched for.
template <int DT, bool FL, int U, typename Emit>
__device__ __forceinline__ void segment_top(TopShared& sh, int top, const Row<DT, FL>& z, int c0, int cn,
                                            const float (&cm)[U], float mine, Emit emit) {
    constexpr int EPC = kEpc<DT>;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int full = min(cn, kThreads) / 64;   // waves whose lanes all hold a chunk
    float low = kNegInf;
    if (wave < full) {
        float v = mine;
        for (int i = 0; i < (top + full - 1) / full; ++i) {
            low = wmax(v);
            const unsigned long long at = __ballot(v == low);
            if (at != 0 && lane == __builtin_ctzll(at)) v = __builtin_nanf("");   // passed over from here on
            if (at == 0) low = kNegInf;
        }
    }
    __syncthreads();   // sh may still be read from the last use
    if (lane == 0) sh.low[wave] = low;
    if (threadIdx.x == 0) sh.count = sh.chunks = 0;
    __syncthreads();
    low = full > 0 ? sh.low[0] : kNegInf;
    for (int w = 1; w < full; ++w) low = fminf(low, sh.low[w]);

#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = u * kThreads + threadIdx.x;
        if (i < cn && cm[u] > low) {
            const int at = atomicAdd(&sh.chunks, 1);
            if (at < kChunkCand) sh.chunk[at] = i;
        }
    }
    __syncthreads();
    const int chunks = sh.chunks;
    auto element = [&](int i, int e, auto f) {
        const int v = z.first(c0 + i) + e;
        if (v >= 0 && v < z.cols) f(z.load_elem(v), v);
    };
    if (chunks <= kChunkCand)
        for (int j = threadIdx.x; j < chunks * EPC; j += kThreads)
            element(sh.chunk[j / EPC], j % EPC, [&](float x, int v) {
                if (!(x > low)) return;
                const int at = atomicAdd(&sh.count, 1);
                if (at < kCand) sh.cand[at] = rank_key(x, v);
            });
    __syncthreads();
    const int n = sh.count;
    if (chunks > kChunkCand || n > kCand) {
        search_ranks(
            sh, top,
            [&](auto f) {
                for (int j = threadIdx.x; j < cn * EPC; j += kThreads)
                    element(j / EPC, j % EPC, [&](float x, int v) { f(rank_key(x, v)); });
            },
            emit);
        return;
    }
    rank_candidates(sh, n, top, emit);
    // NaN ranks with -inf
    auto tie = [&](float x) { return x == low || (x != x && low == kNegInf); };
    int at = n;   // ranks given so far
    for (int b = 0; at < top && b < cn; b += kThreads) {
        const int i = b + threadIdx.x;
        int mine_ties = 0;
        if (i < cn)
            for (int e = 0; e < EPC; ++e) element(i, e, [&](float x, int) { mine_ties += tie(x) ? 1 : 0; });
        int upto = mine_ties;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int v = __shfl_up(upto, o, 64);
            if (lane >= o) upto += v;
        }
        __syncthreads();
        if (lane == 63) sh.ties[wave] = upto;
        __syncthreads();
        int rank = at + upto - mine_ties, all = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            rank += w < wave ? sh.ties[w] : 0;
            all += sh.ties[w];
        }
        if (mine_ties > 0 && rank < top)
            for (int e = 0; e < EPC; ++e)
                element(i, e, [&](float x, int v) {
                    if (tie(x) && rank < top) emit(rank++, rank_key(x, v));
                });
        at += all;
    }
    for (int j = at + threadIdx.x; j < top; j += kThreads) emit(j, 0);   // fewer elements than that
}

// The `top` largest of the keys a workgroup holds (0: none), all different; the
// bound as in segment_top, from the keys' logits.
template <int U, typename Emit>
__device__ __forceinline__ void keys_top(TopShared& sh, int top, const uint64_t (&key)[U], Emit emit) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint64_t most = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) most = most > key[u] ? most : key[u];
    const float mine = most != 0 ? key_value(most) : kNegInf;
    float v = mine, low = kNegInf;
    for (int i = 0; i < (top + 3) / 4; ++i) {
        low = wmax(v);
        const unsigned long long at = __ballot(v == low);
        if (at != 0 && lane == __builtin_ctzll(at)) v = __builtin_nanf("");   // passed over from here on
        if (at == 0) low = kNegInf;
    }
    __syncthreads();   // sh may still be read from the last use
    if (lane == 0) sh.low[wave] = low;
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
    low = fminf(fminf(sh.low[0], sh.low[1]), fminf(sh.low[2], sh.low[3]));
    if (mine >= low)
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (key[u] != 0 && key_value(key[u]) >= low) {
                const int at = atomicAdd(&sh.count, 1);
                if (at < kCand) sh.cand[at] = key[u];
            }
    __syncthreads();
    const int n = sh.count;
    if (n <= kCand) {
        rank_candidates(sh, n, top, emit);
        for (int j = n + threadIdx.x; j < top; j += kThreads) emit(j, 0);
    } else {
        search_ranks(
            sh, top,
            [&](auto f) {
#pragma unroll
                for (int u = 0; u < U; ++u) f(key[u]);
            },
            emit);
    }
}

// Results of a row of log probabilities.
template <int DT, bool FL>
__device__ __forceinline__ void put_logprobs(const LogitsArgs& a, int64_t row, int tok, const Stats& st, Lse l) {
    if (a.logp) a.logp[row] = log_q(Row<DT, FL>(a.z, a.z_ld, row, a.cols).load_elem(tok), a.inv_temp, st);
    if (a.entropy) a.entropy[row] = st.s == st.s ? entropy_of(st, a.inv_temp) : st.s;
    put_lse(a, row, l);
}
template <int NT>
__device__ __forceinline__ void skip_logprobs(const LogitsArgs& a, int64_t row) {
    const int tid = threadIdx.x % NT;
    if (tid == 0) {
        if (a.logp) a.logp[row] = 0.f;
        if (a.entropy) a.entropy[row] = 0.f;
        put_lse(a, row, {0.f, 0.f});
    }
    for (int j = tid; j < a.top; j += NT) {
        a.top_idx[row * a.top + j] = -1;
        a.top_logp[row * a.top + j] = kNegInf;
    }
}
__device__ __forceinline__ void put_alternative(const LogitsArgs& a, int64_t row, const Stats& st, int rank,
                                                uint64_t key) {
    a.top_idx[row * a.top + rank] = key_id(key);
    a.top_logp[row * a.top + rank] = log_q(key_value(key), a.inv_temp, st);
}

// ---- forward passes --------------------------------------------------------------
// One workgroup per segment.  KIND 0: distillation, 1: log probabilities, 2:
// the same with alternatives.  HBM bound: bf16 2048 x 131072 97 us (5.5 TB/s)
// with the join, 4000 x 65537 120 us (4.4 TB/s).
// (Alternatives over bf16 logits are held to the registers of six waves a SIMD
// instead of five: 4000 x 65537 with 5 of them 147 and 138 us, with 20 187 and 178.
// In fp32 it spills more and loses: 2048 x 65536 with 5 of them 104 and 111 us.)
template <int DT, int U, int KIND, bool FL>
__global__ __launch_bounds__(kThreads, KIND == 2 && DT == 0 ? 6 : 1) void forward_kernel(const LogitsArgs a) {
    __shared__ Stats part[4];
    const int64_t row = blockIdx.x / a.plan.segs;
    const int seg = blockIdx.x % a.plan.segs;
    const bool alone = a.plan.segs == 1;
    int tok = 0;
    if constexpr (KIND == 0) {
        if (a.weight && a.weight[row] == 0.f) {
            if (alone && threadIdx.x == 0) {
                a.loss[row] = 0.f;
                put_lse(a, row, {0.f, 0.f});
            }
            return;
        }
    } else {
        if (a.tokens) tok = load_id(a.tokens, a.idx64, row, a.cols);
        if (tok < 0) {
            if (alone) skip_logprobs<kThreads>(a, row);
            return;
        }
    }
    const Row<DT, FL> z(a.z, a.z_ld, row, a.cols);
    const int c0 = seg * a.plan.chunks, cn = min(a.plan.chunks, z.chunks() - c0);
    u32x4 r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = u * kThreads + threadIdx.x;
        r[u] = z.load(i < cn ? c0 + i : kNoChunk);
    }
    const float c = a.inv_temp * kLog2e;
    float cm[U];
    const float mine = chunk_max<DT, U>(r, cm);
    Stats st = wave_stats<DT, U>(r, wmax(mine), c, KIND != 0 && a.entropy != nullptr);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = st;
    __syncthreads();
    st = join(join(part[0], part[1], c), join(part[2], part[3], c), c);
    if (!alone && threadIdx.x == 0) a.part[row * a.plan.segs + seg] = {st.m, st.s, st.e, 0.f};
    const Lse l = make_lse(st, a.inv_temp);
    if constexpr (KIND == 0) {
        if (alone) distill_loss<DT, FL, kThreads>(a, row, st, l);
    } else {
        if (alone && threadIdx.x == 0) put_logprobs<DT, FL>(a, row, tok, st, l);
        if constexpr (KIND == 2) {
            __shared__ TopShared sh;
            segment_top<DT, FL, U>(sh, a.top, z, c0, cn, cm, mine, [&](int rank, uint64_t key) {
                if (alone) put_alternative(a, row, st, rank, key);
                else a.keys[(row * a.plan.segs + seg) * a.top + rank] = key;
            });
        }
    }
}

// Joins the segments of a row: one workgroup, or (WAVE) one wave where a wave
// holds all keys or entries.  Bound by its own latency: 5 us, 7 - 9 us with 5 - 20
// alternatives in one workgroup, 19 with 64.
constexpr int kMergeKeys = 8;   // keys a thread holds
template <int DT, int KIND, bool FL, bool WAVE>
__global__ __launch_bounds__(kThreads) void merge_kernel(const LogitsArgs a) {
    constexpr int NT = WAVE ? 64 : kThreads;
    const int lane = threadIdx.x & 63;
    const int64_t row = WAVE ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
    if (row >= a.rows) return;
    int tok = 0;
    if constexpr (KIND == 0) {
        if (a.weight && a.weight[row] == 0.f) {
            if (threadIdx.x % NT == 0) {
                a.loss[row] = 0.f;
                put_lse(a, row, {0.f, 0.f});
            }
            return;
        }
    } else {
        if (a.tokens) tok = load_id(a.tokens, a.idx64, row, a.cols);
        if (tok < 0) {
            skip_logprobs<NT>(a, row);
            return;
        }
    }
    const float c = a.inv_temp * kLog2e;
    // every wave joins them all, in the same order
    Stats st = kEmpty;
    for (int i = lane; i < a.plan.segs; i += 64) {
        const SegStats p = a.part[row * a.plan.segs + i];
        st = join(st, Stats{p.m, p.s, p.e}, c);
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
        const Stats b = {__shfl_xor(st.m, o, 64), __shfl_xor(st.s, o, 64), __shfl_xor(st.e, o, 64)};
        st = (lane & o) ? join(b, st, c) : join(st, b, c);
    }
    const Lse l = make_lse(st, a.inv_temp);
    if constexpr (KIND == 0) {
        distill_loss<DT, FL, NT>(a, row, st, l);
    } else {
        if (threadIdx.x % NT == 0) put_logprobs<DT, FL>(a, row, tok, st, l);
        if constexpr (KIND == 2) {
            const int64_t n = (int64_t)a.plan.segs * a.top;
            const uint64_t* keys = a.keys + row * n;
            if constexpr (WAVE) {   // a key a lane
                const uint64_t key = lane < n ? keys[lane] : 0;
                int rank = 0;
                for (int j = 0; j < (int)n; ++j) {
                    const uint64_t o = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)key, j) |
                                       (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(key >> 32), j) << 32;
                    rank += o > key ? 1 : 0;
                }
                if (key != 0 && rank < a.top) put_alternative(a, row, st, rank, key);
            } else {
                __shared__ TopShared sh;
                __shared__ uint64_t carry[kMaxTop];
                // A segment's keys are in order: with r = ceil(top / segments), at
                // least `top` keys reach the ceil(top / r)-th largest of the segments'
                // r-th ones, and few more unless the row is full of ties.  (4 x 131072
                // with 64 alternatives: 113 us in batches alone, 19 with this bound.)
                const int segs = min(a.plan.segs, kThreads), r = (a.top + segs - 1) / segs;
                const int i0 = threadIdx.x;
                const uint64_t own = i0 < segs ? keys[(int64_t)i0 * a.top + r - 1] : 0;
                sh.cand[i0] = own;
                if (i0 == 0) sh.count = 0;
                __syncthreads();
                int place = 0;
                for (int j = 0; j < segs; ++j) place += sh.cand[j] > own || (sh.cand[j] == own && j < i0) ? 1 : 0;
                if (i0 < segs && place == (a.top + r - 1) / r - 1) sh.best[0] = own;
                __syncthreads();
                const uint64_t low = sh.best[0];
                for (int64_t i = threadIdx.x; i < n; i += kThreads) {
                    const uint64_t k = keys[i];
                    if (k == 0 || k < low) continue;
                    const int at = atomicAdd(&sh.count, 1);
                    if (at < kCand) sh.cand[at] = k;
                }
                __syncthreads();
                const int found = sh.count;
                if (found <= kCand) {
                    auto put = [&](int rank, uint64_t k) { put_alternative(a, row, st, rank, k); };
                    rank_candidates(sh, found, a.top, put);
                    for (int j = found + threadIdx.x; j < a.top; j += kThreads) put(j, 0);
                    return;
                }
                // batches of keys, the best so far among the next
                const int batch = kThreads * kMergeKeys - a.top;
                for (int64_t b = 0; b < n; b += batch) {
                    uint64_t key[kMergeKeys];
#pragma unroll
                    for (int u = 0; u < kMergeKeys; ++u) {
                        const int i = u * kThreads + threadIdx.x;   // the first `top` are the best so far
                        key[u] = i < a.top ? (b > 0 ? carry[i] : 0)
                                           : (i - a.top < batch && b + i - a.top < n ? keys[b + i - a.top] : 0);
                    }
                    const bool last = b + batch >= n;
                    __syncthreads();
                    keys_top(sh, a.top, key, [&](int rank, uint64_t k) {
                        if (last) put_alternative(a, row, st, rank, k);
                        else carry[rank] = k;
                    });
                    __syncthreads();
                }
            }
        }
    }
}

// ---- gradients from a known lse ------------------------------------------------------
// One workgroup per segment.  KIND 0: distillation, 1: log probabilities.
// In place each chunk is read before its own element is written, and the
// entries' logits before any.  HBM bound: fp32 1024 x 65536 82 us (6.5 TB/s), bf16
// 2048 x 131072 223 us (4.8 TB/s).
// A far row (Softmax::far: s past fp32's range, or fp32 rows of the lowest value
// only) is left to the workgroup of its first segment, which looks for the
// largest logit first.
template <int DT, int KIND, bool FL>
__global__ __launch_bounds__(kThreads) void grad_kernel(const LogitsArgs a) {
    constexpr int U = 4, EPC = kEpc<DT>;
    const int64_t row = blockIdx.x / a.plan.segs;
    const int seg = blockIdx.x % a.plan.segs;
    const Row<DT, FL> z(a.z, a.z_ld, row, a.cols), dz(a.dz, a.dz_ld, row, a.cols);
    int c0 = seg * a.plan.chunks, c1 = min(z.chunks(), c0 + a.plan.chunks);
    const Lse l = get_lse(a, row);
    Softmax q(a.inv_temp, l);
    if (Softmax::far(l)) {
        if (seg > 0) return;
        c1 = z.chunks();
        float m[1] = {kNegInf};
        for (int v = threadIdx.x; v < a.cols; v += kThreads) m[0] = fmaxf(m[0], z.load_elem(v));
        m[0] = wmax(m[0]);
        __shared__ float red0[4][1];
        block_join<kThreads>(m, red0, kNegInf, Max());
        q.set_far(a.inv_temp, m[0]);
    }
    const int v_lo = max(0, z.first(c0)), v_hi = min(a.cols, z.first(c1));   // this segment's columns

    // ---- what the row's gradient is made of ----
    int tok = -1;
    float gl = 0.f, gh = 0.f, scale = 0.f;
    constexpr int KE = KIND == 0 ? kMaxEntries / kThreads : 1;
    int fix_id[KE];
    float fix[KE];
    bool live = true;
    if constexpr (KIND == 1) {
        if (a.tokens) tok = load_id(a.tokens, a.idx64, row, a.cols);
        gl = a.g_logp ? a.g_logp[row] * a.inv_temp : 0.f;
        gh = a.g_entropy ? a.g_entropy[row] * a.inv_temp : 0.f;
        if (a.tokens && tok < 0) gl = gh = 0.f;
        live = !(gl == 0.f && gh == 0.f);
    } else {
        __shared__ float red1[4][2], red2[4][1];
        __shared__ int ids[kMaxEntries];
        __shared__ float ps[kMaxEntries];
        const float w = a.weight ? a.weight[row] : 1.f;   // (none: the second pass of a call without weights)
        live = w != 0.f;
        if (live) {
            Entry x[KE];
            float mx[2] = {kNegInf, 0.f};
#pragma unroll
            for (int i = 0; i < KE; ++i) {
                x[i] = load_entry<DT, FL>(a, z, row, i * kThreads + threadIdx.x);
                mx[0] = fmaxf(mx[0], x[i].u);
                if (!(x[i].u == kNegInf)) mx[1] = 1.f;
            }
            mx[0] = wmax(mx[0]);
            mx[1] = wmax(mx[1]);
            block_join<kThreads>(mx, red1, kNegInf, Max());
            live = mx[1] != 0.f;
            if (live) {
                const float M = a.normalize ? mx[0] : 0.f;
                float sum[1] = {0.f};
#pragma unroll
                for (int i = 0; i < KE; ++i) {
                    const int j = i * kThreads + threadIdx.x;
                    const float e = x[i].u == kNegInf ? 0.f : exp2_hw((x[i].u - M) * kLog2e);
                    sum[0] += e;
                    if (j < a.k) {
                        ids[j] = x[i].id;
                        ps[j] = e;
                    }
                }
                sum[0] = wsum(sum[0]);
                block_join<kThreads>(sum, red2, 0.f, Sum());   // publishes ids, ps
                const float P = a.normalize ? 1.f : sum[0], r = a.normalize ? 1.f / sum[0] : 1.f;
                const float cw = w * a.inv_temp;
                scale = cw * P;
#pragma unroll
                for (int i = 0; i < KE; ++i) {
                    fix_id[i] = x[i].id >= v_lo && x[i].id < v_hi ? x[i].id : -1;
                    fix[i] = 0.f;
                    if (fix_id[i] >= 0)
                        fix[i] = cw * (P * q(z.load_elem(x[i].id)) - r * mass_at(ids, ps, a.k, x[i].id));
                }
            }
        }
        __syncthreads();   // in place: every entry's logit is read before a gradient is stored in the segment
    }
    if (!live) {
        for (int ch = c0 + threadIdx.x; ch < c1; ch += kThreads) dz.store(ch, u32x4{0u, 0u, 0u, 0u}, z.mis);
        return;
    }

    // log probabilities: dz = -q (gl + gh (log q + H)), and gl more at the token
    const float H = KIND == 1 && gh != 0.f ? a.entropy[row] : 0.f;
    const float slope = q.slope * gh, at0 = gl + (gh != 0.f ? gh * (H - q.lo) : 0.f);
    for (int b = c0; b < c1; b += kThreads * U) {
        u32x4 r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int ch = b + u * kThreads + threadIdx.x;
            r[u] = z.load(ch < c1 ? ch : kNoChunk);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int ch = b + u * kThreads + threadIdx.x;
            if (ch >= c1) continue;
            float g[EPC];
#pragma unroll
            for (int e = 0; e < EPC; ++e) {
                const float d = q.diff(elem<DT>(r[u], e)), p = q.at(d);
                if constexpr (KIND == 0) {
                    g[e] = scale * p;
                } else if (gh == 0.f) {
                    g[e] = -gl * p;
                } else {
                    const float t = __builtin_fmaf(d, slope, at0);
                    g[e] = p == 0.f ? 0.f : -p * t;
                }
            }
            if constexpr (KIND == 1) {
                const int d = tok - z.first(ch);
                if (d >= 0 && d < EPC && tok >= 0)
#pragma unroll
                    for (int e = 0; e < EPC; ++e)
                        if (e == d) g[e] += gl;
            }
            dz.store(ch, pack<DT>(g), z.mis);
        }
    }
    if constexpr (KIND == 0) {
        __syncthreads();   // after the stores of the whole segment
#pragma unroll
        for (int i = 0; i < KE; ++i)
            if (fix_id[i] >= 0) dz.store_elem(fix_id[i], fix[i]);
    }
}

// ---- distillation, loss and gradient, the row on chip ---------------------------------
// One workgroup of NT threads a row, U chunks a thread, rows in turn.  A thread
// holds its chunks packed in registers; as each is turned into its gradient and
// stored, the next row's chunk is loaded in its place, so that one row's stores
// and the next one's loads overlap the products between them.
// GRID 0: rows of whole chunks; 1: rows that start or end inside a chunk, z and
// dz on the same grid; 2: on different ones (stored element by element).  The
// elements of a row's partial chunks are held one each by the first threads.
// bf16, 64 entries a row: 2048 x 131072 in 256 us (4.2 TB/s; a large copy
// reaches 4.9), 2048 x 65537 in 159 us (3.4 TB/s); fp32 2048 x 65536 in 236 us
// (4.5 TB/s).  16, 18 and 20 chunks of 1024 threads spill 12, 56 and 104 bytes a
// thread, off the grid 80, 132 and 204: 2048 x 131071 takes 318 us (3.4 TB/s).
template <int DT, int NT, int U, int GRID>
__global__ __launch_bounds__(NT) void distill_row_kernel(const LogitsArgs a) {
    constexpr bool FL = GRID == 0;
    constexpr int EPC = kEpc<DT>, KE = kMaxEntries / NT;
    __shared__ float red1[NT / 64][3], red2[NT / 64][4];
    __shared__ int ids[kMaxEntries];
    __shared__ float ps[kMaxEntries];
    const float c = a.inv_temp * kLog2e;
    auto weight_of = [&](int64_t row) { return row < a.rows ? (a.weight ? a.weight[row] : 1.f) : 0.f; };
    // whole chunk c of a row, -inf otherwise
    auto load = [&](const Row<DT, FL>& z, int ch) __attribute__((always_inline)) {
        const unsigned none = DT == 0 ? 0xff80ff80u : 0xff800000u;
        return z.whole(ch) ? *reinterpret_cast<const u32x4*>(z.at(ch)) : u32x4{none, none, none, none};
    };
    // column this thread holds of the row's partial chunks (-1: none)
    auto edge_of = [&](const Row<DT, FL>& z) {
        if (FL || threadIdx.x >= 2 * EPC) return -1;
        const int e = threadIdx.x % EPC, last = z.chunks() - 1;
        const int ch = threadIdx.x < EPC ? 0 : last;
        if (threadIdx.x >= EPC && last == 0) return -1;   // the first chunk is the last one
        const int col = z.first(ch) + e;
        return z.whole(ch) || col < 0 || col >= z.cols ? -1 : col;
    };

    int64_t row = blockIdx.x;
    float w = weight_of(row), ez = kNegInf;
    u32x4 r[U];
    {
        // a row that counts nothing is not read: no columns
        const Row<DT, FL> z(a.z, a.z_ld, row, w != 0.f ? a.cols : 0);
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = load(z, u * NT + threadIdx.x);
        const int edge = edge_of(z);
        if (edge >= 0) ez = z.load_elem(edge);
    }
    for (; row < a.rows; row += gridDim.x) {
        const Row<DT, FL> z(a.z, a.z_ld, row, a.cols), dz(a.dz, a.dz_ld, row, a.cols);
        const int64_t next = row + gridDim.x;
        const float w_next = weight_of(next);
        const Row<DT, FL> zn(a.z, a.z_ld, next < a.rows ? next : row, w_next != 0.f ? a.cols : 0);

        // ---- largest logit, the teacher's entries ----
        Entry x[KE];
#pragma unroll
        for (int i = 0; i < KE; ++i) x[i] = {-1, kNegInf, 0.f};
        float mx[3] = {kNegInf, 0.f, FL ? kNegInf : ez};   // teacher's largest u, any entry, largest logit
        if (w != 0.f) {
#pragma unroll
            for (int i = 0; i < KE; ++i) {
                x[i] = load_entry<DT, FL>(a, z, row, i * NT + threadIdx.x);
                mx[0] = fmaxf(mx[0], x[i].u);
                if (!(x[i].u == kNegInf)) mx[1] = 1.f;
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < EPC; ++e) mx[2] = fmaxf(mx[2], elem<DT>(r[u], e));
#pragma unroll
            for (int i = 0; i < 3; ++i) mx[i] = wmax(mx[i]);
            block_join<NT>(mx, red1, kNegInf, Max());
        }
        const bool live = mx[1] != 0.f;
        stay_packed(r);

        // ---- sums ----
        const float ref = mx[2] == kNegInf ? 0.f : mx[2], M = a.normalize ? mx[0] : 0.f;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};   // S of the row; S, E, G of the teacher
        Lse l = {0.f, 0.f};
        float scale = 0.f, loss = 0.f, lg = 0.f, fix[KE];   // lg: log2 S
        // from the largest logit, which is at hand here
        auto q = [&](float v) { return exp2_hw(__builtin_fmaf(v - ref, c, -lg)); };
        if (live) {
#pragma unroll
            for (int i = 0; i < KE; ++i) {
                const float e = x[i].u == kNegInf ? 0.f : exp2_hw((x[i].u - M) * kLog2e);
                const int j = i * NT + threadIdx.x;
                if (j < a.k) {
                    ids[j] = x[i].id;
                    ps[j] = e;
                }
                if (e == 0.f) continue;
                sum[1] += e;
                sum[2] += e * (x[i].u - M);
                sum[3] += e * ((x[i].z - ref) * a.inv_temp);
            }
            if (!FL) sum[0] = exp2_hw((ez - ref) * c);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < EPC; ++e) sum[0] += exp2_hw((elem<DT>(r[u], e) - ref) * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] = wsum(sum[i]);
            block_join<NT>(sum, red2, 0.f, Sum());   // publishes ids and ps
            l = make_lse(Stats{mx[2], sum[0], 0.f}, a.inv_temp);
            const TeacherSums t = teacher_sums(a, sum[1], sum[2], sum[3]);
            // b is relative to the row's largest logit: B = -log S
            if (sum[0] != 0.f) lg = __builtin_amdgcn_logf(sum[0]);
            loss = w * (t.loss + t.P * (lg * kLn2));
            const float cw = w * a.inv_temp;
            scale = cw * t.P;
#pragma unroll
            for (int i = 0; i < KE; ++i)
                fix[i] = x[i].id >= 0 ? cw * (t.P * q(x[i].z) - t.scale * mass_at(ids, ps, a.k, x[i].id)) : 0.f;
        }
        if (threadIdx.x == 0) {
            a.loss[row] = loss;
            put_lse(a, row, l);
        }
        stay_packed(r);

        // ---- the gradient, and the next row's loads ----
        const unsigned mask = live ? ~0u : 0u;   // a row that counts nothing gets zeros whatever it holds
        const int edge = edge_of(z);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int ch = u * NT + threadIdx.x;
            float g[EPC];
#pragma unroll
            for (int e = 0; e < EPC; ++e) g[e] = scale * q(elem<DT>(r[u], e));
            if (z.whole(ch)) {
                if constexpr (GRID == 2) {
#pragma unroll
                    for (int e = 0; e < EPC; ++e) dz.store_elem(z.first(ch) + e, live ? g[e] : 0.f);
                } else {
                    *reinterpret_cast<u32x4*>(dz.at(ch)) = pack<DT>(g) & mask;
                }
            }
            r[u] = load(zn, ch);
            __builtin_amdgcn_sched_barrier(0);   // else all chunks of both rows are held at once
        }
        if (!FL) {
            if (edge >= 0) dz.store_elem(edge, live ? scale * q(ez) : 0.f);
            const int edge_next = edge_of(zn);
            ez = edge_next >= 0 ? zn.load_elem(edge_next) : kNegInf;
        }
        __syncthreads();   // the row's stores before those of its entries; ids and ps are free
        if (live)
#pragma unroll
            for (int i = 0; i < KE; ++i)
                if (x[i].id >= 0) dz.store_elem(x[i].id, fix[i]);
        w = w_next;
    }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// chunks a row takes at the worst alignment
int64_t row_chunks(int32_t cols, int32_t dtype) { return cdiv(cols, dtype == 0 ? 8 : 4) + 1; }
// ... and of these rows: one less where every row starts a chunk
int64_t row_chunks(const LogitsArgs& a) {
    const int epc = a.dtype == 0 ? 8 : 4;
    const bool flush = (reinterpret_cast<uintptr_t>(a.z) & 15) == 0 && (a.z_ld % epc == 0 || a.rows == 1);
    return cdiv(a.cols, epc) + (flush ? 0 : 1);
}

// every row of both starts and ends on the 16-byte grid
bool flush(const LogitsArgs& a) {
    const int epc = a.dtype == 0 ? 8 : 4;
    auto on = [&](const void* p, int64_t ld) {
        return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld % epc == 0 || a.rows == 1);
    };
    return a.cols % epc == 0 && on(a.z, a.z_ld) && (a.dz == nullptr || on(a.dz, a.dz_ld));
}

// The call's rows [r, r + n).
LogitsArgs rows_of(const LogitsArgs& a, int64_t r, int32_t n) {
    LogitsArgs b = a;
    b.rows = n;
    auto on = [&](auto& p, int64_t bytes) {
        using P = std::remove_reference_t<decltype(p)>;
        if (p != nullptr) p = reinterpret_cast<P>(reinterpret_cast<uintptr_t>(p) + (uintptr_t)(r * bytes));
    };
    const int64_t es = a.dtype == 0 ? 2 : 4, id = a.idx64 ? 8 : 4;
    on(b.z, a.z_ld * es);
    on(b.dz, a.dz_ld * es);
    on(b.idx, a.k * id);
    on(b.t, a.t_ld * 4);
    on(b.weight, 4);
    on(b.loss, 4);
    on(b.lse, 8);
    on(b.tokens, id);
    on(b.logp, 4);
    on(b.entropy, 4);
    on(b.top_idx, a.top * 4);
    on(b.top_logp, a.top * 4);
    on(b.g_logp, 4);
    on(b.g_entropy, 4);
    on(b.part, a.plan.segs * (int64_t)sizeof(SegStats));
    on(b.keys, a.plan.segs * (int64_t)sizeof(uint64_t) * a.top);
    return b;
}
// Launches f over all rows: a launch holds at most 2^32 - 1 threads, so rows
// past that follow in further ones.
template <typename F>
hipError_t in_launches(const LogitsArgs& a, F f) {
    const int64_t most = std::max<int64_t>(1, UINT32_MAX / kThreads / a.plan.segs);
    if (a.rows <= most) return f(a);
    for (int64_t r = 0; r < a.rows; r += most) {
        const hipError_t e = f(rows_of(a, r, (int32_t)std::min<int64_t>(most, a.rows - r)));
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int DT, int KIND, bool FL>
hipError_t forward_fl(const LogitsArgs& a, hipStream_t s) {
    const dim3 grid((uint32_t)((int64_t)a.rows * a.plan.segs)), block(kThreads);
    switch (a.plan.u) {
        case 1: hipLaunchKernelGGL((forward_kernel<DT, 1, KIND, FL>), grid, block, 0, s, a); break;
        case 2: hipLaunchKernelGGL((forward_kernel<DT, 2, KIND, FL>), grid, block, 0, s, a); break;
        case 4: hipLaunchKernelGGL((forward_kernel<DT, 4, KIND, FL>), grid, block, 0, s, a); break;
        default: hipLaunchKernelGGL((forward_kernel<DT, 8, KIND, FL>), grid, block, 0, s, a); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.plan.segs == 1) return e;
    const bool wave = KIND == 0 ? a.k <= 64 : KIND == 1 || (int64_t)a.plan.segs * a.top <= 64;
    if (wave) hipLaunchKernelGGL((merge_kernel<DT, KIND, FL, true>), dim3((uint32_t)cdiv(a.rows, 4)), block, 0, s, a);
    else hipLaunchKernelGGL((merge_kernel<DT, KIND, FL, false>), dim3(a.rows), block, 0, s, a);
    return hipGetLastError();
}

template <int KIND>
hipError_t forward(const LogitsArgs& a, hipStream_t s) {
    const bool fl = flush(a);
    return in_launches(a, [&](const LogitsArgs& b) {
        if (fl) return b.dtype == 0 ? forward_fl<0, KIND, true>(b, s) : forward_fl<1, KIND, true>(b, s);
        return b.dtype == 0 ? forward_fl<0, KIND, false>(b, s) : forward_fl<1, KIND, false>(b, s);
    });
}

template <int KIND, bool FL>
hipError_t grad_fl(const LogitsArgs& a, hipStream_t s) {
    const dim3 grid((uint32_t)((int64_t)a.rows * a.plan.segs));
    if (a.dtype == 0) hipLaunchKernelGGL((grad_kernel<0, KIND, FL>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((grad_kernel<1, KIND, FL>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}
template <int KIND>
hipError_t grad(LogitsArgs a, hipStream_t s) {
    a.plan = seg_plan(a.rows, a.cols, a.dtype);
    const bool fl = flush(a);
    return in_launches(a, [&](const LogitsArgs& b) {
        return fl ? grad_fl<KIND, true>(b, s) : grad_fl<KIND, false>(b, s);
    });
}

template <int DT, int NT, int U, int GRID>
hipError_t row_launch(const LogitsArgs& a, hipStream_t s) {
    static const int cus = [] { const int c = device_cus(); return c > 0 ? c : 256; }();
    // workgroups the chip holds at once (64 registers a thread up to four chunks, 128 above)
    const int64_t most = (int64_t)cus * ((U <= 4 ? 2048 : 1024) / NT);
    hipLaunchKernelGGL((distill_row_kernel<DT, NT, U, GRID>), dim3((uint32_t)std::min<int64_t>(a.rows, most)), dim3(NT),
                       0, s, a);
    return hipGetLastError();
}

// The fewest threads and chunks that hold a row: 2048 x 131071 in bf16, which
// needs 17 chunks of 1024 threads, takes 321 us with 18 and 353 us with 20.
template <int DT, int GRID>
hipError_t row_size(const LogitsArgs& a, hipStream_t s) {
    const int64_t n = row_chunks(a);
    if constexpr (GRID == 2) {   // rare, and bound by its stores: fewer sizes
        if (n <= 256 * 8) return row_launch<DT, 256, 8, GRID>(a, s);
        if (n <= 1024 * 8) return row_launch<DT, 1024, 8, GRID>(a, s);
        return row_launch<DT, 1024, 20, GRID>(a, s);
    } else {
        if (n <= 256 * 1) return row_launch<DT, 256, 1, GRID>(a, s);
        if (n <= 256 * 2) return row_launch<DT, 256, 2, GRID>(a, s);
        if (n <= 256 * 3) return row_launch<DT, 256, 3, GRID>(a, s);
        if (n <= 256 * 4) return row_launch<DT, 256, 4, GRID>(a, s);
        if (n <= 256 * 6) return row_launch<DT, 256, 6, GRID>(a, s);
        if (n <= 256 * 8) return row_launch<DT, 256, 8, GRID>(a, s);
        if (n <= 512 * 6) return row_launch<DT, 512, 6, GRID>(a, s);
        if (n <= 512 * 8) return row_launch<DT, 512, 8, GRID>(a, s);
        if (n <= 1024 * 6) return row_launch<DT, 1024, 6, GRID>(a, s);
        if (n <= 1024 * 8) return row_launch<DT, 1024, 8, GRID>(a, s);
        if (n <= 1024 * 12) return row_launch<DT, 1024, 12, GRID>(a, s);
        if (n <= 1024 * 16) return row_launch<DT, 1024, 16, GRID>(a, s);
        if (n <= 1024 * 18) return row_launch<DT, 1024, 18, GRID>(a, s);
        return row_launch<DT, 1024, 20, GRID>(a, s);
    }
}
template <int GRID>
hipError_t row_dt(const LogitsArgs& a, hipStream_t s) {
    return a.dtype == 0 ? row_size<0, GRID>(a, s) : row_size<1, GRID>(a, s);
}

// z's and dz's rows start at the same place of the 16-byte grid.
bool same_grid(const LogitsArgs& a) {
    const int epc = a.dtype == 0 ? 8 : 4;
    const int64_t apart = reinterpret_cast<intptr_t>(a.z) - reinterpret_cast<intptr_t>(a.dz);
    return apart % 16 == 0 && ((a.z_ld - a.dz_ld) % epc == 0 || a.rows == 1);
}

}  // namespace

SegPlan seg_plan(int32_t rows, int32_t cols, int32_t dtype) {
    const int64_t n = row_chunks(cols, dtype);
    // a thousand workgroups fill the chip; the smaller the segments, the more
    // there is to join
    int u = 8;
    while (u > 1 && rows * cdiv(n, kThreads * (int64_t)u) < 1024) u /= 2;
    SegPlan p;
    p.u = u;
    p.segs = (int32_t)cdiv(n, kThreads * u);
    p.chunks = (int32_t)cdiv(n, p.segs);
    return p;
}

// One pass over a row that fits 1024 threads x 20 chunks (of 128 registers a
// thread 80), against a forward pass and a gradient, on the device: bf16 2048 x
// 131072 256 against 326 us, 2048 x 65537 159 against 196 us, 8192 x 10001 109
// against 135 us, 1 to 256 x 32000 8 to 11 against 12 to 20 us; at the upper end
// 2048 x 163000 357 against 405 us, and 163001, whose rows are off the grid, 409
// against 429 us.  A few long rows lose by it: 1, 16, 64 and 128 x 131072 18, 19, 21
// and 24 against 12, 15, 21 and 29 us, within the 17 us the host takes for a call.
bool distill_on_chip(int32_t cols, int32_t dtype) { return row_chunks(cols, dtype) <= 1024 * 20; }

hipError_t launch_distill(const LogitsArgs& a, hipStream_t s) { return forward<0>(a, s); }
hipError_t launch_distill_on_chip(const LogitsArgs& a, hipStream_t s) {
    return flush(a) ? row_dt<0>(a, s) : same_grid(a) ? row_dt<1>(a, s) : row_dt<2>(a, s);
}
hipError_t launch_distill_grad(const LogitsArgs& a, hipStream_t s) { return grad<0>(a, s); }
hipError_t launch_logprobs(const LogitsArgs& a, hipStream_t s) {
    return a.top > 0 ? forward<2>(a, s) : forward<1>(a, s);
}
hipError_t launch_logprobs_grad(const LogitsArgs& a, hipStream_t s) { return grad<1>(a, s); }

}  // namespace himuon
