// C entry points of the operators around the optimiser step: the experts'
// products and the losses over logits.  Argument checks and launches; see
// include/himuon.h for the contract.
#include <cmath>
#include <new>
#include <stdexcept>

#include "api_util.h"
#include "grouped.h"
#include "logits.h"

using namespace himuon;

namespace {

// No exception crosses the C interface: the checks below sort descriptor lists
// in host memory, which can run out.
template <typename F>
himuon_status_t guarded(F f) {
    try {
        return f();
    } catch (const std::bad_alloc&) {
    } catch (const std::length_error&) {
    }
    return hip_fail(hipErrorOutOfMemory);
}

himuon_status_t check_dtype(himuon_dtype_t dt) {
    return dt == HIMUON_BF16 || dt == HIMUON_FP32 ? HIMUON_OK : HIMUON_ERR_UNSUPPORTED;
}

// A matrix whose rows are tokens: as check_matrix, but it may have no rows.
himuon_status_t check_rows(const himuon_matrix_t& d, size_t es) {
    if (d.rows != 0) return check_matrix(d, es);
    if (d.cols < 1 || d.ld < d.cols) return HIMUON_ERR_INVALID_ARGUMENT;
    return d.cols > INT32_MAX ? HIMUON_ERR_LAYOUT : HIMUON_OK;
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Rows of whole 16-byte chunks, and 256 of them within 32-bit byte offsets.
bool chunked(const himuon_matrix_t& d) { return aligned(d.ptr, 16) && d.ld % 8 == 0 && d.ld <= (1 << 22); }

// Byte range of a contiguous device array, as an extent of one row.
Extent array_extent(const void* p, int64_t bytes) {
    return extent_of(himuon_matrix_t{const_cast<void*>(p), 1, bytes, bytes}, 1, 0);
}

#define HIMUON_TRY(call)                           \
    do {                                           \
        const himuon_status_t st_ = (call);        \
        if (st_ != HIMUON_OK) return st_;          \
    } while (0)

himuon_status_t check_workspace(const void* ws, size_t bytes, size_t need) {
    if (need == 0) return HIMUON_OK;
    if (ws == nullptr || bytes < need) return HIMUON_ERR_WORKSPACE;
    return aligned(ws, 16) ? HIMUON_OK : HIMUON_ERR_LAYOUT;
}

// ---- the experts' products ------------------------------------------------------
// Checks of X, ends and n; fills the arguments every launch of the call shares.
himuon_status_t grouped_args(const himuon_matrix_t* X, const himuon_matrix_t* W, int32_t n, const int32_t* ends,
                             himuon_dtype_t dt, GroupedArgs& a) {
    himuon_status_t st = check_dtype(dt);
    if (st != HIMUON_OK) return st;
    if (X == nullptr || W == nullptr || ends == nullptr || n < 1) return HIMUON_ERR_INVALID_ARGUMENT;
    if (!aligned(ends, sizeof(int32_t))) return HIMUON_ERR_LAYOUT;
    const size_t es = elem_size(dt);
    if ((st = check_rows(*X, es)) != HIMUON_OK) return st;
    for (int32_t e = 0; e < n; ++e) {
        if ((st = check_matrix(W[e], es)) != HIMUON_OK) return st;
        if (W[e].rows != W[0].rows || W[e].cols != W[0].cols) return HIMUON_ERR_INVALID_ARGUMENT;
    }
    for (const int64_t side : {X->rows, X->cols, W[0].rows, W[0].cols})
        if (side > kMaxSide) return HIMUON_ERR_LAYOUT;
    a.x = X->ptr;
    a.x_ld = X->ld;
    a.ends = ends;
    a.rows = (int32_t)X->rows;
    a.kdim = (int32_t)X->cols;
    a.dtype = dt == HIMUON_FP32 ? 1 : 0;
    a.total = n;
    return HIMUON_OK;
}

// True if f holds for every launch of the call (the full ones and the last).
template <typename F>
bool all_launches(GroupedArgs a, F f) {
    for (const int32_t part : {std::min(kExperts, a.total), (a.total - 1) % kExperts + 1}) {
        a.n = part;
        if (!f(a)) return false;
    }
    return true;
}

// Runs f over the launches of the call.
template <typename F>
himuon_status_t each_launch(GroupedArgs& a, const himuon_matrix_t* W, int32_t n, F f) {
    for (int32_t e0 = 0; e0 < n; e0 += kExperts) {
        a.e0 = e0;
        a.n = std::min(kExperts, n - e0);
        a.last = e0 + a.n == n;
        for (int32_t i = 0; i < a.n; ++i) {
            a.w[i] = W[e0 + i].ptr;
            a.w_ld[i] = W[e0 + i].ld;
        }
        const himuon_status_t st = f();
        if (st != HIMUON_OK) return st;
    }
    return HIMUON_OK;
}

himuon_status_t grouped_mm(const himuon_matrix_t* X, const himuon_matrix_t* W, int32_t n, int32_t trans_w,
                           const int32_t* ends, const himuon_matrix_t* Y, himuon_dtype_t dt, void* stream) {
    GroupedArgs a{};
    himuon_status_t st = grouped_args(X, W, n, ends, dt, a);
    if (st != HIMUON_OK) return st;
    if (Y == nullptr) return HIMUON_ERR_INVALID_ARGUMENT;
    const size_t es = elem_size(dt);
    if ((st = check_rows(*Y, es)) != HIMUON_OK) return st;
    const int64_t K = trans_w ? W[0].cols : W[0].rows, N = trans_w ? W[0].rows : W[0].cols;
    if (X->cols != K || Y->cols != N || X->rows != Y->rows) return HIMUON_ERR_INVALID_ARGUMENT;
    if (a.rows == 0) return HIMUON_OK;
    const Extent y = extent_of(*Y, es, 0);
    if (share_element(y, extent_of(*X, es, 0))) return HIMUON_ERR_OVERLAP;
    for (int32_t e = 0; e < n; ++e)
        if (share_element(y, extent_of(W[e], es, 0))) return HIMUON_ERR_OVERLAP;
    if (share_element(y, array_extent(ends, 4 * (int64_t)n))) return HIMUON_ERR_OVERLAP;
    a.y = Y->ptr;
    a.y_ld = Y->ld;
    a.ndim = (int32_t)N;
    a.vec = chunked(*X) && chunked(*Y) && K % 8 == 0 && N % 8 == 0;
    for (int32_t e = 0; e < n; ++e) a.vec = a.vec && chunked(W[e]);
    if (!all_launches(a, grouped_mm_fits)) return HIMUON_ERR_LAYOUT;
    return each_launch(a, W, n, [&] {
        const hipError_t e = launch_grouped_mm(a, trans_w != 0, reinterpret_cast<hipStream_t>(stream));
        return e == hipSuccess ? HIMUON_OK : hip_fail(e);
    });
}

// Workspace of the launch that takes the most: the parts' sums.
size_t wgrad_bytes(const GroupedArgs& a) {
    int64_t most = 0;
    all_launches(a, [&](const GroupedArgs& l) {
        const int64_t parts = l.rows > 0 ? grouped_wgrad_parts(l) : 1;
        if (parts > 1) most = std::max(most, parts * grouped_wgrad_part_bytes(l));
        return true;
    });
    return (size_t)most;
}

himuon_status_t grouped_wgrad(const himuon_matrix_t* X, const himuon_matrix_t* D, const int32_t* ends,
                              const himuon_matrix_t* G, int32_t n, himuon_dtype_t dt, void* workspace,
                              size_t workspace_bytes, void* stream) {
    GroupedArgs a{};
    himuon_status_t st = grouped_args(X, G, n, ends, dt, a);
    if (st != HIMUON_OK) return st;
    if (D == nullptr) return HIMUON_ERR_INVALID_ARGUMENT;
    const size_t es = elem_size(dt);
    if ((st = check_rows(*D, es)) != HIMUON_OK) return st;
    if (G[0].rows != X->cols || G[0].cols != D->cols || X->rows != D->rows) return HIMUON_ERR_INVALID_ARGUMENT;
    std::vector<Extent> ex;
    for (int32_t e = 0; e < n; ++e) ex.push_back(extent_of(G[e], es, e));
    const Extent en = array_extent(ends, 4 * (int64_t)n);
    for (const Extent& g : ex) {
        if (a.rows > 0 && (share_element(g, extent_of(*X, es, 0)) || share_element(g, extent_of(*D, es, 0))))
            return HIMUON_ERR_OVERLAP;
        if (share_element(g, en)) return HIMUON_ERR_OVERLAP;
    }
    if ((st = check_overlap(ex)) != HIMUON_OK) return st;
    a.d = D->ptr;
    a.d_ld = D->ld;
    a.ndim = (int32_t)D->cols;
    a.vec = chunked(*X) && chunked(*D) && a.kdim % 8 == 0 && a.ndim % 8 == 0;
    for (int32_t e = 0; e < n; ++e) a.vec = a.vec && chunked(G[e]);
    if (!all_launches(a, grouped_wgrad_fits)) return HIMUON_ERR_LAYOUT;
    HIMUON_TRY(check_workspace(workspace, workspace_bytes, wgrad_bytes(a)));
    a.sums = reinterpret_cast<float*>(workspace);
    return each_launch(a, G, n, [&] {
        a.parts = grouped_wgrad_parts(a);
        const hipError_t e = launch_grouped_wgrad(a, reinterpret_cast<hipStream_t>(stream));
        return e == hipSuccess ? HIMUON_OK : hip_fail(e);
    });
}

// ---- losses over logits -----------------------------------------------------------
constexpr int64_t kMaxCols = 1 << 29;   // the kernels' chunk offsets within a row fit 32 bits

// Workspace of a forward pass over the rows in segments: the segments' sums,
// then their best keys.  0 where a row is one segment.
size_t parts_bytes(int64_t rows, const SegPlan& p) {
    return p.segs > 1 ? (size_t)rows * p.segs * sizeof(SegStats) : 0;
}
size_t keys_bytes(int64_t rows, const SegPlan& p, int32_t top) {
    return p.segs > 1 ? (size_t)rows * p.segs * top * sizeof(uint64_t) : 0;
}
// Distillation with a gradient where rows are not kept on chip: the sums, and
// the lse between the passes.
size_t distill_bytes(int32_t rows, int32_t cols, int32_t dtype, bool with_grad) {
    if (rows == 0 || (with_grad && distill_on_chip(cols, dtype))) return 0;
    return parts_bytes(rows, seg_plan(rows, cols, dtype)) + (with_grad ? (size_t)rows * 2 * sizeof(float) : 0);
}

// Shape checks of the workspace queries.
himuon_status_t check_shape(const himuon_matrix_t* Z, himuon_dtype_t dt, const size_t* bytes) {
    if (Z == nullptr || bytes == nullptr) return HIMUON_ERR_INVALID_ARGUMENT;
    if (Z->rows < 0 || Z->cols < 1) return HIMUON_ERR_INVALID_ARGUMENT;
    if (Z->rows > INT32_MAX || Z->cols > kMaxCols) return HIMUON_ERR_LAYOUT;
    return check_dtype(dt);
}

himuon_status_t logits_args(const himuon_matrix_t* Z, himuon_index_t it, float temperature, himuon_dtype_t dt,
                            LogitsArgs& a) {
    himuon_status_t st = check_dtype(dt);
    if (st != HIMUON_OK) return st;
    if (it != HIMUON_I32 && it != HIMUON_I64) return HIMUON_ERR_UNSUPPORTED;
    if (Z == nullptr) return HIMUON_ERR_INVALID_ARGUMENT;
    if ((st = check_rows(*Z, elem_size(dt))) != HIMUON_OK) return st;
    if (Z->cols > kMaxCols) return HIMUON_ERR_LAYOUT;
    // (the kernels scale exponents by log2(e) / temperature)
    if (!(temperature > 0.f) || !std::isfinite(temperature) || !std::isfinite(1.4426951f * (1.f / temperature)))
        return HIMUON_ERR_INVALID_ARGUMENT;
    a.z = Z->ptr;
    a.z_ld = Z->ld;
    a.rows = (int32_t)Z->rows;
    a.cols = (int32_t)Z->cols;
    a.dtype = dt == HIMUON_FP32 ? 1 : 0;
    a.plan = seg_plan(a.rows, a.cols, a.dtype);
    if ((int64_t)a.rows * a.plan.segs > INT32_MAX) return HIMUON_ERR_LAYOUT;
    a.idx64 = it == HIMUON_I64;
    a.inv_temp = 1.f / temperature;
    return HIMUON_OK;
}

// dZ: the shape of Z, and Z itself or apart from it.
himuon_status_t grad_arg(const himuon_matrix_t* Z, const himuon_matrix_t* dZ, size_t es, LogitsArgs& a) {
    const himuon_status_t st = check_rows(*dZ, es);
    if (st != HIMUON_OK) return st;
    if (dZ->rows != Z->rows || dZ->cols != Z->cols) return HIMUON_ERR_INVALID_ARGUMENT;
    a.dz = dZ->ptr;
    a.dz_ld = dZ->ld;
    if (Z->rows == 0 || (dZ->ptr == Z->ptr && dZ->ld == Z->ld)) return HIMUON_OK;
    return share_element(extent_of(*dZ, es, 0), extent_of(*Z, es, 0)) ? HIMUON_ERR_OVERLAP : HIMUON_OK;
}

// Device arrays of a call: none written may share memory with another one, or
// with the matrices.
struct Arrays {
    std::vector<Extent> written, read;
    himuon_status_t add(const void* p, int64_t count, size_t es, bool write) {
        if (p == nullptr || count == 0) return HIMUON_OK;
        if (!aligned(p, es)) return HIMUON_ERR_LAYOUT;
        (write ? written : read).push_back(array_extent(p, count * (int64_t)es));
        return HIMUON_OK;
    }
    void add(const himuon_matrix_t* m, size_t es, bool write) {
        if (m != nullptr && m->rows > 0) (write ? written : read).push_back(extent_of(*m, es, 0));
    }
    himuon_status_t check() const {
        for (size_t i = 0; i < written.size(); ++i) {
            for (size_t j = i + 1; j < written.size(); ++j)
                if (share_element(written[i], written[j])) return HIMUON_ERR_OVERLAP;
            for (const Extent& r : read)
                if (share_element(written[i], r)) return HIMUON_ERR_OVERLAP;
        }
        return HIMUON_OK;
    }
};

himuon_status_t teacher_args(const himuon_matrix_t* Z, const void* idx, const himuon_matrix_t* T, int32_t normalize,
                             LogitsArgs& a, Arrays& arr) {
    if (T == nullptr) return HIMUON_ERR_INVALID_ARGUMENT;
    HIMUON_TRY(check_rows(*T, 4));
    if (T->rows != Z->rows) return HIMUON_ERR_INVALID_ARGUMENT;
    if (T->cols > kMaxEntries) return HIMUON_ERR_UNSUPPORTED;
    if (a.rows > 0 && idx == nullptr) return HIMUON_ERR_INVALID_ARGUMENT;
    HIMUON_TRY(arr.add(idx, T->rows * T->cols, a.idx64 ? 8 : 4, false));
    arr.add(T, 4, false);
    a.idx = idx;
    a.t = reinterpret_cast<const float*>(T->ptr);
    a.t_ld = T->ld;
    a.k = (int32_t)T->cols;
    a.normalize = normalize != 0;
    return HIMUON_OK;
}

himuon_status_t distill(const himuon_matrix_t* Z, const void* idx, himuon_index_t it, const himuon_matrix_t* T,
                        float temperature, int32_t normalize, const float* weight, float* loss, float* lse,
                        const himuon_matrix_t* dZ, himuon_dtype_t dt, void* workspace, size_t workspace_bytes,
                        void* stream) {
    LogitsArgs a{};
    Arrays arr;
    const size_t es = elem_size(dt);
    HIMUON_TRY(logits_args(Z, it, temperature, dt, a));
    HIMUON_TRY(teacher_args(Z, idx, T, normalize, a, arr));
    if (dZ != nullptr) HIMUON_TRY(grad_arg(Z, dZ, es, a));
    if (a.rows > 0 && loss == nullptr) return HIMUON_ERR_INVALID_ARGUMENT;
    HIMUON_TRY(arr.add(weight, a.rows, 4, false));
    HIMUON_TRY(arr.add(loss, a.rows, 4, true));
    HIMUON_TRY(arr.add(lse, 2 * (int64_t)a.rows, 4, true));
    if (dZ != nullptr) arr.add(dZ, es, true);
    if (dZ == nullptr || dZ->ptr != Z->ptr) arr.add(Z, es, false);
    HIMUON_TRY(arr.check());
    HIMUON_TRY(check_workspace(workspace, workspace_bytes, distill_bytes(a.rows, a.cols, a.dtype, dZ != nullptr)));
    if (a.rows == 0) return HIMUON_OK;
    a.weight = weight;
    a.loss = loss;
    a.lse = lse;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    hipError_t e;
    if (dZ != nullptr && distill_on_chip(a.cols, a.dtype)) {
        e = launch_distill_on_chip(a, s);
    } else {
        a.part = reinterpret_cast<SegStats*>(workspace);
        if (dZ != nullptr && a.lse == nullptr)
            a.lse = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + parts_bytes(a.rows, a.plan));
        e = launch_distill(a, s);
        if (e == hipSuccess && dZ != nullptr) e = launch_distill_grad(a, s);
    }
    return e == hipSuccess ? HIMUON_OK : hip_fail(e);
}

himuon_status_t distill_grad(const himuon_matrix_t* Z, const void* idx, himuon_index_t it, const himuon_matrix_t* T,
                             float temperature, int32_t normalize, const float* lse, const float* g,
                             const himuon_matrix_t* dZ, himuon_dtype_t dt, void* stream) {
    LogitsArgs a{};
    Arrays arr;
    const size_t es = elem_size(dt);
    HIMUON_TRY(logits_args(Z, it, temperature, dt, a));
    HIMUON_TRY(teacher_args(Z, idx, T, normalize, a, arr));
    if (dZ == nullptr) return HIMUON_ERR_INVALID_ARGUMENT;
    HIMUON_TRY(grad_arg(Z, dZ, es, a));
    if (a.rows > 0 && (lse == nullptr || g == nullptr)) return HIMUON_ERR_INVALID_ARGUMENT;
    HIMUON_TRY(arr.add(lse, 2 * (int64_t)a.rows, 4, false));
    HIMUON_TRY(arr.add(g, a.rows, 4, false));
    arr.add(dZ, es, true);
    HIMUON_TRY(arr.check());
    if (a.rows == 0) return HIMUON_OK;
    a.lse = const_cast<float*>(lse);
    a.weight = g;
    const hipError_t e = launch_distill_grad(a, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? HIMUON_OK : hip_fail(e);
}

himuon_status_t token_logprobs(const himuon_matrix_t* Z, const void* tokens, himuon_index_t it, float temperature,
                               int32_t top, float* logp, float* entropy, float* lse, int32_t* top_idx,
                               float* top_logp, himuon_dtype_t dt, void* workspace, size_t workspace_bytes,
                               void* stream) {
    LogitsArgs a{};
    Arrays arr;
    HIMUON_TRY(logits_args(Z, it, temperature, dt, a));
    if (top < 0 || top > a.cols) return HIMUON_ERR_INVALID_ARGUMENT;
    if (top > kMaxTop) return HIMUON_ERR_UNSUPPORTED;
    if (tokens == nullptr && logp != nullptr) return HIMUON_ERR_INVALID_ARGUMENT;
    if (top > 0 && a.rows > 0 && (top_idx == nullptr || top_logp == nullptr)) return HIMUON_ERR_INVALID_ARGUMENT;
    HIMUON_TRY(arr.add(tokens, a.rows, a.idx64 ? 8 : 4, false));
    HIMUON_TRY(arr.add(logp, a.rows, 4, true));
    HIMUON_TRY(arr.add(entropy, a.rows, 4, true));
    HIMUON_TRY(arr.add(lse, 2 * (int64_t)a.rows, 4, true));
    if (top > 0) {
        HIMUON_TRY(arr.add(top_idx, (int64_t)a.rows * top, 4, true));
        HIMUON_TRY(arr.add(top_logp, (int64_t)a.rows * top, 4, true));
    }
    arr.add(Z, elem_size(dt), false);
    HIMUON_TRY(arr.check());
    HIMUON_TRY(check_workspace(workspace, workspace_bytes,
                               parts_bytes(a.rows, a.plan) + keys_bytes(a.rows, a.plan, top)));
    if (a.rows == 0) return HIMUON_OK;
    a.part = reinterpret_cast<SegStats*>(workspace);
    a.keys = reinterpret_cast<uint64_t*>(reinterpret_cast<char*>(workspace) + parts_bytes(a.rows, a.plan));
    a.tokens = tokens;
    a.top = top;
    a.logp = logp;
    a.entropy = entropy;
    a.lse = lse;
    a.top_idx = top_idx;
    a.top_logp = top_logp;
    const hipError_t e = launch_logprobs(a, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? HIMUON_OK : hip_fail(e);
}

himuon_status_t token_logprobs_grad(const himuon_matrix_t* Z, const void* tokens, himuon_index_t it,
                                    float temperature, const float* lse, const float* entropy, const float* g_logp,
                                    const float* g_entropy, const himuon_matrix_t* dZ, himuon_dtype_t dt,
                                    void* stream) {
    LogitsArgs a{};
    Arrays arr;
    const size_t es = elem_size(dt);
    HIMUON_TRY(logits_args(Z, it, temperature, dt, a));
    if (dZ == nullptr) return HIMUON_ERR_INVALID_ARGUMENT;
    HIMUON_TRY(grad_arg(Z, dZ, es, a));
    if (a.rows > 0 && lse == nullptr) return HIMUON_ERR_INVALID_ARGUMENT;
    if ((g_logp != nullptr && tokens == nullptr) || (g_entropy != nullptr && entropy == nullptr))
        return HIMUON_ERR_INVALID_ARGUMENT;
    HIMUON_TRY(arr.add(tokens, a.rows, a.idx64 ? 8 : 4, false));
    HIMUON_TRY(arr.add(lse, 2 * (int64_t)a.rows, 4, false));
    HIMUON_TRY(arr.add(entropy, a.rows, 4, false));
    HIMUON_TRY(arr.add(g_logp, a.rows, 4, false));
    HIMUON_TRY(arr.add(g_entropy, a.rows, 4, false));
    arr.add(dZ, es, true);
    HIMUON_TRY(arr.check());
    if (a.rows == 0) return HIMUON_OK;
    a.tokens = tokens;
    a.lse = const_cast<float*>(lse);
    a.entropy = const_cast<float*>(entropy);
    a.g_logp = g_logp;
    a.g_entropy = g_entropy;
    const hipError_t e = launch_logprobs_grad(a, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? HIMUON_OK : hip_fail(e);
}

}  // namespace

extern "C" {

himuon_status_t himuon_grouped_mm(const himuon_matrix_t* X, const himuon_matrix_t* W, int32_t n, int32_t trans_w,
                                  const int32_t* ends, const himuon_matrix_t* Y, himuon_dtype_t dt, void* stream) {
    return guarded([&] { return grouped_mm(X, W, n, trans_w, ends, Y, dt, stream); });
}

himuon_status_t himuon_grouped_wgrad(const himuon_matrix_t* X, const himuon_matrix_t* D, const int32_t* ends,
                                     const himuon_matrix_t* G, int32_t n, himuon_dtype_t dt, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    return guarded([&] { return grouped_wgrad(X, D, ends, G, n, dt, workspace, workspace_bytes, stream); });
}

himuon_status_t himuon_grouped_wgrad_workspace(const himuon_matrix_t* X, const himuon_matrix_t* D, int32_t n,
                                               himuon_dtype_t dt, size_t* bytes) {
    if (X == nullptr || D == nullptr || bytes == nullptr || n < 1) return HIMUON_ERR_INVALID_ARGUMENT;
    if (X->rows < 0 || X->rows != D->rows || X->cols < 1 || D->cols < 1) return HIMUON_ERR_INVALID_ARGUMENT;
    for (const int64_t side : {X->rows, X->cols, D->cols})
        if (side > kMaxSide) return HIMUON_ERR_LAYOUT;
    HIMUON_TRY(check_dtype(dt));
    GroupedArgs a{};   // vec = 0: as many parts as any alignment may take
    a.rows = (int32_t)X->rows;
    a.kdim = (int32_t)X->cols;
    a.ndim = (int32_t)D->cols;
    a.dtype = dt == HIMUON_FP32 ? 1 : 0;
    a.total = n;
    *bytes = wgrad_bytes(a);
    return HIMUON_OK;
}

himuon_status_t himuon_distill(const himuon_matrix_t* Z, const void* idx, himuon_index_t it, const himuon_matrix_t* T,
                               float temperature, int32_t normalize, const float* weight, float* loss, float* lse,
                               const himuon_matrix_t* dZ, himuon_dtype_t dt, void* workspace, size_t workspace_bytes,
                               void* stream) {
    return guarded([&] {
        return distill(Z, idx, it, T, temperature, normalize, weight, loss, lse, dZ, dt, workspace, workspace_bytes,
                       stream);
    });
}

himuon_status_t himuon_distill_workspace(const himuon_matrix_t* Z, himuon_dtype_t dt, int32_t with_grad,
                                         size_t* bytes) {
    HIMUON_TRY(check_shape(Z, dt, bytes));
    *bytes = distill_bytes((int32_t)Z->rows, (int32_t)Z->cols, dt == HIMUON_FP32 ? 1 : 0, with_grad != 0);
    return HIMUON_OK;
}

himuon_status_t himuon_distill_grad(const himuon_matrix_t* Z, const void* idx, himuon_index_t it,
                                    const himuon_matrix_t* T, float temperature, int32_t normalize, const float* lse,
                                    const float* g, const himuon_matrix_t* dZ, himuon_dtype_t dt, void* stream) {
    return guarded([&] { return distill_grad(Z, idx, it, T, temperature, normalize, lse, g, dZ, dt, stream); });
}

himuon_status_t himuon_token_logprobs(const himuon_matrix_t* Z, const void* tokens, himuon_index_t it,
                                      float temperature, int32_t top, float* logp, float* entropy, float* lse,
                                      int32_t* top_idx, float* top_logp, himuon_dtype_t dt, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    return guarded([&] {
        return token_logprobs(Z, tokens, it, temperature, top, logp, entropy, lse, top_idx, top_logp, dt, workspace,
                              workspace_bytes, stream);
    });
}

himuon_status_t himuon_token_logprobs_workspace(const himuon_matrix_t* Z, int32_t top, himuon_dtype_t dt,
                                                size_t* bytes) {
    HIMUON_TRY(check_shape(Z, dt, bytes));
    if (top < 0 || top > Z->cols) return HIMUON_ERR_INVALID_ARGUMENT;
    if (top > kMaxTop) return HIMUON_ERR_UNSUPPORTED;
    const SegPlan p = seg_plan((int32_t)Z->rows, (int32_t)Z->cols, dt == HIMUON_FP32 ? 1 : 0);
    *bytes = parts_bytes(Z->rows, p) + keys_bytes(Z->rows, p, top);
    return HIMUON_OK;
}

himuon_status_t himuon_token_logprobs_grad(const himuon_matrix_t* Z, const void* tokens, himuon_index_t it,
                                           float temperature, const float* lse, const float* entropy,
                                           const float* g_logp, const float* g_entropy, const himuon_matrix_t* dZ,
                                           himuon_dtype_t dt, void* stream) {
    return guarded([&] {
        return token_logprobs_grad(Z, tokens, it, temperature, lse, entropy, g_logp, g_entropy, dZ, dt, stream);
    });
}

}  // extern "C"
