// C entry points of layer normalisation and of the AdamW step.  Argument checks
// and launches; see include/himuon.h for the contract.
#include <cmath>
#include <utility>

#include "adamw.h"
#include "api_util.h"
#include "norm.h"

using namespace himuon;

static_assert(kMaxNormCols == HIMUON_MAX_NORM_COLS && kAdamwBlock == HIMUON_ADAMW_BLOCK, "limits of the header");

namespace {

// ---- layer normalisation -----------------------------------------------------------
himuon_status_t norm_args(const himuon_matrix_t* X, himuon_dtype_t dt, NormArgs& a) {
    HIMUON_TRY(check_dtype(dt));
    if (X == nullptr) return HIMUON_ERR_INVALID_ARGUMENT;
    HIMUON_TRY(check_rows(*X, elem_size(dt)));
    if (X->cols > kMaxNormCols) return HIMUON_ERR_UNSUPPORTED;
    a.x = X->ptr;
    a.x_ld = X->ld;
    a.rows = (int32_t)X->rows;
    a.cols = (int32_t)X->cols;
    a.dtype = dt == HIMUON_FP32 ? 1 : 0;
    return HIMUON_OK;
}

bool same_place(const himuon_matrix_t* a, const himuon_matrix_t* b) { return a->ptr == b->ptr && a->ld == b->ld; }
bool same_shape(const himuon_matrix_t* a, const himuon_matrix_t* b) { return a->rows == b->rows && a->cols == b->cols; }

himuon_status_t layer_norm(const himuon_matrix_t* X, const void* weight, const void* bias, float eps,
                           const himuon_matrix_t* Y, float* stats, himuon_dtype_t dt, void* stream) {
    NormArgs a{};
    Arrays arr;
    const size_t es = elem_size(dt);
    HIMUON_TRY(norm_args(X, dt, a));
    if (Y == nullptr || !(eps >= 0.f) || !std::isfinite(eps)) return HIMUON_ERR_INVALID_ARGUMENT;
    HIMUON_TRY(check_rows(*Y, es));
    if (!same_shape(X, Y)) return HIMUON_ERR_INVALID_ARGUMENT;
    HIMUON_TRY(arr.add(weight, a.cols, es, false));
    HIMUON_TRY(arr.add(bias, a.cols, es, false));
    HIMUON_TRY(arr.add(stats, 2 * (int64_t)a.rows, 4, true));
    if (!aligned(stats, 8)) return HIMUON_ERR_LAYOUT;
    arr.add(Y, es, true);
    if (!same_place(X, Y)) arr.add(X, es, false);
    HIMUON_TRY(arr.check());
    if (a.rows == 0) return HIMUON_OK;
    a.weight = weight;
    a.bias = bias;
    a.eps = eps;
    a.y = Y->ptr;
    a.y_ld = Y->ld;
    a.stats = stats;
    const hipError_t e = launch_layer_norm(a, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? HIMUON_OK : hip_fail(e);
}

himuon_status_t layer_norm_grad(const himuon_matrix_t* X, const void* weight, const float* stats,
                                const himuon_matrix_t* dY, const himuon_matrix_t* dX, void* dweight, void* dbias,
                                himuon_dtype_t dt, void* workspace, size_t workspace_bytes, void* stream) {
    NormArgs a{};
    Arrays arr;
    const size_t es = elem_size(dt);
    HIMUON_TRY(norm_args(X, dt, a));
    if (dY == nullptr || (a.rows > 0 && stats == nullptr)) return HIMUON_ERR_INVALID_ARGUMENT;
    HIMUON_TRY(check_rows(*dY, es));
    if (!same_shape(X, dY)) return HIMUON_ERR_INVALID_ARGUMENT;
    if (dX != nullptr) {
        HIMUON_TRY(check_rows(*dX, es));
        if (!same_shape(X, dX)) return HIMUON_ERR_INVALID_ARGUMENT;
        arr.add(dX, es, true);
    }
    if (dX == nullptr || !same_place(X, dX)) arr.add(X, es, false);
    if (dX == nullptr || !same_place(dY, dX)) arr.add(dY, es, false);
    HIMUON_TRY(arr.add(weight, a.cols, es, false));
    HIMUON_TRY(arr.add(stats, 2 * (int64_t)a.rows, 4, false));
    if (!aligned(stats, 8)) return HIMUON_ERR_LAYOUT;
    HIMUON_TRY(arr.add(dweight, a.cols, es, true));
    HIMUON_TRY(arr.add(dbias, a.cols, es, true));
    const bool sums = dweight != nullptr || dbias != nullptr;
    if (sums) {
        const int64_t need = norm_grad_bytes(a.rows, a.cols, a.dtype);
        HIMUON_TRY(check_workspace(workspace, workspace_bytes, (size_t)need));
        HIMUON_TRY(arr.add(workspace, need, 1, true));
    }
    HIMUON_TRY(arr.check());
    if (!sums && (dX == nullptr || a.rows == 0)) return HIMUON_OK;
    a.weight = weight;
    a.stats = const_cast<float*>(stats);
    a.dy = dY->ptr;
    a.dy_ld = dY->ld;
    a.dx = dX != nullptr ? dX->ptr : nullptr;
    a.dx_ld = dX != nullptr ? dX->ld : 0;
    a.dw = dweight;
    a.db = dbias;
    a.part = sums ? reinterpret_cast<float*>(workspace) : nullptr;
    const hipError_t e = launch_layer_norm_grad(a, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? HIMUON_OK : hip_fail(e);
}

// ---- AdamW -------------------------------------------------------------------------
// Whether any extent that is written shares memory with another one.  The extents
// come in runs (one for each kind of operand).  Where every run is in the order of its
// addresses and apart from the other runs, as flat buffers are, there is nothing to sort.
bool plainly_apart(const std::vector<Extent>& ex, size_t run) {
    std::vector<std::pair<uintptr_t, uintptr_t>> spans;
    for (size_t from = 0; from < ex.size(); from += run) {
        const size_t to = std::min(from + run, ex.size());
        for (size_t i = from + 1; i < to; ++i)
            if (ex[i].lo < ex[i - 1].hi) return false;
        spans.emplace_back(ex[from].lo, ex[to - 1].hi);
    }
    std::sort(spans.begin(), spans.end());
    for (size_t i = 1; i < spans.size(); ++i)
        if (spans[i].first < spans[i - 1].second) return false;
    return true;
}
himuon_status_t check_apart(const std::vector<Extent>& ex, size_t run) {
    if (plainly_apart(ex, run)) return HIMUON_OK;
    struct At {
        uintptr_t lo;
        uint32_t i;
    };
    std::vector<At> at(ex.size());
    for (size_t i = 0; i < ex.size(); ++i) at[i] = {ex[i].lo, (uint32_t)i};
    const auto less = [](const At& a, const At& b) { return a.lo < b.lo; };
    for (size_t from = 0; from < at.size(); from += run) {
        const auto b = at.begin() + from, e = at.begin() + std::min(from + run, at.size());
        if (!std::is_sorted(b, e, less)) std::sort(b, e, less);
        std::inplace_merge(at.begin(), b, e, less);
    }
    for (size_t i = 0; i < at.size(); ++i)
        for (size_t j = i + 1; j < at.size() && at[j].lo < ex[at[i].i].hi; ++j) {
            const Extent &a = ex[at[i].i], &b = ex[at[j].i];
            if ((a.id != 0 || b.id != 0) && share_element(a, b)) return HIMUON_ERR_OVERLAP;
        }
    return HIMUON_OK;
}

himuon_status_t adamw_step(const himuon_matrix_t* W, const himuon_matrix_t* G, const himuon_adamw_state_t* S, int32_t n,
                           int32_t bits, double lr, double beta1, double beta2, double eps, double weight_decay,
                           int64_t step, const float* grad_scale, himuon_dtype_t w_dt, himuon_dtype_t g_dt,
                           void* stream) {
    HIMUON_TRY(check_dtype(w_dt));
    HIMUON_TRY(check_dtype(g_dt));
    if (bits != 8 && bits != 32) return HIMUON_ERR_UNSUPPORTED;
    if (n < 0 || (n > 0 && (W == nullptr || G == nullptr || S == nullptr))) return HIMUON_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(lr) || !std::isfinite(weight_decay) || !(beta1 >= 0. && beta1 < 1.) ||
        !(beta2 >= 0. && beta2 < 1.) || !(eps >= 1.2e-38) || !std::isfinite((float)eps) || step < 1)
        return HIMUON_ERR_INVALID_ARGUMENT;
    if (!aligned(grad_scale, 4)) return HIMUON_ERR_LAYOUT;
    const size_t ws = elem_size(w_dt), gs = elem_size(g_dt);
    std::vector<Extent> ex;
    ex.reserve((size_t)n * 6 + 1);
    // by kind, so that each kind is in the order of its addresses where the tensors are
    for (int32_t i = 0; i < n; ++i) {
        HIMUON_TRY(check_matrix(W[i], ws));
        ex.push_back(extent_of(W[i], ws, 1));
    }
    for (int32_t i = 0; i < n; ++i) {
        HIMUON_TRY(check_matrix(G[i], gs));
        if (!same_shape(&W[i], &G[i])) return HIMUON_ERR_INVALID_ARGUMENT;
        ex.push_back(extent_of(G[i], gs, 0));
    }
    const auto add = [&](const void* p, int64_t bytes, size_t es) {
        if (p == nullptr) return HIMUON_ERR_INVALID_ARGUMENT;
        if (!aligned(p, es)) return HIMUON_ERR_LAYOUT;
        Extent e = array_extent(p, bytes);
        e.id = 1;
        ex.push_back(e);
        return HIMUON_OK;
    };
    const auto numel = [&](int32_t i) { return W[i].rows * W[i].cols; };
    const auto blocks = [&](int32_t i) { return (numel(i) + kAdamwBlock - 1) / kAdamwBlock; };
    const size_t ss = bits / 8;
    for (int32_t i = 0; i < n; ++i) HIMUON_TRY(add(S[i].m, numel(i) * (int64_t)ss, ss));
    for (int32_t i = 0; i < n; ++i) HIMUON_TRY(add(S[i].v, numel(i) * (int64_t)ss, ss));
    if (bits == 8) {
        for (int32_t i = 0; i < n; ++i) HIMUON_TRY(add(S[i].m_scale, blocks(i) * 4, 4));
        for (int32_t i = 0; i < n; ++i) HIMUON_TRY(add(S[i].v_scale, blocks(i) * 4, 4));
    }
    const size_t run = (size_t)n;
    if (n > 0 && grad_scale != nullptr) ex.push_back(array_extent(grad_scale, 4));
    if (n > 0) HIMUON_TRY(check_apart(ex, run));

    AdamwArgs a;
    a.w_dtype = w_dt == HIMUON_FP32 ? 1 : 0;
    a.g_dtype = g_dt == HIMUON_FP32 ? 1 : 0;
    a.bits = bits;
    uint32_t k = (uint32_t)step * 0x9AD24435u + 0xB3B07CC5u;
    a.key = (k ^ (k >> 16)) * 0xB06A350Du;
    a.beta1 = (float)beta1;
    a.rest1 = (float)(1. - beta1);
    a.beta2 = (float)beta2;
    a.rest2 = (float)(1. - beta2);
    a.keep = (float)(1. - lr * weight_decay);
    a.rate = (float)(lr / (1. - std::pow(beta1, (double)step)));
    a.root = (float)(1. / std::sqrt(1. - std::pow(beta2, (double)step)));
    a.eps = (float)eps;
    a.grad_scale = grad_scale;
    // tensors whose units one launch can count
    const auto units = [&](int32_t i) { return (numel(i) + kAdamwUnit - 1) / kAdamwUnit; };
    for (int32_t i = 0; i < n; ++i)
        if (units(i) > INT32_MAX) return HIMUON_ERR_LAYOUT;
    for (int32_t i = 0; i < n;) {
        a.n = 0;
        a.units = 0;
        for (; i < n && a.n < kAdamwTensors && a.units + units(i) <= INT32_MAX; ++i) {
            AdamwTensor& t = a.t[a.n++];
            t.w = W[i].ptr;
            t.g = G[i].ptr;
            t.m = S[i].m;
            t.v = S[i].v;
            t.m_scale = bits == 8 ? S[i].m_scale : nullptr;
            t.v_scale = bits == 8 ? S[i].v_scale : nullptr;
            t.numel = numel(i);
            const auto dense = [](const himuon_matrix_t& d) { return d.rows == 1 || d.ld == d.cols; };
            t.cols = dense(W[i]) && dense(G[i]) ? 0 : W[i].cols;
            t.w_ld = W[i].ld;
            t.g_ld = G[i].ld;
            t.first = a.units;
            a.units += (uint32_t)units(i);
        }
        const hipError_t e = launch_adamw(a, reinterpret_cast<hipStream_t>(stream));
        if (e != hipSuccess) return hip_fail(e);
    }
    return HIMUON_OK;
}

}  // namespace

extern "C" {

himuon_status_t himuon_layer_norm(const himuon_matrix_t* X, const void* weight, const void* bias, float eps,
                                  const himuon_matrix_t* Y, float* stats, himuon_dtype_t dt, void* stream) {
    return guarded([&] { return layer_norm(X, weight, bias, eps, Y, stats, dt, stream); });
}

himuon_status_t himuon_layer_norm_grad(const himuon_matrix_t* X, const void* weight, const float* stats,
                                       const himuon_matrix_t* dY, const himuon_matrix_t* dX, void* dweight,
                                       void* dbias, himuon_dtype_t dt, void* workspace, size_t workspace_bytes,
                                       void* stream) {
    return guarded([&] {
        return layer_norm_grad(X, weight, stats, dY, dX, dweight, dbias, dt, workspace, workspace_bytes, stream);
    });
}

himuon_status_t himuon_layer_norm_grad_workspace(const himuon_matrix_t* X, himuon_dtype_t dt, size_t* bytes) {
    if (X == nullptr || bytes == nullptr || X->rows < 0 || X->cols < 1) return HIMUON_ERR_INVALID_ARGUMENT;
    HIMUON_TRY(check_dtype(dt));
    if (X->rows > INT32_MAX) return HIMUON_ERR_LAYOUT;
    if (X->cols > kMaxNormCols) return HIMUON_ERR_UNSUPPORTED;
    *bytes = (size_t)norm_grad_bytes((int32_t)X->rows, (int32_t)X->cols, dt == HIMUON_FP32 ? 1 : 0);
    return HIMUON_OK;
}

himuon_status_t himuon_adamw_step(const himuon_matrix_t* W, const himuon_matrix_t* G, const himuon_adamw_state_t* S,
                                  int32_t n, int32_t bits, double lr, double beta1, double beta2, double eps,
                                  double weight_decay, int64_t step, const float* grad_scale, himuon_dtype_t w_dt,
                                  himuon_dtype_t g_dt, void* stream) {
    return guarded([&] {
        return adamw_step(W, G, S, n, bits, lr, beta1, beta2, eps, weight_decay, step, grad_scale, w_dt, g_dt, stream);
    });
}

}  // extern "C"
