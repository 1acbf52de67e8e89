// Argument checks shared by the C entry points (api.cpp, api_model.cpp, api_train.cpp).
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <new>
#include <stdexcept>
#include <vector>

#include "himuon.h"

namespace himuon {

// Records e for himuon_last_hip_error (per thread) and returns HIMUON_ERR_HIP.
himuon_status_t hip_fail(hipError_t e);

inline size_t elem_size(himuon_dtype_t dt) { return dt == HIMUON_FP32 ? 4 : 2; }
// Storage is bf16 for HIMUON_BF16 and HIMUON_BF16_PRECISE.
inline bool bf16_storage(himuon_dtype_t dt) { return dt != HIMUON_FP32; }

inline himuon_status_t check_matrix(const himuon_matrix_t& d, size_t es) {
    if (d.ptr == nullptr) return HIMUON_ERR_INVALID_ARGUMENT;
    if (d.rows < 1 || d.cols < 1 || d.ld < d.cols) return HIMUON_ERR_INVALID_ARGUMENT;
    if (d.rows > INT32_MAX || d.cols > INT32_MAX) return HIMUON_ERR_LAYOUT;
    if ((reinterpret_cast<uintptr_t>(d.ptr) % es) != 0) return HIMUON_ERR_LAYOUT;
    // extent in bytes must fit in int64
    const double ext = ((double)(d.rows - 1) * (double)d.ld + (double)d.cols) * (double)es;
    if (ext > 9.0e18) return HIMUON_ERR_LAYOUT;
    return HIMUON_OK;
}

struct Extent {
    uintptr_t lo, hi;  // [lo, hi) bytes
    int64_t ld, cols;
    int64_t rows;
    size_t es;
    int id;
};

// True if two matrices share an element.  Byte ranges that overlap can still
// be disjoint when both use the same row stride and occupy different column
// ranges of the same rows (column blocks of one fused tensor).
inline bool share_element(const Extent& a, const Extent& b) {
    if (a.hi <= b.lo || b.hi <= a.lo) return false;
    if (a.ld != b.ld || a.es != b.es) return true;
    const Extent& x = a.lo <= b.lo ? a : b;
    const Extent& y = a.lo <= b.lo ? b : a;
    const uintptr_t d = y.lo - x.lo;
    const uintptr_t row_bytes = (uintptr_t)x.ld * x.es;
    if (d % x.es != 0) return true;
    const int64_t dc = (int64_t)((d % row_bytes) / x.es);   // column offset of y inside x's rows
    // y's columns [dc, dc + y.cols) must avoid x's [0, x.cols) in every row both touch,
    // including y rows that wrap past ld.
    if (dc < x.cols) return true;
    if (dc + y.cols > x.ld) return true;   // wraps into x's next row
    return false;
}

inline himuon_status_t check_overlap(std::vector<Extent>& ex) {
    std::sort(ex.begin(), ex.end(), [](const Extent& a, const Extent& b) { return a.lo < b.lo; });
    for (size_t i = 0; i < ex.size(); ++i)
        for (size_t j = i + 1; j < ex.size() && ex[j].lo < ex[i].hi; ++j)
            if (share_element(ex[i], ex[j])) return HIMUON_ERR_OVERLAP;
    return HIMUON_OK;
}

inline Extent extent_of(const himuon_matrix_t& d, size_t es, int id) {
    Extent e;
    e.lo = reinterpret_cast<uintptr_t>(d.ptr);
    e.hi = e.lo + (uintptr_t)(((d.rows - 1) * d.ld + d.cols) * (int64_t)es);
    e.ld = d.ld;
    e.cols = d.cols;
    e.rows = d.rows;
    e.es = es;
    e.id = id;
    return e;
}

// ---- the operators around the optimiser step
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

inline himuon_status_t check_dtype(himuon_dtype_t dt) {
    return dt == HIMUON_BF16 || dt == HIMUON_FP32 ? HIMUON_OK : HIMUON_ERR_UNSUPPORTED;
}

// A matrix whose rows are tokens: as check_matrix, but it may have no rows.
inline himuon_status_t check_rows(const himuon_matrix_t& d, size_t es) {
    if (d.rows != 0) return check_matrix(d, es);
    if (d.cols < 1 || d.ld < d.cols) return HIMUON_ERR_INVALID_ARGUMENT;
    return d.cols > INT32_MAX ? HIMUON_ERR_LAYOUT : HIMUON_OK;
}

inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Rows of whole 16-byte chunks, and 256 of them within 32-bit byte offsets.
inline bool chunked(const himuon_matrix_t& d) { return aligned(d.ptr, 16) && d.ld % 8 == 0 && d.ld <= (1 << 22); }

// Byte range of a contiguous device array, as an extent of one row.
inline Extent array_extent(const void* p, int64_t bytes) {
    return extent_of(himuon_matrix_t{const_cast<void*>(p), 1, bytes, bytes}, 1, 0);
}

#define HIMUON_TRY(call)                           \
    do {                                           \
        const himuon_status_t st_ = (call);        \
        if (st_ != HIMUON_OK) return st_;          \
    } while (0)

inline himuon_status_t check_workspace(const void* ws, size_t bytes, size_t need) {
    if (need == 0) return HIMUON_OK;
    if (ws == nullptr || bytes < need) return HIMUON_ERR_WORKSPACE;
    return aligned(ws, 16) ? HIMUON_OK : HIMUON_ERR_LAYOUT;
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

}  // namespace himuon
