// Argument checks shared by the C entry points (api.cpp, api_model.cpp).
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
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

}  // namespace himuon
