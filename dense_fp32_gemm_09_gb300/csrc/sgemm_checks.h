// Argument checks that the C entry points of the operators around the product share.
#pragma once

#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <exception>

#include "sgemm_internal.h"

namespace sgemm {

constexpr int kMaxDim = 1 << 30;

inline int refuse(int status, const char* fmt, ...) {
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    set_last_error_message(msg);
    return status;
}

// No C++ exception leaves a C entry point.
template <typename F>
int guarded(F f) {
    try {
        return f();
    } catch (const std::exception& e) {
        return refuse(SGEMM_ERR_LAUNCH, "exception: %s", e.what());
    } catch (...) {
        return refuse(SGEMM_ERR_LAUNCH, "unknown exception");
    }
}

inline int launched(cudaError_t e, const char* what, int n = 1) {
    if (e == cudaSuccess) {
        count_launches(n);
        return SGEMM_OK;
    }
    set_cuda_error(what, e);
    return SGEMM_ERR_LAUNCH;
}

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
inline int elem_size(int dtype) { return dtype == SGEMM_F32 ? 4 : 2; }

inline int check_dtype(int dtype) {
    if (dtype == SGEMM_F32 || dtype == SGEMM_BF16 || dtype == SGEMM_F16) return SGEMM_OK;
    return refuse(SGEMM_ERR_INVALID_ARG, "unknown element type %d", dtype);
}
inline int check_extent(const char* what, int rows, int cols) {
    if (rows < 0 || cols < 0)
        return refuse(SGEMM_ERR_INVALID_ARG, "%s: negative size %d x %d", what, rows, cols);
    if (rows > kMaxDim || cols > kMaxDim)
        return refuse(SGEMM_ERR_UNSUPPORTED, "%s: dimension above 2^30: %d x %d", what, rows, cols);
    return SGEMM_OK;
}

// A strided matrix argument: name, address, rows, width and leading dimension.
struct Mat {
    const char* name;
    const void* p;
    long long rows, cols, ld;
    int elem;
    long long bytes() const {
        return rows <= 0 || cols <= 0 ? 0 : ((rows - 1) * ld + cols) * elem;
    }
};
inline int check_mat(const Mat& m) {
    if (m.ld < (m.cols > 1 ? m.cols : 1) && m.rows > 1)
        return refuse(SGEMM_ERR_INVALID_ARG, "%s: leading dimension %lld below row width %lld",
                      m.name, m.ld, m.cols);
    if (m.rows > 0 && m.cols > 0 && m.p == nullptr)
        return refuse(SGEMM_ERR_INVALID_ARG, "%s: null pointer with non-empty extent", m.name);
    if (!aligned(m.p, m.elem))
        return refuse(SGEMM_ERR_INVALID_ARG, "%s: not aligned to its %d-byte elements", m.name,
                      m.elem);
    return SGEMM_OK;
}
// Every output apart from every input and from every other output.
template <int NO, int NI>
int check_apart(const Mat (&out)[NO], const Mat (&in)[NI]) {
    for (int o = 0; o < NO; ++o) {
        for (int i = 0; i < NI; ++i)
            if (byte_ranges_overlap(out[o].p, out[o].bytes(), in[i].p, in[i].bytes()))
                return refuse(SGEMM_ERR_INVALID_ARG, "%s overlaps %s", out[o].name, in[i].name);
        for (int i = 0; i < o; ++i)
            if (byte_ranges_overlap(out[o].p, out[o].bytes(), out[i].p, out[i].bytes()))
                return refuse(SGEMM_ERR_INVALID_ARG, "%s overlaps %s", out[o].name, out[i].name);
    }
    return SGEMM_OK;
}

#define SGEMM_TRY(expr)                        \
    do {                                       \
        const int st_ = (expr);                \
        if (st_ != SGEMM_OK) return st_;       \
    } while (0)

}  // namespace sgemm
