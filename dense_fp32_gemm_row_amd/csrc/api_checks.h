// Checks of arguments and the launch on the caller's stream, shared by the
// entry points of gemm_mxfp4.h and gemm_f32_fused.h.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "../../include/gemm_f32.h"
#include "errors.h"

namespace gemm_f32_impl {

// The kernels count rows, columns and k in 32 bits, up to the end of the last tile.
constexpr int64_t kSizeMax = (int64_t{1} << 31) - 1024;
constexpr int64_t kSpanMax = int64_t{1} << 60;  // bytes that one operand may span

struct Bytes {
    uintptr_t lo, hi;
};
inline bool overlap(Bytes a, Bytes b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

// last + 1 byte of `batch` matrices of `rows` rows, or -1 beyond kSpanMax
inline int64_t span(int64_t batch, int64_t stride, int64_t rows, int64_t ld, int64_t row_bytes) {
    if (batch <= 0 || rows <= 0 || row_bytes <= 0) return 0;
    const __int128 n = static_cast<__int128>(batch - 1) * stride +
                       static_cast<__int128>(rows - 1) * ld + row_bytes;
    return n > kSpanMax ? -1 : static_cast<int64_t>(n);
}

inline int check_size(const char *name, int64_t n) {
    if (n < 0) return fail(GEMM_F32_EINVAL, "negative %s %lld", name, (long long)n);
    if (n > kSizeMax) return fail(GEMM_F32_EINVAL, "%s=%lld above 2^31-1024", name, (long long)n);
    return GEMM_F32_OK;
}

// An FP32 operand; `apart`: its matrices must not overlap (it is written).
inline int check_float(const char *name, const float *p, int64_t batch, int64_t rows, int64_t cols,
                int64_t ld, int64_t stride, bool apart, Bytes *out) {
    out->lo = out->hi = reinterpret_cast<uintptr_t>(p);
    if (ld < (cols > 1 ? cols : 1))
        return fail(GEMM_F32_EINVAL, "leading dimension %lld of %s < max(1, %lld)", (long long)ld,
                    name, (long long)cols);
    if (ld > kSpanMax / 8) return fail(GEMM_F32_EINVAL, "leading dimension of %s too large", name);
    if (stride < 0) return fail(GEMM_F32_EINVAL, "negative batch stride of %s", name);
    if (stride > kSpanMax / 8) return fail(GEMM_F32_EINVAL, "batch stride of %s too large", name);
    if (batch == 0 || rows == 0 || cols == 0) return GEMM_F32_OK;
    if (p == nullptr) return fail(GEMM_F32_EINVAL, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % 4)
        return fail(GEMM_F32_EINVAL, "%s not 4-byte aligned", name);
    const int64_t one = span(1, 0, rows, ld * 4, cols * 4);
    const int64_t n = span(batch, stride * 4, rows, ld * 4, cols * 4);
    if (one >= 0 && apart && batch > 1 && stride * 4 < one)
        return fail(GEMM_F32_EINVAL, "batch stride %lld of %s: its matrices overlap",
                    (long long)stride, name);
    if (n < 0) return fail(GEMM_F32_EINVAL, "%s spans more than 2^60 bytes", name);
    out->hi += static_cast<uintptr_t>(n);
    return GEMM_F32_OK;
}

// No written range may overlap any other range.
inline int check_apart(std::initializer_list<Bytes> written, std::initializer_list<Bytes> read) {
    for (auto w = written.begin(); w != written.end(); ++w) {
        for (const Bytes &r : read)
            if (overlap(*w, r)) return fail(GEMM_F32_EINVAL, "an output overlaps an input");
        for (auto v = w + 1; v != written.end(); ++v)
            if (overlap(*w, *v)) return fail(GEMM_F32_EINVAL, "two outputs overlap");
    }
    return GEMM_F32_OK;
}

// Makes the device of `stream` current while it lives.  The null stream and
// the runtime's other predefined handles belong to the current device.
struct OnDeviceOf {
    int back = -1;
    hipError_t err = hipSuccess;
    explicit OnDeviceOf(void *stream) {
        if (reinterpret_cast<uintptr_t>(stream) < 16) return;
        hipDevice_t d = 0;
        int current = 0;
        if ((err = hipGetDevice(&current)) != hipSuccess) return;
        if ((err = hipStreamGetDevice(static_cast<hipStream_t>(stream), &d)) != hipSuccess) return;
        if (static_cast<int>(d) == current) return;
        if ((err = hipSetDevice(static_cast<int>(d))) == hipSuccess) back = current;
    }
    ~OnDeviceOf() {
        if (back >= 0) (void)hipSetDevice(back);
    }
};

template <class F>
int enqueue(void *stream, F launch) {
    OnDeviceOf guard(stream);
    hipError_t err = guard.err;
    if (err == hipSuccess) err = launch(static_cast<hipStream_t>(stream));
    if (err != hipSuccess) return fail(GEMM_F32_EHIP, "launch failed: %s", hipGetErrorString(err));
    return GEMM_F32_OK;
}

}  // namespace gemm_f32_impl
