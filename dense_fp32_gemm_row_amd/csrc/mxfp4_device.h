// Device helpers of the MXFP4 kernels.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "device_common.h"
#include "gemm_internal.h"
#include "mxfp4.h"

namespace gemm_f32_impl {
namespace mx {

// The conversion instructions take a scale as a float and use its exponent
// byte alone: 0 is 2^-127 and 255 NaN, as in the format.
__device__ __forceinline__ float scale_of(uint32_t e) { return __builtin_bit_cast(float, e << 23); }

typedef __attribute__((address_space(3))) void *lptr_t;

constexpr int kStream = 2;  // cache policy of buffer stores: non-temporal

// A buffer of `bytes` bytes from p: loads past its end give zeros, stores
// there are dropped.
constexpr int kOutside = static_cast<int>(0x80000000u);  // an offset past every buffer
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0,
                                             static_cast<int>(min(bytes, int64_t{0x7fffffff})),
                                             0x00020000);
}

// Stores the first min(V, left) of a lane's V (4 or 2) neighbours of a row at
// byte `at` of the buffer.
template <int V>
__device__ __forceinline__ void store_neighbours(const float (&v)[V], __amdgpu_buffer_rsrc_t to, int at,
                                                 int left) {
    static_assert(V == 4 || V == 2, "");
    if (left >= V) {
        if constexpr (V == 4)
            __builtin_amdgcn_raw_buffer_store_b128(
                __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}), to, at, 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, f32x2{v[0], v[1]}), to, at, 0, 0);
    } else {
#pragma unroll
        for (int j = 0; j < V - 1; ++j)
            if (j < left) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v[j]), to, at + 4 * j, 0, 0);
    }
}

// Rows of an operand from a tile's first one, as a buffer: offsets past the
// operand's last byte, as the rows past an edge make, read as zeros.
struct Rows {
    __amdgpu_buffer_rsrc_t rsrc;
    int ld;
};
__device__ __forceinline__ Rows rows_from(const uint8_t *base, int64_t ld, int first, int rows,
                                          int row_bytes) {
    return {buffer_of(base + first * ld, (rows - 1 - first) * ld + row_bytes), static_cast<int>(ld)};
}

// One tile of one product (one slice of K of it), as a workgroup meets it:
// tiles of 8 rows of tiles are consecutive, K is `chunks` chunks, `len` a slice.
struct Place {
    int64_t slice;  // batch * splits + split
    int m0, n0, g0, g1;  // first row and column, chunks of K [g0, g1)
};

template <int BM, int BN>
__device__ __forceinline__ Place place_of(const Product &p, int64_t id, int tiles_m, int tiles_n,
                                          int chunks, int len) {
    const int per = tiles_m * tiles_n;
    Place q;
    q.slice = id / per;
    int tm, tn;
    grouped_tile(static_cast<int>(id - q.slice * per), tiles_m, tiles_n, 8, tm, tn);
    q.m0 = tm * BM;
    q.n0 = tn * BN;
    const int split = static_cast<int>(q.slice % p.splits);
    q.g0 = split * len;
    q.g1 = min(q.g0 + len, chunks);
    return q;
}

}  // namespace mx
}  // namespace gemm_f32_impl
