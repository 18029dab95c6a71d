// C-ABI entry points of the MXFP4 operators (declared in
// include/gemm_mxfp4.h): argument checks, then one or two launches on the
// caller's stream.

#include "../../include/gemm_mxfp4.h"

#include <initializer_list>

#include "errors.h"
#include "gemm_internal.h"
#include "mxfp4.h"

namespace gemm_f32_impl {
namespace {

// The kernels count rows, columns and k in 32 bits, up to the end of the last tile.
constexpr int64_t kSizeMax = (int64_t{1} << 31) - 1024;
constexpr int64_t kSpanMax = int64_t{1} << 60;  // bytes that one operand may span

struct Bytes {
    uintptr_t lo, hi;
};
bool overlap(Bytes a, Bytes b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

// last + 1 byte of `batch` matrices of `rows` rows, or -1 beyond kSpanMax
int64_t span(int64_t batch, int64_t stride, int64_t rows, int64_t ld, int64_t row_bytes) {
    if (batch <= 0 || rows <= 0 || row_bytes <= 0) return 0;
    const __int128 n = static_cast<__int128>(batch - 1) * stride +
                       static_cast<__int128>(rows - 1) * ld + row_bytes;
    return n > kSpanMax ? -1 : static_cast<int64_t>(n);
}

int check_size(const char *name, int64_t n) {
    if (n < 0) return fail(GEMM_F32_EINVAL, "negative %s %lld", name, (long long)n);
    if (n > kSizeMax) return fail(GEMM_F32_EINVAL, "%s=%lld above 2^31-1024", name, (long long)n);
    return GEMM_F32_OK;
}

// An FP32 operand; `apart`: its matrices must not overlap (it is written).
int check_float(const char *name, const float *p, int64_t batch, int64_t rows, int64_t cols,
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

// An operand in the format.  Rows of scales span whole 4-byte words.
int check_matrix(const char *name, const gemm_mxfp4_matrix *m, int64_t batch, int64_t rows,
                 int64_t cols, bool apart, Bytes *codes, Bytes *scales) {
    *codes = *scales = Bytes{0, 0};
    if (batch == 0 || rows == 0 || cols == 0) return GEMM_F32_OK;
    if (m == nullptr) return fail(GEMM_F32_EINVAL, "%s is NULL", name);
    const int64_t nb = mx::blocks_of(cols), cb = nb * mx::kBlockBytes, sb = (nb + 3) / 4 * 4;
    if (m->codes == nullptr || m->scales == nullptr)
        return fail(GEMM_F32_EINVAL, "codes or scales of %s are NULL", name);
    if (reinterpret_cast<uintptr_t>(m->codes) % 16 || m->ld_codes % 16 || m->stride_codes % 16)
        return fail(GEMM_F32_EINVAL, "codes of %s: pointer, row and batch strides must be multiples of 16",
                    name);
    if (reinterpret_cast<uintptr_t>(m->scales) % 4 || m->ld_scales % 4 || m->stride_scales % 4)
        return fail(GEMM_F32_EINVAL, "scales of %s: pointer, row and batch strides must be multiples of 4",
                    name);
    if (m->ld_codes < cb || m->ld_codes > kSpanMax)
        return fail(GEMM_F32_EINVAL, "ld_codes=%lld of %s outside [%lld, 2^60]",
                    (long long)m->ld_codes, name, (long long)cb);
    if (m->ld_scales < sb || m->ld_scales > kSpanMax)
        return fail(GEMM_F32_EINVAL, "ld_scales=%lld of %s outside [%lld, 2^60]",
                    (long long)m->ld_scales, name, (long long)sb);
    if (m->stride_codes < 0 || m->stride_scales < 0)
        return fail(GEMM_F32_EINVAL, "negative batch stride of %s", name);
    const int64_t one_c = span(1, 0, rows, m->ld_codes, cb), one_s = span(1, 0, rows, m->ld_scales, sb);
    const int64_t nc = span(batch, m->stride_codes, rows, m->ld_codes, cb);
    const int64_t ns = span(batch, m->stride_scales, rows, m->ld_scales, sb);
    if (nc < 0 || ns < 0) return fail(GEMM_F32_EINVAL, "%s spans more than 2^60 bytes", name);
    if (apart && batch > 1 && (m->stride_codes < one_c || m->stride_scales < one_s))
        return fail(GEMM_F32_EINVAL, "batch strides of %s: its matrices overlap", name);
    codes->lo = reinterpret_cast<uintptr_t>(m->codes);
    codes->hi = codes->lo + static_cast<uintptr_t>(nc);
    scales->lo = reinterpret_cast<uintptr_t>(m->scales);
    scales->hi = scales->lo + static_cast<uintptr_t>(ns);
    return GEMM_F32_OK;
}

// No written range may overlap any other range.
int check_apart(std::initializer_list<Bytes> written, std::initializer_list<Bytes> read) {
    for (auto w = written.begin(); w != written.end(); ++w) {
        for (const Bytes &r : read)
            if (overlap(*w, r)) return fail(GEMM_F32_EINVAL, "an output overlaps an input");
        for (auto v = w + 1; v != written.end(); ++v)
            if (overlap(*w, *v)) return fail(GEMM_F32_EINVAL, "two outputs overlap");
    }
    return GEMM_F32_OK;
}

mx::View view_of(const gemm_mxfp4_matrix *m) {
    if (m == nullptr) return {};
    return {static_cast<const uint8_t *>(m->codes), m->ld_codes, m->stride_codes,
            static_cast<const uint8_t *>(m->scales), m->ld_scales, m->stride_scales};
}
mx::Out out_of(const gemm_mxfp4_matrix *m) {
    if (m == nullptr) return {};
    return {static_cast<uint8_t *>(m->codes), m->ld_codes, m->stride_codes,
            static_cast<uint8_t *>(m->scales), m->ld_scales, m->stride_scales};
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

int64_t split_bytes(int splits, int64_t batch, int64_t M, int64_t N) {
    return splits > 1 ? splits * batch * M * N * static_cast<int64_t>(sizeof(float)) : 0;
}
bool plain_sizes(int64_t batch, int64_t M, int64_t N, int64_t K) {
    return batch > 0 && M > 0 && N > 0 && K > 0 && batch <= kSizeMax && M <= kSizeMax &&
           N <= kSizeMax && K <= kSizeMax;
}

// Checks C and the workspace, then runs the product: `weight` picks the kind.
int run_product(bool weight, mx::Product &p, int64_t M, int64_t N, int64_t K, Bytes in0, Bytes in1,
                Bytes in2, Bytes in3, int splits, void *workspace, int64_t workspace_bytes,
                void *stream) {
    Bytes c;
    int rc = check_float("C", p.C, p.batch, M, N, p.ldc, p.sc, true, &c);
    if (rc != GEMM_F32_OK) return rc;
    if (M == 0 || N == 0 || p.batch == 0) return GEMM_F32_OK;
    Bytes w{0, 0};
    p.splits = 1;
    p.W = nullptr;
    if (workspace != nullptr && splits > 1) {
        const int64_t need = split_bytes(splits, p.batch, M, N);
        if (workspace_bytes < need)
            return fail(GEMM_F32_EINVAL, "workspace of %lld bytes needed, %lld given",
                        (long long)need, (long long)workspace_bytes);
        if (reinterpret_cast<uintptr_t>(workspace) % 4)
            return fail(GEMM_F32_EINVAL, "workspace not 4-byte aligned");
        w.lo = reinterpret_cast<uintptr_t>(workspace);
        w.hi = w.lo + static_cast<uintptr_t>(need);
        p.W = static_cast<float *>(workspace);
        p.splits = splits;
    }
    rc = check_apart({c, w}, {in0, in1, in2, in3});
    if (rc != GEMM_F32_OK) return rc;
    return enqueue(stream, [&](hipStream_t s) {
        if (K == 0)
            return launch_zero_fill(p.C, p.M, p.N, p.ldc, static_cast<int>(p.batch), p.sc, s);
        return weight ? mx::launch_weight(p, s) : mx::launch_product(p, s);
    });
}

int check_sizes(int64_t batch, int64_t M, int64_t N, int64_t K) {
    int rc = check_size("batch", batch);
    if (rc == GEMM_F32_OK) rc = check_size("M", M);
    if (rc == GEMM_F32_OK) rc = check_size("N", N);
    if (rc == GEMM_F32_OK) rc = check_size("K", K);
    return rc;
}

}  // namespace
}  // namespace gemm_f32_impl

using namespace gemm_f32_impl;

extern "C" {

int gemm_mxfp4_quantize(int64_t batch, int64_t rows, int64_t cols, const float *X, int64_t ldx,
                        int64_t strideX, const gemm_mxfp4_matrix *Q, const gemm_mxfp4_matrix *QT,
                        void *stream) {
    clear_error();
    int rc = check_size("batch", batch);
    if (rc == GEMM_F32_OK) rc = check_size("rows", rows);
    if (rc == GEMM_F32_OK) rc = check_size("cols", cols);
    if (rc != GEMM_F32_OK) return rc;
    if (Q == nullptr && QT == nullptr) return fail(GEMM_F32_EINVAL, "Q and QT are both NULL");
    Bytes x, qc{0, 0}, qs{0, 0}, tc{0, 0}, ts{0, 0};
    rc = check_float("X", X, batch, rows, cols, ldx, strideX, false, &x);
    if (rc == GEMM_F32_OK && Q) rc = check_matrix("Q", Q, batch, rows, cols, true, &qc, &qs);
    if (rc == GEMM_F32_OK && QT) rc = check_matrix("QT", QT, batch, cols, rows, true, &tc, &ts);
    if (rc == GEMM_F32_OK) rc = check_apart({qc, qs, tc, ts}, {x});
    if (rc != GEMM_F32_OK) return rc;
    if (batch == 0 || rows == 0 || cols == 0) return GEMM_F32_OK;
    const mx::Quantize q{batch, static_cast<int>(rows), static_cast<int>(cols), X, ldx, strideX,
                         Q != nullptr, QT != nullptr, out_of(Q), out_of(QT)};
    return enqueue(stream, [&](hipStream_t s) { return mx::launch_quantize(q, s); });
}

int gemm_mxfp4_dequantize(int64_t batch, int64_t rows, int64_t cols, const gemm_mxfp4_matrix *Q,
                          float *Y, int64_t ldy, int64_t strideY, void *stream) {
    clear_error();
    int rc = check_size("batch", batch);
    if (rc == GEMM_F32_OK) rc = check_size("rows", rows);
    if (rc == GEMM_F32_OK) rc = check_size("cols", cols);
    if (rc != GEMM_F32_OK) return rc;
    Bytes y, qc, qs;
    rc = check_float("Y", Y, batch, rows, cols, ldy, strideY, true, &y);
    if (rc == GEMM_F32_OK) rc = check_matrix("Q", Q, batch, rows, cols, false, &qc, &qs);
    if (rc == GEMM_F32_OK) rc = check_apart({y}, {qc, qs});
    if (rc != GEMM_F32_OK) return rc;
    if (batch == 0 || rows == 0 || cols == 0) return GEMM_F32_OK;
    const mx::Dequantize d{batch, static_cast<int>(rows), static_cast<int>(cols), view_of(Q), Y,
                           ldy, strideY};
    return enqueue(stream, [&](hipStream_t s) { return mx::launch_dequantize(d, s); });
}

int gemm_mxfp4(int64_t batch, int64_t M, int64_t N, int64_t K, const gemm_mxfp4_matrix *A,
               const gemm_mxfp4_matrix *B, float *C, int64_t ldc, int64_t strideC,
               void *workspace, int64_t workspace_bytes, void *stream) {
    clear_error();
    int rc = check_sizes(batch, M, N, K);
    if (rc != GEMM_F32_OK) return rc;
    const int64_t used = M && N ? batch : 0;  // an empty product reads nothing
    Bytes ac, as, bc, bs;
    rc = check_matrix("A", A, used, M, K, false, &ac, &as);
    if (rc == GEMM_F32_OK) rc = check_matrix("B", B, used, N, K, false, &bc, &bs);
    if (rc != GEMM_F32_OK) return rc;
    mx::Product p{};
    p.batch = batch;
    p.M = static_cast<int>(M), p.N = static_cast<int>(N), p.K = static_cast<int>(K);
    p.a = view_of(A), p.b = view_of(B);
    p.b_transposed = true;
    p.C = C, p.ldc = ldc, p.sc = strideC;
    const int splits = plain_sizes(batch, M, N, K) ? mx::product_splits(batch, M, N, K) : 1;
    return run_product(false, p, M, N, K, ac, as, bc, bs, splits, workspace, workspace_bytes,
                       stream);
}

int64_t gemm_mxfp4_workspace_size(int64_t batch, int64_t M, int64_t N, int64_t K) {
    if (!plain_sizes(batch, M, N, K)) return 0;
    return split_bytes(mx::product_splits(batch, M, N, K), batch, M, N);
}

int gemm_mxfp4_weight(int opW, int64_t batch, int64_t M, int64_t N, int64_t K, const float *A,
                      int64_t lda, int64_t strideA, const gemm_mxfp4_matrix *W, float *C,
                      int64_t ldc, int64_t strideC, void *workspace, int64_t workspace_bytes,
                      void *stream) {
    clear_error();
    if (opW != GEMM_F32_OP_N && opW != GEMM_F32_OP_T)
        return fail(GEMM_F32_EINVAL, "opW must be GEMM_F32_OP_N or GEMM_F32_OP_T");
    int rc = check_sizes(batch, M, N, K);
    if (rc != GEMM_F32_OK) return rc;
    const bool t = opW == GEMM_F32_OP_T;
    const int64_t used = M && N ? batch : 0;
    Bytes a, wc, ws;
    rc = check_float("A", A, used, M, K, lda, strideA, false, &a);
    if (rc == GEMM_F32_OK)
        rc = check_matrix("W", W, used, t ? N : K, t ? K : N, false, &wc, &ws);
    if (rc != GEMM_F32_OK) return rc;
    mx::Product p{};
    p.batch = batch;
    p.M = static_cast<int>(M), p.N = static_cast<int>(N), p.K = static_cast<int>(K);
    p.x = A, p.ldx = lda, p.sx = strideA;
    p.b = view_of(W);
    p.b_transposed = t;
    p.C = C, p.ldc = ldc, p.sc = strideC;
    const int splits = plain_sizes(batch, M, N, K) ? mx::weight_splits(t, batch, M, N, K) : 1;
    return run_product(true, p, M, N, K, a, wc, ws, Bytes{0, 0}, splits, workspace,
                       workspace_bytes, stream);
}

int64_t gemm_mxfp4_weight_workspace_size(int opW, int64_t batch, int64_t M, int64_t N, int64_t K) {
    if ((opW != GEMM_F32_OP_N && opW != GEMM_F32_OP_T) || !plain_sizes(batch, M, N, K)) return 0;
    return split_bytes(mx::weight_splits(opW == GEMM_F32_OP_T, batch, M, N, K), batch, M, N);
}

int gemm_mxfp4_abi_version(void) { return 1; }

}  // extern "C"
