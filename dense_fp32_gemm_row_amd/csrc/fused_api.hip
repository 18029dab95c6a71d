// C-ABI entry points of the fused operators (declared in
// include/gemm_f32_fused.h): argument checks, a workspace's parts, then
// launches on the caller's stream.

#include "../../include/gemm_f32_fused.h"

#include <algorithm>

#include "api_checks.h"
#include "errors.h"
#include "fused.h"
#include "gemm_internal.h"

namespace gemm_f32_impl {
namespace {

using fused::div_up;

bool known_op(int op) { return op == GEMM_F32_OP_N || op == GEMM_F32_OP_T; }
bool known_activation(int a) { return a >= GEMM_F32_ACT_NONE && a <= GEMM_F32_ACT_SILU; }

// Sizes of workspaces saturate: more than kSpanMax is refused wherever it is met.
int64_t times(int64_t a, int64_t b) {
    const __int128 n = static_cast<__int128>(a) * b;
    return n > 2 * static_cast<__int128>(kSpanMax) ? 2 * kSpanMax : static_cast<int64_t>(n);
}
int64_t plus(int64_t a, int64_t b) { return std::min(a + b, 2 * kSpanMax); }

int check_op(const char *name, int op) {
    if (known_op(op)) return GEMM_F32_OK;
    return fail(GEMM_F32_EINVAL, "%s must be GEMM_F32_OP_N or GEMM_F32_OP_T", name);
}
int check_activation(int a) {
    if (known_activation(a)) return GEMM_F32_OK;
    return fail(GEMM_F32_EINVAL, "activation %d is none of GEMM_F32_ACT_*", a);
}
int check_sizes(int64_t batch, int64_t M, int64_t N, int64_t K) {
    int rc = check_size("batch", batch);
    if (rc == GEMM_F32_OK) rc = check_size("M", M);
    if (rc == GEMM_F32_OK) rc = check_size("N", N);
    if (rc == GEMM_F32_OK) rc = check_size("K", K);
    return rc;
}
bool valid_sizes(int64_t batch, int64_t M, int64_t N, int64_t K) {
    return batch >= 0 && M >= 0 && N >= 0 && K >= 0 && batch <= kSizeMax && M <= kSizeMax && N <= kSizeMax &&
           K <= kSizeMax;
}
int check_workspace(void *workspace, int64_t bytes, int64_t need, Bytes *out) {
    *out = Bytes{0, 0};
    if (need == 0) return GEMM_F32_OK;
    if (need > kSpanMax) return fail(GEMM_F32_EINVAL, "a workspace of more than 2^60 bytes needed");
    if (workspace == nullptr || bytes < need)
        return fail(GEMM_F32_EINVAL, "workspace of %lld bytes needed, %lld given", (long long)need,
                    (long long)(workspace == nullptr ? 0 : bytes));
    if (reinterpret_cast<uintptr_t>(workspace) % 4)
        return fail(GEMM_F32_EINVAL, "workspace not 4-byte aligned");
    out->lo = reinterpret_cast<uintptr_t>(workspace);
    out->hi = out->lo + static_cast<uintptr_t>(need);
    return GEMM_F32_OK;
}

// Bytes of a product's own workspace, and of two.
int64_t space_of(bool tb, int64_t batch, int64_t M, int64_t N, int64_t K, fused::Use use = fused::kPlain) {
    if (batch == 0 || M == 0 || N == 0 || K == 0) return 0;
    return fused::product_space(tb, batch, M, N, K, use);
}

int64_t space_of(const fused::Sizes &p, const fused::Sizes &q) {
    auto one = [](const fused::Sizes &x) { return space_of(x.tb, x.batch, x.M, x.N, x.K, x.use); };
    auto empty = [](const fused::Sizes &x) { return x.batch == 0 || x.M == 0 || x.N == 0 || x.K == 0; };
    return empty(p) || empty(q) ? std::max(one(p), one(q)) : fused::two_space(p, q);
}

fused::Product plain_product(int64_t batch, int64_t M, int64_t N, int64_t K, bool ta, fused::Operand a, bool tb,
                             fused::Operand b, fused::Result c, float *space, fused::Use use = fused::kPlain) {
    fused::Product p{};
    p.batch = batch;
    p.M = static_cast<int>(M), p.N = static_cast<int>(N), p.K = static_cast<int>(K);
    p.ta = ta, p.tb = tb;
    p.a = a, p.b = b, p.c = c;
    p.space = space;
    p.mode = fused::kStore;
    p.use = use;
    return p;
}

// A launch function's product, unless it is empty.
hipError_t run(const fused::Product &p, hipStream_t s) {
    if (p.batch == 0 || p.M == 0 || p.N == 0) return hipSuccess;
    return fused::launch_product(p, s);
}

hipError_t run(const fused::Product &p, const fused::Product &q, int64_t bytes, hipStream_t s) {
    auto empty = [](const fused::Product &x) { return x.batch == 0 || x.M == 0 || x.N == 0; };
    if (!empty(p) && !empty(q)) return fused::launch_two(p, q, bytes, s);
    return empty(p) ? run(q, s) : run(p, s);
}

// ---- the parts of a gradient's workspace, in floats ----
struct GradParts {
    int64_t dz, partial, space;
    int blocks, rows;
    int64_t bytes() const { return times(4, plus(plus(dz, partial), space)); }
};
GradParts grad_parts(bool ta, bool tb, int64_t batch, int64_t M, int64_t N, int64_t K, int activation, bool dA, bool dB,
                     bool dbias) {
    GradParts g{};
    // blocks of rows of the bias gradient's first sums: enough to fill the GPU
    const int64_t strips = std::max<int64_t>(1, times(batch, div_up(N, 256)));
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(fused::kSlopeBlocks, 1024 / strips));
    // a few rows of not too many columns: one block, whose sums need no second launch
    const bool one = M <= 256 && times(times(batch, M), N) <= 1 << 18;
    g.rows = static_cast<int>(one ? std::max<int64_t>(1, M) : std::max<int64_t>(8, div_up(M, most)));
    g.blocks = static_cast<int>(div_up(M, g.rows));
    if (activation != GEMM_F32_ACT_NONE && (dA || dB)) g.dz = times(times(batch, M), N);
    if (dbias && g.blocks > 1) g.partial = times(times(batch, g.blocks), N);
    // the products as they are run
    const fused::Sizes none{}, a = ta ? fused::Sizes{tb, true, batch, K, M, N, fused::kPlain}
                                             : fused::Sizes{false, !tb, batch, M, K, N, fused::kPlain};
    const fused::Sizes b = tb ? fused::Sizes{true, ta, batch, N, K, M, fused::kPlain}
                              : fused::Sizes{!ta, false, batch, K, N, M, fused::kPlain};
    g.space = space_of(dA ? a : none, dB ? b : none) / 4;
    return g;
}

// ---- the parts of a cross entropy's workspace ----
int groups_of(int64_t T, int64_t V) { return static_cast<int>(div_up(V, fused::group_columns(T))); }
int64_t stats_bytes(int64_t T, int64_t V) {  // logit at the target, lse, statistics
    return plus(times(times(8, T), groups_of(T, V)), times(8, T));
}
// Logits are held in whole lines, from a line's start where the workspace begins at one.
int64_t line(int64_t floats) { return div_up(floats, 32) * 32; }
// The gradient works on at most `rows` tokens at a time, whose logits it holds.  (A
// last piece of few tokens has statistics of more groups.)
int64_t piece_bytes(int64_t rows, int64_t V) {
    if (rows == 0) return 0;
    const int64_t few = std::min<int64_t>(rows, fused::kFineTokens);
    return plus(times(times(4, rows), line(V)) + 4 * 32,
                std::max(stats_bytes(rows, V), stats_bytes(few, V)));
}
int64_t piece_space(int64_t rows, int64_t V, int64_t K) {
    return std::max(space_of(true, 1, rows, V, K, fused::kStatistics),
                    space_of(fused::Sizes{false, false, 1, rows, K, V, fused::kProbabilities},
                             fused::Sizes{true, false, 1, V, K, rows, fused::kProbabilities}));
}
constexpr int64_t kPieceBytes = int64_t{4} << 30;
constexpr int64_t kPieceRows = 256;
int64_t piece_rows(int64_t T, int64_t V) {
    if (T <= kPieceRows) return T;
    int64_t rows = kPieceBytes / std::max<int64_t>(1, times(4, line(V))) / kPieceRows * kPieceRows;
    rows = std::max(rows, kPieceRows);
    if (rows >= T) return T;
    // pieces of about the same size, whole tiles
    return div_up(div_up(T, div_up(T, rows)), kPieceRows) * kPieceRows;
}
int64_t piece_least(int64_t T) { return std::min<int64_t>(T, 64); }

int check_tokens(int64_t T, int64_t V, int64_t K, const float *X, int64_t ldx, const float *W, int64_t ldw,
                 const int64_t *target, Bytes *x, Bytes *w, Bytes *t) {
    int rc = check_size("T", T);
    if (rc == GEMM_F32_OK) rc = check_size("V", V);
    if (rc == GEMM_F32_OK) rc = check_size("K", K);
    if (rc != GEMM_F32_OK) return rc;
    if (V == 0 && T > 0) return fail(GEMM_F32_EINVAL, "an empty vocabulary");
    rc = check_float("X", X, 1, T, K, ldx, 0, false, x);
    if (rc == GEMM_F32_OK) rc = check_float("W", W, T ? 1 : 0, V, K, ldw, 0, false, w);
    if (rc != GEMM_F32_OK) return rc;
    t->lo = t->hi = reinterpret_cast<uintptr_t>(target);
    if (T == 0) return GEMM_F32_OK;
    if (target == nullptr) return fail(GEMM_F32_EINVAL, "target is NULL");
    if (t->lo % 8) return fail(GEMM_F32_EINVAL, "target not 8-byte aligned");
    t->hi += static_cast<uintptr_t>(8 * T);
    return GEMM_F32_OK;
}
int check_vector(const char *name, const float *p, int64_t n, Bytes *out) {
    *out = Bytes{0, 0};
    return p == nullptr ? GEMM_F32_OK : check_float(name, p, 1, 1, n, std::max<int64_t>(n, 1), 0, false, out);
}

}  // namespace
}  // namespace gemm_f32_impl

using namespace gemm_f32_impl;

extern "C" {

int gemm_f32_fused(int opA, int opB, int64_t batch, int64_t M, int64_t N, int64_t K, const float *A, int64_t lda,
                   int64_t strideA, const float *B, int64_t ldb, int64_t strideB, const gemm_f32_epilogue *epilogue,
                   float *C, int64_t ldc, int64_t strideC, void *workspace, int64_t workspace_bytes, void *stream) {
    clear_error();
    int rc = check_op("opA", opA);
    if (rc == GEMM_F32_OK) rc = check_op("opB", opB);
    const gemm_f32_epilogue none{};
    const gemm_f32_epilogue &e = epilogue != nullptr ? *epilogue : none;
    if (rc == GEMM_F32_OK) rc = check_activation(e.activation);
    if (rc == GEMM_F32_OK) rc = check_sizes(batch, M, N, K);
    if (rc != GEMM_F32_OK) return rc;
    const bool ta = opA == GEMM_F32_OP_T, tb = opB == GEMM_F32_OP_T;
    const int64_t used = M && N ? batch : 0;  // an empty product reads nothing
    Bytes a, b, bias, residual{0, 0}, c, pre{0, 0}, w{0, 0};
    rc = check_float("A", A, used, ta ? K : M, ta ? M : K, lda, strideA, false, &a);
    if (rc == GEMM_F32_OK) rc = check_float("B", B, used, tb ? N : K, tb ? K : N, ldb, strideB, false, &b);
    if (rc == GEMM_F32_OK) rc = check_float("C", C, batch, M, N, ldc, strideC, true, &c);
    bias = Bytes{0, 0};
    if (rc == GEMM_F32_OK && e.bias != nullptr)
        rc = check_float("bias", e.bias, used, 1, N, std::max<int64_t>(N, 1), e.stride_bias, false, &bias);
    if (rc == GEMM_F32_OK && e.residual != nullptr)
        rc = check_float("residual", e.residual, used, M, N, e.ld_residual, e.stride_residual, false, &residual);
    if (rc == GEMM_F32_OK && e.pre != nullptr)
        rc = check_float("pre", e.pre, batch, M, N, e.ld_pre, e.stride_pre, true, &pre);
    if (rc != GEMM_F32_OK) return rc;
    if (used == 0) return GEMM_F32_OK;
    const int64_t need = workspace != nullptr ? space_of(tb, batch, M, N, K) : 0;
    rc = check_workspace(workspace, workspace_bytes, need, &w);
    if (rc != GEMM_F32_OK) return rc;
    // the residual may be C itself: an element is read by the thread that writes it, before
    const bool in_place = e.residual != nullptr && e.residual == C && (M == 1 || e.ld_residual == ldc) &&
                          (batch == 1 || e.stride_residual == strideC);
    rc = check_apart({c, pre, w}, {a, b, bias, in_place ? Bytes{0, 0} : residual});
    if (rc != GEMM_F32_OK) return rc;
    const bool many = batch > 1;
    fused::Product p = plain_product(batch, M, N, K, ta, {A, lda, many ? strideA : 0}, tb, {B, ldb, many ? strideB : 0},
                                     {C, ldc, many ? strideC : 0}, need > 0 ? static_cast<float *>(workspace) : nullptr);
    p.e.activation = e.activation;
    p.e.bias = {e.bias, 0, many ? e.stride_bias : 0};
    p.e.residual = {e.residual, e.ld_residual, many ? e.stride_residual : 0};
    p.e.pre = {e.pre, e.ld_pre, many ? e.stride_pre : 0};
    return enqueue(stream, [&](hipStream_t s) { return run(p, s); });
}

int64_t gemm_f32_fused_workspace_size(int opA, int opB, int64_t batch, int64_t M, int64_t N, int64_t K) {
    if (!known_op(opA) || !known_op(opB) || !valid_sizes(batch, M, N, K)) return 0;
    return space_of(opB == GEMM_F32_OP_T, batch, M, N, K);
}

int gemm_f32_fused_grad(int opA, int opB, int64_t batch, int64_t M, int64_t N, int64_t K, const float *dC,
                        int64_t lddc, int64_t stride_dC, int activation, const float *pre, int64_t ld_pre,
                        int64_t stride_pre, const float *A, int64_t lda, int64_t strideA, const float *B,
                        int64_t ldb, int64_t strideB, float *dA, int64_t ldda, int64_t stride_dA, float *dB,
                        int64_t lddb, int64_t stride_dB, float *dbias, int64_t stride_dbias, void *workspace,
                        int64_t workspace_bytes, void *stream) {
    clear_error();
    int rc = check_op("opA", opA);
    if (rc == GEMM_F32_OK) rc = check_op("opB", opB);
    if (rc == GEMM_F32_OK) rc = check_activation(activation);
    if (rc == GEMM_F32_OK) rc = check_sizes(batch, M, N, K);
    if (rc != GEMM_F32_OK) return rc;
    const bool ta = opA == GEMM_F32_OP_T, tb = opB == GEMM_F32_OP_T, sloped = activation != GEMM_F32_ACT_NONE;
    const bool want_a = dA != nullptr, want_b = dB != nullptr, want_bias = dbias != nullptr;
    Bytes g{0, 0}, z{0, 0}, a{0, 0}, b{0, 0}, da{0, 0}, db{0, 0}, dbi{0, 0}, w{0, 0};
    rc = check_float("dC", dC, batch, M, N, lddc, stride_dC, false, &g);
    if (rc == GEMM_F32_OK && sloped) rc = check_float("pre", pre, batch, M, N, ld_pre, stride_pre, false, &z);
    if (rc == GEMM_F32_OK && want_b) rc = check_float("A", A, batch, ta ? K : M, ta ? M : K, lda, strideA, false, &a);
    if (rc == GEMM_F32_OK && want_a) rc = check_float("B", B, batch, tb ? N : K, tb ? K : N, ldb, strideB, false, &b);
    if (rc == GEMM_F32_OK && want_a)
        rc = check_float("dA", dA, batch, ta ? K : M, ta ? M : K, ldda, stride_dA, true, &da);
    if (rc == GEMM_F32_OK && want_b)
        rc = check_float("dB", dB, batch, tb ? N : K, tb ? K : N, lddb, stride_dB, true, &db);
    if (rc == GEMM_F32_OK && want_bias)
        rc = check_float("dbias", dbias, batch, 1, N, std::max<int64_t>(N, 1), stride_dbias, true, &dbi);
    if (rc != GEMM_F32_OK) return rc;
    const GradParts parts = grad_parts(ta, tb, batch, M, N, K, activation, want_a, want_b, want_bias);
    rc = check_workspace(workspace, workspace_bytes, parts.bytes(), &w);
    if (rc == GEMM_F32_OK) rc = check_apart({da, db, dbi, w}, {g, z, a, b});
    if (rc != GEMM_F32_OK) return rc;
    if (batch == 0) return GEMM_F32_OK;
    const bool many = batch > 1;
    float *at = static_cast<float *>(workspace);
    float *dz = at, *partial = at + parts.dz, *space = parts.space ? at + parts.dz + parts.partial : nullptr;
    fused::Operand grad{dC, lddc, many ? stride_dC : 0};
    fused::Slope s{};
    s.batch = batch, s.M = static_cast<int>(M), s.N = static_cast<int>(N), s.activation = activation;
    s.dc = grad, s.pre = {pre, ld_pre, many ? stride_pre : 0};
    if (parts.dz) {
        s.dz = {dz, N, M * N};
        grad = {dz, N, M * N};
    }
    if (want_bias) s.partial = partial, s.dbias = {dbias, 0, many ? stride_dbias : 0};
    s.blocks = parts.blocks, s.rows = parts.rows;
    const fused::Operand oa{A, lda, many ? strideA : 0}, ob{B, ldb, many ? strideB : 0};
    const fused::Result ra{dA, ldda, many ? stride_dA : 0}, rb{dB, lddb, many ? stride_dB : 0};
    return enqueue(stream, [&](hipStream_t q) {
        hipError_t err = hipSuccess;
        if (N > 0 && (want_bias || parts.dz > 0)) err = fused::launch_slope(s, q);
        // dA = dZ op(B)^T, or its transpose op(B) dZ^T
        const fused::Product pa = ta ? plain_product(batch, K, M, N, tb, ob, true, grad, ra, space)
                                     : plain_product(batch, M, K, N, false, grad, !tb, ob, ra, space);
        // dB = op(A)^T dZ, or its transpose dZ^T op(A)
        const fused::Product pb = tb ? plain_product(batch, N, K, M, true, grad, ta, oa, rb, space)
                                     : plain_product(batch, K, N, M, !ta, oa, false, grad, rb, space);
        if (err == hipSuccess) err = want_a && want_b ? run(pa, pb, 4 * parts.space, q) : want_a ? run(pa, q) : want_b ? run(pb, q) : err;
        return err;
    });
}

int64_t gemm_f32_fused_grad_workspace_size(int opA, int opB, int64_t batch, int64_t M, int64_t N, int64_t K,
                                           int activation, int want_dA, int want_dB, int want_dbias) {
    if (!known_op(opA) || !known_op(opB) || !known_activation(activation) || !valid_sizes(batch, M, N, K)) return 0;
    return grad_parts(opA == GEMM_F32_OP_T, opB == GEMM_F32_OP_T, batch, M, N, K, activation, want_dA, want_dB, want_dbias)
        .bytes();
}

int gemm_f32_cross_entropy(int64_t T, int64_t V, int64_t K, const float *X, int64_t ldx, const float *W, int64_t ldw,
                           const int64_t *target, int64_t ignore_index, float *loss, float *lse, void *workspace,
                           int64_t workspace_bytes, void *stream) {
    clear_error();
    Bytes x, w, t, lo, ls, ws;
    int rc = check_tokens(T, V, K, X, ldx, W, ldw, target, &x, &w, &t);
    if (rc == GEMM_F32_OK) rc = check_vector("loss", loss, T, &lo);
    if (rc == GEMM_F32_OK) rc = check_vector("lse", lse, T, &ls);
    if (rc != GEMM_F32_OK || T == 0) return rc;
    rc = check_workspace(workspace, workspace_bytes, gemm_f32_cross_entropy_workspace_size(T, V, K), &ws);
    if (rc == GEMM_F32_OK) rc = check_apart({lo, ls, ws}, {x, w, t});
    if (rc != GEMM_F32_OK) return rc;
    float *at = static_cast<float *>(workspace);
    float *space = space_of(true, 1, T, V, K, fused::kStatistics) ? at + stats_bytes(T, V) / 4 : nullptr;
    fused::Product p = plain_product(1, T, V, K, false, {X, ldx, 0}, true, {W, ldw, 0}, {}, space, fused::kStatistics);
    p.mode = fused::kStats;
    p.at_target = at, p.stats = reinterpret_cast<fused::stat2 *>(at + 2 * T), p.groups = groups_of(T, V);
    p.target = target, p.ignore = ignore_index;
    fused::Loss l{};
    l.T = p.M, l.V = p.N, l.stats = p.stats, l.groups = p.groups, l.at_target = p.at_target;
    l.target = target, l.ignore = ignore_index, l.loss = loss, l.lse = lse != nullptr ? lse : at + T;
    return enqueue(stream, [&](hipStream_t s) {
        const hipError_t err = run(p, s);
        return err == hipSuccess ? fused::launch_loss(l, s) : err;
    });
}

int64_t gemm_f32_cross_entropy_workspace_size(int64_t T, int64_t V, int64_t K) {
    return valid_sizes(1, T, V, K) ? plus(stats_bytes(T, V), space_of(true, 1, T, V, K, fused::kStatistics)) : 0;
}

int gemm_f32_cross_entropy_grad(int64_t T, int64_t V, int64_t K, const float *X, int64_t ldx, const float *W,
                                int64_t ldw, const int64_t *target, int64_t ignore_index, const float *grad_loss,
                                float *loss, float *lse, float *dX, int64_t lddx, float *dW, int64_t lddw,
                                void *workspace, int64_t workspace_bytes, void *stream) {
    clear_error();
    Bytes x, w, t, g, lo, ls, dx{0, 0}, dw{0, 0}, ws;
    int rc = check_tokens(T, V, K, X, ldx, W, ldw, target, &x, &w, &t);
    if (rc == GEMM_F32_OK) rc = check_vector("grad_loss", grad_loss, T, &g);
    if (rc == GEMM_F32_OK) rc = check_vector("loss", loss, T, &lo);
    if (rc == GEMM_F32_OK) rc = check_vector("lse", lse, T, &ls);
    if (rc == GEMM_F32_OK && dX != nullptr) rc = check_float("dX", dX, 1, T, K, lddx, 0, true, &dx);
    if (rc == GEMM_F32_OK && dW != nullptr) rc = check_float("dW", dW, 1, V, K, lddw, 0, true, &dw);
    if (rc != GEMM_F32_OK) return rc;
    // as many tokens at a time as the workspace holds
    const int64_t best = piece_rows(T, V), full = plus(piece_bytes(best, V), piece_space(best, V, K));
    int64_t rows = best, bytes = full;
    const bool sliced = workspace_bytes >= full;
    if (!sliced && T > 0) {
        const int64_t one = piece_bytes(1, V), each = piece_bytes(2, V) - one;
        rows = std::min(best, std::max<int64_t>(workspace_bytes - one, 0) / each + 1);
        if (rows > kPieceRows) rows = rows / kPieceRows * kPieceRows;
        rows = std::max(rows, piece_least(T));
        bytes = piece_bytes(rows, V);
    }
    rc = check_workspace(workspace, workspace_bytes, bytes, &ws);
    if (rc == GEMM_F32_OK) rc = check_apart({lo, ls, dx, dw, ws}, {x, w, t, g});
    if (rc != GEMM_F32_OK) return rc;
    float *at = static_cast<float *>(workspace);
    return enqueue(stream, [&](hipStream_t s) {
        hipError_t err = hipSuccess;
        if (T == 0 && dW != nullptr)  // no token: the empty sum
            return run(plain_product(1, V, K, 0, true, {}, false, {}, {dW, lddw, 0}, nullptr), s);
        for (int64_t t0 = 0; t0 < T && err == hipSuccess; t0 += rows) {
            const int64_t n = std::min(rows, T - t0);
            float *logits = at + line(2 * n + 2 * n * groups_of(n, V));
            const int64_t ldl = line(V);
            float *space = sliced && bytes > piece_bytes(best, V) ? at + piece_bytes(best, V) / 4 : nullptr;
            // (the last piece may be shorter, and ask for more)
            auto room = [&](bool tb, int64_t M, int64_t N, int64_t k, fused::Use use) {
                return space != nullptr && space_of(tb, 1, M, N, k, use) <= full - piece_bytes(best, V) ? space : nullptr;
            };
            const float *Xt = X + t0 * ldx;
            fused::Product p = plain_product(1, n, V, K, false, {Xt, ldx, 0}, true, {W, ldw, 0}, {logits, ldl, 0}, room(true, n, V, K, fused::kStatistics),
                                             fused::kStatistics);
            p.mode = fused::kStoreStats;
            p.at_target = at, p.stats = reinterpret_cast<fused::stat2 *>(at + 2 * n), p.groups = groups_of(n, V);
            p.target = target + t0, p.ignore = ignore_index;
            err = run(p, s);
            fused::Loss l{};
            l.T = p.M, l.V = p.N, l.stats = p.stats, l.groups = p.groups, l.at_target = p.at_target;
            l.target = p.target, l.ignore = ignore_index;
            l.loss = loss != nullptr ? loss + t0 : nullptr, l.lse = lse != nullptr ? lse + t0 : at + n;
            l.grad_loss = grad_loss != nullptr ? grad_loss + t0 : nullptr, l.logits = logits, l.ld = ldl;
            if (dX == nullptr && dW == nullptr) {
                if (err == hipSuccess) err = fused::launch_loss(l, s);
                continue;
            }
            fused::Product px = plain_product(1, n, K, V, false, {logits, ldl, 0}, false, {W, ldw, 0},
                                              {dX != nullptr ? dX + t0 * lddx : nullptr, lddx, 0}, room(false, n, K, V, fused::kProbabilities),
                                              fused::kProbabilities);
            px.mode = fused::kStoreSome, px.target = target + t0, px.ignore = ignore_index;
            fused::Product pw = plain_product(1, V, K, n, true, {logits, ldl, 0}, false, {Xt, ldx, 0}, {dW, lddw, 0},
                                              room(false, V, K, n, fused::kProbabilities), fused::kProbabilities);
            pw.target_k = target + t0, pw.ignore = ignore_index;
            if (t0 > 0) pw.e.residual = {dW, lddw, 0};  // the pieces before
            if (n * V <= 1 << 18) {
                if (err == hipSuccess) err = fused::launch_loss_and_probabilities(l, s);
            } else {
                if (err == hipSuccess) err = fused::launch_loss(l, s);
                if (err == hipSuccess) err = fused::launch_probabilities(l, s);
            }
            if (err == hipSuccess)
                err = dX != nullptr && dW != nullptr ? run(px, pw, px.space != nullptr ? full - piece_bytes(best, V) : 0, s) : dX != nullptr ? run(px, s) : run(pw, s);
        }
        return err;
    });
}

int64_t gemm_f32_cross_entropy_grad_workspace_size(int64_t T, int64_t V, int64_t K) {
    if (!valid_sizes(1, T, V, K)) return 0;
    const int64_t rows = piece_rows(T, V);
    return plus(piece_bytes(rows, V), piece_space(rows, V, K));
}

int64_t gemm_f32_cross_entropy_grad_workspace_least(int64_t T, int64_t V, int64_t K) {
    return valid_sizes(1, T, V, K) ? piece_bytes(piece_least(T), V) : 0;
}

int gemm_f32_fused_abi_version(void) { return 1; }

}  // extern "C"
