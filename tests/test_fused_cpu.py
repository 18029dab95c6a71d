"""The fused operators without a GPU: exports, refusals and workspace sizes
(no call here reaches HIP)."""

import ctypes
import os
import re

import pytest
import torch

from dense_fp32_gemm_row_amd import binding as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_f32_fused.h")
A, B, C, D, R, Z, WS = (0x100000 * i for i in range(1, 8))  # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(b.LIBRARY):
        import __graft_entry__

        __graft_entry__.build()
    return b.load()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(gemm_f32\w*)\s*\(", text)))
    assert len(names) == 10, names
    raw = ctypes.CDLL(b.LIBRARY)
    for name in names:
        assert hasattr(raw, name), name
    assert b.gemm_f32_fused_abi_version() == 1


def test_activations_are_the_headers():
    text = open(HEADER).read()
    got = {n.lower(): int(v) for n, v in re.findall(r"#define GEMM_F32_ACT_(\w+) (\d)", text)}
    assert got == b.ACTIVATIONS


def epilogue(**kw):
    e = b.Epilogue(kw.pop("activation", 0))
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def fused(**kw):
    d = dict(opA=0, opB=0, batch=1, M=4, N=6, K=5, A=A, lda=5, sA=0, B=B, ldb=6, sB=0, epilogue=None, C=C, ldc=6,
             sC=0, workspace=None, workspace_bytes=0)
    assert set(kw) <= set(d)
    return b.gemm_f32_fused(*{**d, **kw}.values(), None)


FUSED_BAD = [
    (dict(opA=2), "opA"), (dict(opB=-1), "opB"), (dict(M=-1), "negative M"), (dict(K=1 << 31), "2^31"),
    (dict(batch=-1), "negative batch"), (dict(lda=4), "of A"), (dict(ldb=5), "of B"), (dict(ldc=5), "of C"),
    (dict(opA=1, lda=3), "of A"), (dict(opB=1, ldb=4), "of B"), (dict(A=None), "A is NULL"), (dict(C=None), "C is NULL"),
    (dict(A=A + 2), "aligned"), (dict(C=A + 8), "overlaps an input"), (dict(C=B), "overlaps an input"),
    (dict(batch=2, sA=20, sB=30, sC=23), "overlap"), (dict(sA=-1), "negative batch stride"),
    (dict(epilogue=epilogue(activation=5)), "activation 5"), (dict(epilogue=epilogue(activation=-1)), "activation -1"),
    (dict(epilogue=epilogue(bias=C, stride_bias=0)), "overlaps an input"),
    (dict(epilogue=epilogue(bias=D + 1)), "bias not 4-byte"),
    (dict(epilogue=epilogue(residual=R, ld_residual=5)), "of residual"),
    (dict(epilogue=epilogue(residual=C + 4, ld_residual=6)), "overlaps an input"),
    (dict(epilogue=epilogue(residual=C, ld_residual=7)), "overlaps an input"),
    (dict(batch=2, sA=20, sB=30, sC=24, epilogue=epilogue(residual=C, ld_residual=6)), "overlaps an input"),
    (dict(epilogue=epilogue(pre=Z, ld_pre=5)), "of pre"), (dict(epilogue=epilogue(pre=C, ld_pre=6)), "outputs overlap"),
    (dict(epilogue=epilogue(pre=A, ld_pre=6)), "overlaps an input"),
    (dict(epilogue=epilogue(pre=R, ld_pre=6, residual=R, ld_residual=6)), "overlaps an input"),
]


@pytest.mark.parametrize("kw,detail", FUSED_BAD, ids=[str(i) for i in range(len(FUSED_BAD))])
def test_fused_refuses(kw, detail):
    assert fused(**kw) == b.GEMM_F32_EINVAL
    assert detail in b.gemm_f32_last_error()


def test_empty_products_enqueue_nothing():
    assert fused(M=0, A=None, C=None) == b.GEMM_F32_OK
    assert fused(N=0, B=None, C=None) == b.GEMM_F32_OK
    assert fused(batch=0, A=None, B=None, C=None) == b.GEMM_F32_OK
    assert fused(M=0, lda=4, K=5) == b.GEMM_F32_EINVAL  # a wrong argument is wrong all the same


def grad(**kw):
    d = dict(opA=0, opB=0, batch=1, M=4, N=6, K=5, dC=C, lddc=6, sdC=0, activation=0, pre=None, ld_pre=6, s_pre=0, A=A,
             lda=5, sA=0, B=B, ldb=6, sB=0, dA=D, ldda=5, sdA=0, dB=R, lddb=6, sdB=0, dbias=None, sdbias=0,
             workspace=WS, workspace_bytes=1 << 20)
    assert set(kw) <= set(d)
    return b.gemm_f32_fused_grad(*{**d, **kw}.values(), None)


GRAD_BAD = [
    (dict(opA=7), "opA"), (dict(activation=9), "activation 9"), (dict(N=-1), "negative N"), (dict(lddc=5), "of dC"),
    (dict(activation=1), "pre is NULL"), (dict(activation=1, pre=Z, ld_pre=5), "of pre"), (dict(A=None), "A is NULL"),
    (dict(B=None), "B is NULL"), (dict(ldda=4), "of dA"), (dict(lddb=5), "of dB"), (dict(opB=1, ldb=6, lddb=4), "of dB"),
    (dict(opA=1, ldda=3), "of dA"), (dict(dA=A), "overlaps an input"), (dict(dB=C), "overlaps an input"),
    (dict(dB=D), "outputs overlap"), (dict(dbias=D + 4), "outputs overlap"), (dict(dbias=Z + 2), "dbias not 4-byte"),
    (dict(activation=1, pre=Z, workspace=None), "workspace of"),
    (dict(activation=1, pre=Z, workspace_bytes=95), "workspace of 96 bytes needed, 95"),
    (dict(activation=1, pre=Z, workspace=WS + 2), "workspace not 4-byte"),
    (dict(activation=1, pre=Z, workspace=A), "overlaps an input"),
    (dict(batch=2, sdC=24, sA=20, sB=30, sdA=0, sdB=30), "dA: its matrices overlap"),
    (dict(batch=2, sdC=24, sA=20, sB=30, sdA=20, sdB=30, dbias=Z, sdbias=0), "dbias: its matrices overlap"),
]


@pytest.mark.parametrize("kw,detail", GRAD_BAD, ids=[str(i) for i in range(len(GRAD_BAD))])
def test_fused_grad_refuses(kw, detail):
    assert grad(**kw) == b.GEMM_F32_EINVAL
    assert detail in b.gemm_f32_last_error()


def loss(**kw):
    d = dict(T=4, V=6, K=5, X=A, ldx=5, W=B, ldw=5, target=C, ignore=-100, loss=D, lse=R, workspace=WS,
             workspace_bytes=1 << 20)
    assert set(kw) <= set(d)
    return b.gemm_f32_cross_entropy(*{**d, **kw}.values(), None)


def loss_grad(**kw):
    d = dict(T=4, V=6, K=5, X=A, ldx=5, W=B, ldw=5, target=C, ignore=-100, grad_loss=None, loss=None, lse=None, dX=D,
             lddx=5, dW=R, lddw=5, workspace=WS, workspace_bytes=1 << 20)
    assert set(kw) <= set(d)
    return b.gemm_f32_cross_entropy_grad(*{**d, **kw}.values(), None)


LOSS_BAD = [
    (dict(T=-1), "negative T"), (dict(V=0), "empty vocabulary"), (dict(K=1 << 31), "2^31"), (dict(ldx=4), "of X"),
    (dict(ldw=4), "of W"), (dict(X=None), "X is NULL"), (dict(W=None), "W is NULL"), (dict(target=None), "target is NULL"),
    (dict(target=C + 4), "target not 8-byte"), (dict(loss=D + 1), "loss not 4-byte"), (dict(loss=C), "overlaps an input"),
    (dict(loss=Z, lse=Z), "outputs overlap"), (dict(workspace=None), "workspace of"),
    (dict(workspace_bytes=8), "8 given"), (dict(workspace=WS + 1), "workspace not 4-byte"), (dict(workspace=A), "overlaps an input"),
]


@pytest.mark.parametrize("kw,detail", LOSS_BAD, ids=[str(i) for i in range(len(LOSS_BAD))])
def test_cross_entropy_refuses(kw, detail):
    for call in (loss, loss_grad):
        assert call(**kw) == b.GEMM_F32_EINVAL
        assert detail in b.gemm_f32_last_error()


@pytest.mark.parametrize("kw,detail", [(dict(lddx=4), "of dX"), (dict(lddw=4), "of dW"), (dict(dX=A), "overlaps an input"),
                                       (dict(dW=D), "outputs overlap"), (dict(grad_loss=Z + 2), "grad_loss not 4-byte"),
                                       (dict(grad_loss=D), "overlaps an input")])
def test_cross_entropy_grad_refuses(kw, detail):
    assert loss_grad(**kw) == b.GEMM_F32_EINVAL
    assert detail in b.gemm_f32_last_error()


def test_no_tokens():
    assert loss(T=0, X=None, target=None, workspace=None) == b.GEMM_F32_OK
    assert loss(T=0, V=0, X=None, W=None, target=None, workspace=None) == b.GEMM_F32_OK
    assert loss_grad(T=0, X=None, W=None, target=None, dW=None, workspace=None) == b.GEMM_F32_OK


@pytest.mark.parametrize("T,V,K", [(1, 1, 1), (64, 1000, 256), (517, 32003, 1001), (4096, 131072, 2048),
                                   (100000, 200000, 64), (300, 1 << 30, 8)])
def test_workspace_sizes(T, V, K):
    size, least = (f(T, V, K) for f in (b.gemm_f32_cross_entropy_grad_workspace_size,
                                        b.gemm_f32_cross_entropy_grad_workspace_least))
    assert 0 < least <= size
    # the least holds some rows' logits; the size no more than 4 GiB of them, unless 256 rows need it
    assert least >= 4 * min(T, 64) * V
    assert size <= max(4 << 30, 4 * 256 * V) * 1.25 + 64 * 4 * (T + V) * K
    assert b.gemm_f32_cross_entropy_workspace_size(T, V, K) < 4 * T * V + 64 * T  # not the logits
    assert loss_grad(T=T, V=V, K=K, ldx=K, ldw=K, X=1 << 40, W=1 << 44, target=1 << 48, dX=1 << 49, lddx=K, dW=1 << 50,
                     lddw=K, workspace_bytes=least - 1, workspace=1 << 52) == b.GEMM_F32_EINVAL


def test_sizes_that_overflow_are_refused():
    big = (1 << 31) - 1024
    assert b.gemm_f32_fused_grad_workspace_size(0, 0, big, big, big, 1, 1, 1, 1, 0) > 1 << 60
    assert grad(batch=big, M=big, N=big, K=1, lddc=big, activation=1, pre=Z, ld_pre=big, lda=1, ldb=big, ldda=1,
                sdA=big, lddb=big, sdB=big) == b.GEMM_F32_EINVAL
    assert b.gemm_f32_cross_entropy_grad_workspace_size(big, big, 1) > 0
    assert b.gemm_f32_cross_entropy_workspace_size(-1, 4, 4) == 0
    assert b.gemm_f32_fused_workspace_size(0, 3, 1, 4, 4, 4) == 0


def test_tensor_calls_refuse():
    x, w = torch.zeros(3, 4), torch.zeros(4, 5)
    for call in (lambda: b.gemm_fused(x, w), lambda: b.gemm_fused_grad(torch.zeros(3, 5), x, w),
                 lambda: b.cross_entropy(x, x, torch.zeros(3, dtype=torch.int64)),
                 lambda: b.cross_entropy_grad(x, x, torch.zeros(3, dtype=torch.int64))):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="none, relu"):
        b._activation("swish")
    with pytest.raises(ValueError):
        b._activation([])
