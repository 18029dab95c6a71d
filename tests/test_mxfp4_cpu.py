"""The MXFP4 entry points without a GPU: declarations, refusals (all of them
before anything reaches the device) and the plain implementation that the
GPU tests compare with."""

import ctypes
import os
import re
import shutil
import subprocess
import sys

import numpy as np
import pytest

from dense_fp32_gemm_row_amd import binding as b
from tests import mxfp4_oracle as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_mxfp4.h")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(b.LIBRARY):
        import __graft_entry__

        __graft_entry__.build()
    return b.load()


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(gemm_mxfp4\w*)\s*\(", text)))


def test_every_declared_symbol_is_exported(lib):
    names = declared()
    assert {"gemm_mxfp4", "gemm_mxfp4_weight", "gemm_mxfp4_quantize",
            "gemm_mxfp4_dequantize"} <= set(names)
    raw = ctypes.CDLL(b.LIBRARY)
    for name in names:
        assert hasattr(raw, name), name
    assert b.gemm_mxfp4_abi_version() == 1


def test_header_serves_a_c_caller(lib, tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    fns = "\n".join(f"        (void (*)(void))&{n}," for n in declared())
    src = tmp_path / "caller.c"
    src.write_text(f"""
#include <stdio.h>
#include "gemm_mxfp4.h"
int main(void) {{
    void (*fns[])(void) = {{
{fns}
    }};
    gemm_mxfp4_matrix m = {{0, 16, 0, 0, 4, 0}};
    if (gemm_mxfp4(1, -1, 1, 1, &m, &m, NULL, 1, 0, NULL, 0, NULL) != GEMM_F32_EINVAL) return 1;
    if (gemm_f32_last_error()[0] == 0) return 2;
    if (gemm_mxfp4(1, 0, 1, 1, &m, &m, NULL, 1, 0, NULL, 0, NULL) != GEMM_F32_OK) return 3;
    printf("%d %d\\n", gemm_mxfp4_abi_version(), (int)(sizeof fns / sizeof fns[0]));
    return 0;
}}
""")
    exe = tmp_path / "caller"
    libdir = os.path.dirname(b.LIBRARY)
    res = subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                          os.path.join(ROOT, "include"), str(src), "-L", libdir, "-lgemm_f32",
                          f"-Wl,-rpath,{libdir}", "-o", str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout.split() == ["1", str(len(declared()))]


# ---- refusals: fake addresses, never dereferenced -----------------------------

def matrix(codes=0x100000, ldq=64, sq=0, scales=0x200000, lds=4, ss=0):
    return b.Mxfp4Matrix(codes, ldq, sq, scales, lds, ss)


# changes to one operand of a 4 x 100 matrix (64 bytes of codes, 4 of scales a row)
BAD_MATRIX = [
    ("codes NULL", dict(codes=0), "NULL"),
    ("scales NULL", dict(scales=0), "NULL"),
    ("codes misaligned", dict(codes=0x100008), "multiples of 16"),
    ("ld_codes not whole blocks", dict(ldq=72), "multiples of 16"),
    ("ld_codes too small", dict(ldq=48), "ld_codes"),
    ("stride_codes not whole blocks", dict(sq=1000), "multiples of 16"),
    ("scales misaligned", dict(scales=0x200002), "multiples of 4"),
    ("ld_scales not whole words", dict(lds=6), "multiples of 4"),
    ("ld_scales too small", dict(lds=0), "ld_scales"),
    ("negative batch stride", dict(sq=-16), "negative batch stride"),
    ("negative scale stride", dict(ss=-4), "negative batch stride"),
    ("span", dict(ldq=1 << 59), "2^60"),
]


@pytest.mark.parametrize("change,detail", [(c, d) for _, c, d in BAD_MATRIX],
                         ids=[n for n, _, _ in BAD_MATRIX])
def test_refused_matrices(lib, change, detail):
    good, bad = matrix(codes=0x300000, scales=0x400000), matrix(**change)
    C, X, none = 0x500000, 0x600000, None
    calls = [
        lambda: b.gemm_mxfp4_product(1, 4, 4, 100, bad, good, C, 4, 0),
        lambda: b.gemm_mxfp4_product(1, 4, 4, 100, good, bad, C, 4, 0),
        lambda: b.gemm_mxfp4_weight_product(b.OP_T, 1, 4, 4, 100, X, 100, 0, bad, C, 4, 0),
        lambda: b.gemm_mxfp4_weight_product(b.OP_N, 1, 4, 100, 4, X, 4, 0, bad, C, 100, 0),
        lambda: b.gemm_mxfp4_quantize(1, 4, 100, X, 100, 0, bad, none),
        lambda: b.gemm_mxfp4_quantize(1, 100, 4, X, 4, 0, none, bad),
        lambda: b.gemm_mxfp4_dequantize(1, 4, 100, bad, X, 100, 0),
    ]
    for call in calls:
        assert call() == b.GEMM_F32_EINVAL
        assert detail in b.gemm_f32_last_error(), b.gemm_f32_last_error()


def test_refused_sizes_and_pointers(lib):
    A, B = matrix(), matrix(codes=0x300000, scales=0x400000)
    C = 0x500000

    def bad(rc, detail):
        assert rc == b.GEMM_F32_EINVAL
        assert detail in b.gemm_f32_last_error(), b.gemm_f32_last_error()

    p = b.gemm_mxfp4_product
    bad(p(1, -1, 4, 100, A, B, C, 4, 0), "negative M")
    bad(p(-1, 4, 4, 100, A, B, C, 4, 0), "negative batch")
    bad(p(1, 4, 1 << 31, 100, A, B, C, 1 << 31, 0), "N=2147483648 above")
    bad(p(1, 4, 4, 1 << 31, A, B, C, 4, 0), "K=2147483648 above")
    bad(p(1, 4, 4, 100, A, B, C, 3, 0), "leading dimension 3 of C")
    bad(p(1, 4, 4, 100, A, B, 0, 4, 0), "C is NULL")
    bad(p(1, 4, 4, 100, A, B, C + 2, 4, 0), "4-byte aligned")
    bad(p(1, 4, 4, 100, None, B, C, 4, 0), "A is NULL")
    bad(p(2, 4, 4, 100, A, B, C, 4, 15), "overlap")
    bad(p(1, 4, 4, 100, A, B, 0x100000 + 4 * 64 - 4, 4, 0), "overlaps an input")
    bad(p(1, 4, 4, 100, A, B, 0x400000 - 60, 4, 0), "overlaps an input")
    bad(p(1, 4, 4, 100, A, B, C, 1 << 59, 0), "too large")
    bad(p(2, 1 << 31 - 1, 4, 0, A, B, C, 1 << 56, 1 << 56), "2^60")
    w = b.gemm_mxfp4_weight_product
    bad(w(2, 1, 4, 4, 100, C, 100, 0, B, C, 4, 0), "opW")
    bad(w(b.OP_T, 1, 4, 4, 100, 0x600000, 99, 0, B, C, 4, 0), "leading dimension 99 of A")
    bad(w(b.OP_T, 1, 4, 4, 100, 0, 100, 0, B, C, 4, 0), "A is NULL")
    bad(w(b.OP_T, 1, 4, 4, 100, C - 4, 100, 0, B, C, 4, 0), "overlaps an input")
    bad(w(b.OP_N, 1, 4, 4, 100, 0x600000, 100, -1, B, C, 4, 0), "negative batch stride of A")
    q = b.gemm_mxfp4_quantize
    bad(q(1, 4, 100, 0x600000, 100, 0, None, None), "both NULL")
    bad(q(1, 4, 100, 0x600000, 99, 0, A, None), "leading dimension 99 of X")
    bad(q(1, 4, 100, 0x600001, 100, 0, A, None), "4-byte aligned")
    bad(q(1, 4, 100, 0x100000, 100, 0, A, None), "overlaps an input")
    bad(q(1, 4, 100, 0x600000, 100, 0, A, matrix(ldq=16)), "two outputs overlap")
    bad(q(1, 4, 100, 0x600000, 100, 0, matrix(scales=0x100010), None), "two outputs overlap")
    bad(q(2, 4, 100, 0x600000, 100, 400, matrix(sq=128, ss=16), None), "overlap")
    bad(q(2, 4, 100, 0x600000, 100, 400, matrix(sq=256, ss=12), None), "overlap")
    d = b.gemm_mxfp4_dequantize
    bad(d(1, 4, 100, A, 0, 100, 0), "Y is NULL")
    bad(d(2, 4, 100, A, 0x600000, 100, 399), "overlap")
    bad(d(1, 4, 100, None, 0x600000, 100, 0), "Q is NULL")


def test_empty_calls_enqueue_nothing(lib):
    m = matrix()
    for M, N, batch in ((0, 4, 1), (4, 0, 1), (4, 4, 0)):
        assert b.gemm_mxfp4_product(batch, M, N, 100, None, None, 0, max(N, 1), 0) == 0
        for op in (b.OP_N, b.OP_T):
            assert b.gemm_mxfp4_weight_product(op, batch, M, N, 100, 0, 100, 0, None, 0, max(N, 1), 0) == 0
        assert b.gemm_mxfp4_quantize(batch, M, N, 0, max(N, 1), 0, m, m) == 0
        assert b.gemm_mxfp4_dequantize(batch, M, N, m, 0, max(N, 1), 0) == 0
    assert b.gemm_f32_last_error() == ""


def test_workspace_sizes(lib):
    f, w = b.gemm_mxfp4_workspace_size, b.gemm_mxfp4_weight_workspace_size
    for args in ((0, 4, 4, 4), (1, -1, 4, 4), (1, 4, 4, 0), (1, 4, 4, 1 << 31)):
        assert f(*args) == 0 and w(b.OP_T, *args) == 0 and w(b.OP_N, *args) == 0
    assert w(2, 1, 64, 64, 65536) == 0
    for args in ((1, 8192, 8192, 8192), (64, 1024, 1024, 1024), (1, 64, 64, 64)):
        assert f(*args) == 0, "many tiles or a short K: no slices"
    for M, N, K in ((1024, 1024, 65536), (64, 64, 65536), (1, 32, 1 << 30)):
        for n in (f(1, M, N, K), w(b.OP_T, 1, M, N, K), w(b.OP_N, 1, M, N, K)):
            assert n >= 0 and n % (4 * M * N) == 0


def test_tensor_calls_refuse_cpu_tensors(lib):
    torch = pytest.importorskip("torch")
    with pytest.raises(TypeError):
        b.mxfp4_quantize(torch.zeros(3, 4))
    with pytest.raises(TypeError):
        b.Mxfp4(torch.zeros(3, 16, dtype=torch.uint8), torch.zeros(3, 4, dtype=torch.uint8), 32)


# ---- the plain implementation ---------------------------------------------------

def test_plain_quantize_hand_worked():
    x = np.zeros((1, 64), np.float32)
    x[0, :8] = [6.0, 0.25, 0.75, 2.5, 5.0, 3.5, -0.25, 7.9]
    x[0, 32:36] = [1e-3, 0.0, -0.0, np.inf]
    codes, scales = ref.quantize(x)
    # amax 7.9: floor(log2) = 2, scale 2^0
    assert scales.tolist() == [[127, 255, 0, 0]]
    v = ref.values(codes, scales, 64)[0]
    # ties to the even code: .25 -> 0, .75 -> 1, 2.5 -> 2, 5 -> 4, 3.5 -> 4; 7.9 -> 6
    assert v[:8].tolist() == [6.0, 0.0, 1.0, 2.0, 4.0, 4.0, 0.0, 6.0]
    assert np.signbit(v[6]) and np.isnan(v[32:]).all()
    assert codes[0, 0] == 0x07 and codes[0, 16:].max() == 0  # low half first


def test_plain_quantize_error_is_half_a_step():
    """Below saturation the error is at most half the spacing of elements."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((50, 96)).astype(np.float32)
    c, s = ref.quantize(x)
    v = ref.values(c, s, 96)
    step = np.repeat(2.0 ** (s[:, :3].astype(int) - 127), 32, axis=1)
    m = np.abs(x) / step
    gap = np.where(m < 2, 0.5, np.where(m < 4, 1.0, 2.0))
    ok = np.abs(v - x) / step <= gap / 2
    assert (ok | (m > 6)).all() and (m < 8).all()


def test_plain_requantizes_to_itself():
    """Values of the format whose block reaches the top binade come back."""
    rng = np.random.default_rng(4)
    c, s = ref.random_matrix(rng, (20,), 64)
    c[:, ::16] = 0x77  # an element of 6 in every block
    v = ref.values(c, s, 64)
    c2, s2 = ref.quantize(v.astype(np.float32))
    assert np.array_equal(ref.values(c2, s2, 64), v) and np.array_equal(s2[:, :2], s[:, :2])


def test_sizes_just_above_the_limit(lib):
    """Sizes whose last tile would end past what 32 bits count."""
    n, one = (1 << 31) - 1023, matrix(ldq=1 << 31, lds=1 << 31)
    calls = [
        lambda: b.gemm_mxfp4_product(1, 1, 1, n, one, one, 0x500000, 1, 0),
        lambda: b.gemm_mxfp4_product(1, 1, n, 32, one, one, 0x500000, n, 0),
        lambda: b.gemm_mxfp4_product(1, n, 1, 32, one, one, 0x500000, 1, 0),
        lambda: b.gemm_mxfp4_product(n, 1, 1, 32, one, one, 0x500000, 1, 1),
        lambda: b.gemm_mxfp4_weight_product(b.OP_T, 1, 1, 1, n, 0x600000, n, 0, one, 0x500000, 1, 0),
        lambda: b.gemm_mxfp4_weight_product(b.OP_N, 1, 1, n, 1, 0x600000, 1, 0, one, 0x500000, n, 0),
        lambda: b.gemm_mxfp4_quantize(1, 1, n, 0x600000, n, 0, one, None),
        lambda: b.gemm_mxfp4_quantize(1, n, 1, 0x600000, 1, 0, None, one),
        lambda: b.gemm_mxfp4_dequantize(1, 1, n, one, 0x600000, n, 0),
    ]
    for call in calls:
        assert call() == b.GEMM_F32_EINVAL
        assert "above 2^31-1024" in b.gemm_f32_last_error(), b.gemm_f32_last_error()
    for sizes in ((1, 1, 1, n), (1, n, 1, 1), (n, 1, 1, 1)):
        assert b.gemm_mxfp4_workspace_size(*sizes) == 0
        assert b.gemm_mxfp4_weight_workspace_size(b.OP_T, *sizes) == 0


@pytest.mark.parametrize("shape", [(64,), (2, 3, 4, 64), (), (4, -1), (-4, 64), (-2, 4, 64)])
def test_empty_refuses_shapes_that_no_call_takes(lib, shape):
    with pytest.raises(ValueError):
        b.mxfp4_empty(shape, "cuda:0")


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_empty_refuses_other_devices(lib, device):
    with pytest.raises(TypeError, match="GPU"):
        b.mxfp4_empty((4, 64), device)


def test_package_exports_what_its_calls_take(lib):
    """`op` of gemm_mxfp4_weight and the `out` of a quantisation, without the binding's own name."""
    import dense_fp32_gemm_row_amd as pkg

    assert (pkg.OP_N, pkg.OP_T) == (b.OP_N, b.OP_T) and pkg.mxfp4_empty is b.mxfp4_empty
    for name in set(pkg.__all__) - {"workloads"}:
        assert getattr(pkg, name) is getattr(b, name)
    with pytest.raises(AttributeError):
        pkg.no_such_name


def test_package_gives_its_workloads():
    """In a fresh interpreter: an attribute access must import the module, not ask itself for it."""
    code = "import dense_fp32_gemm_row_amd as p; assert p.workloads.__name__ == 'dense_fp32_gemm_row_amd.workloads'"
    run = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stderr[-300:]
