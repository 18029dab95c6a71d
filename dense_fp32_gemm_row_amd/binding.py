"""ctypes binding of libgemm_f32.so (declared in include/gemm_f32.h and
include/gemm_mxfp4.h).

Argument marshalling only: every step of the product runs in the HIP
kernels behind the C ABI.  PyTorch provides device memory and streams; it
computes nothing here.  There is no fallback: if the library is missing the
calls raise.

Functions with the C names take raw integers (sizes, device addresses,
leading dimensions, a hipStream_t address) and return the C status code.
``gemm`` is the tensor-level convenience used by tests and the benchmark;
``Mxfp4`` and the functions below it are the same for matrices held in
microscaled 4-bit floating point.
"""

from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(HERE, "libgemm_f32.so")

GEMM_F32_OK = 0
GEMM_F32_EINVAL = -1
GEMM_F32_EHIP = -2
GEMM_F32_ENOKERNEL = -3

OP_N = 0  # operand as stored
OP_T = 1  # operand transposed

VARIANT_NAIVE = 0
VARIANT_LDS = 1
VARIANT_REGBLOCK = 2
VARIANT_MFMA = 3
VARIANTS = {"naive": VARIANT_NAIVE, "lds": VARIANT_LDS, "regblock": VARIANT_REGBLOCK,
            "mfma": VARIANT_MFMA}

_i64 = ctypes.c_int64
_vp = ctypes.c_void_p
_int = ctypes.c_int

_LIB: ctypes.CDLL | None = None
_torch = None  # the module, once load() has run


class GemmError(RuntimeError):
    def __init__(self, code: int, detail: str):
        self.code = code
        super().__init__(f"{gemm_f32_strerror(code)} ({code}): {detail}")


def load(path: str = LIBRARY) -> ctypes.CDLL:
    """Loads the library (once).  Raises if it has not been built."""
    global _LIB, _torch
    if _LIB is not None:
        return _LIB
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
    # torch ships its own HIP runtime.  Loading torch first makes the
    # library's libamdhip64.so.7 dependency resolve (by soname) to that copy,
    # so the library launches into the same runtime that owns torch's memory
    # and streams.  Loaded the other way round, the process would hold two
    # HIP runtimes and torch's stream handles would be foreign to ours.
    import torch

    _torch = torch
    lib = ctypes.CDLL(path)
    lib.gemm_f32.restype = _int
    lib.gemm_f32.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp]
    lib.gemm_f32_variant.restype = _int
    lib.gemm_f32_variant.argtypes = [_int, _int, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp,
                                     _i64, _vp]
    lib.gemm_f32_strided_batched.restype = _int
    lib.gemm_f32_strided_batched.argtypes = [_i64, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64,
                                             _i64, _vp, _i64, _i64, _vp]
    lib.gemm_f32_strided_batched_variant.restype = _int
    lib.gemm_f32_strided_batched_variant.argtypes = [_int, _int, _i64, _i64, _i64, _i64, _vp, _i64,
                                                     _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp]
    lib.gemm_f32_ex.restype = _int
    lib.gemm_f32_ex.argtypes = [_int, _int, _int, _int, _i64, _i64, _i64, _i64, _vp, _i64, _i64,
                                _vp, _i64, _i64, _vp, _i64, _i64, _vp]
    lib.gemm_f32_splitk.restype = _int
    lib.gemm_f32_splitk.argtypes = [_int, _int, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp,
                                    _i64, _vp, _i64, _vp]
    lib.gemm_f32_splitk_noalloc.restype = _int
    lib.gemm_f32_splitk_noalloc.argtypes = [_int, _int, _i64, _i64, _i64, _i64, _vp, _i64, _vp,
                                            _i64, _vp, _i64, _vp]
    lib.gemm_f32_splitk_workspace_size.restype = _i64
    lib.gemm_f32_splitk_workspace_size.argtypes = [_i64, _i64, _i64, _i64]
    lib.gemm_f32_strerror.restype = ctypes.c_char_p
    lib.gemm_f32_strerror.argtypes = [_int]
    lib.gemm_f32_last_error.restype = ctypes.c_char_p
    lib.gemm_f32_last_error.argtypes = []
    lib.gemm_f32_config_count.restype = _int
    lib.gemm_f32_config_count.argtypes = [_int]
    lib.gemm_f32_config_name.restype = ctypes.c_char_p
    lib.gemm_f32_config_name.argtypes = [_int, _int]
    lib.gemm_f32_select.restype = _int
    lib.gemm_f32_select.argtypes = [_i64, _i64, _i64, _i64, _i64, _i64,
                                    ctypes.POINTER(_int), ctypes.POINTER(_int)]
    lib.gemm_f32_plan.restype = _int
    lib.gemm_f32_plan.argtypes = [_i64, _i64, _i64, _i64, _i64, _i64, ctypes.POINTER(_int),
                                  ctypes.POINTER(_int), ctypes.POINTER(_i64),
                                  ctypes.POINTER(_int), ctypes.POINTER(_int)]
    lib.gemm_f32_abi_version.restype = _int
    lib.gemm_f32_abi_version.argtypes = []
    lib.gemm_mxfp4_quantize.restype = _int
    lib.gemm_mxfp4_quantize.argtypes = [_i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _vp]
    lib.gemm_mxfp4_dequantize.restype = _int
    lib.gemm_mxfp4_dequantize.argtypes = [_i64, _i64, _i64, _vp, _vp, _i64, _i64, _vp]
    lib.gemm_mxfp4.restype = _int
    lib.gemm_mxfp4.argtypes = [_i64, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _i64, _vp, _i64, _vp]
    lib.gemm_mxfp4_workspace_size.restype = _i64
    lib.gemm_mxfp4_workspace_size.argtypes = [_i64, _i64, _i64, _i64]
    lib.gemm_mxfp4_weight.restype = _int
    lib.gemm_mxfp4_weight.argtypes = [_int, _i64, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp,
                                      _i64, _i64, _vp, _i64, _vp]
    lib.gemm_mxfp4_weight_workspace_size.restype = _i64
    lib.gemm_mxfp4_weight_workspace_size.argtypes = [_int, _i64, _i64, _i64, _i64]
    lib.gemm_mxfp4_abi_version.restype = _int
    lib.gemm_mxfp4_abi_version.argtypes = []
    _LIB = lib
    return lib


# ---- the C entry points, same names, raw arguments -------------------------

def gemm_f32(M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> int:
    return load().gemm_f32(M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_f32_variant(variant, config_id, M, N, K, A, lda, B, ldb, C, ldc, stream=None) -> int:
    return load().gemm_f32_variant(variant, config_id, M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_f32_strided_batched(batch, M, N, K, A, lda, sA, B, ldb, sB, C, ldc, sC,
                             stream=None) -> int:
    return load().gemm_f32_strided_batched(batch, M, N, K, A, lda, sA, B, ldb, sB, C, ldc, sC,
                                           stream)


def gemm_f32_strided_batched_variant(variant, config_id, batch, M, N, K, A, lda, sA, B, ldb, sB,
                                     C, ldc, sC, stream=None) -> int:
    return load().gemm_f32_strided_batched_variant(variant, config_id, batch, M, N, K, A, lda, sA,
                                                   B, ldb, sB, C, ldc, sC, stream)


def gemm_f32_ex(variant, config_id, opA, opB, batch, M, N, K, A, lda, sA, B, ldb, sB, C, ldc,
                sC, stream=None) -> int:
    return load().gemm_f32_ex(variant, config_id, opA, opB, batch, M, N, K, A, lda, sA, B, ldb,
                              sB, C, ldc, sC, stream)


def gemm_f32_splitk(variant, config_id, splits, M, N, K, A, lda, B, ldb, C, ldc, workspace,
                    workspace_bytes, stream=None) -> int:
    return load().gemm_f32_splitk(variant, config_id, splits, M, N, K, A, lda, B, ldb, C, ldc,
                                  workspace, workspace_bytes, stream)


def gemm_f32_splitk_noalloc(variant, config_id, splits, M, N, K, A, lda, B, ldb, C, ldc,
                            stream=None) -> int:
    return load().gemm_f32_splitk_noalloc(variant, config_id, splits, M, N, K, A, lda, B, ldb, C,
                                          ldc, stream)


SPLITK_SCRATCH_BYTES = 33554432  # GEMM_F32_SPLITK_SCRATCH_BYTES


def gemm_f32_splitk_workspace_size(M, N, K, splits) -> int:
    return load().gemm_f32_splitk_workspace_size(M, N, K, splits)


def gemm_f32_strerror(code: int) -> str:
    return load().gemm_f32_strerror(code).decode()


def gemm_f32_last_error() -> str:
    return load().gemm_f32_last_error().decode()


def gemm_f32_config_count(variant: int) -> int:
    return load().gemm_f32_config_count(variant)


def gemm_f32_config_name(variant: int, config_id: int) -> str | None:
    name = load().gemm_f32_config_name(variant, config_id)
    return None if name is None else name.decode()


def gemm_f32_select(M, N, K, lda, ldb, ldc) -> tuple[int, int]:
    v, c = _int(), _int()
    rc = load().gemm_f32_select(M, N, K, lda, ldb, ldc, ctypes.byref(v), ctypes.byref(c))
    if rc != GEMM_F32_OK:
        raise GemmError(rc, gemm_f32_last_error())
    return v.value, c.value


def gemm_f32_plan(M, N, K, lda, ldb, ldc) -> dict:
    """How gemm_f32 runs one product: {"parts", "axis", "split", "configs": [(variant,
    config_id), ...]} with one entry per launch."""
    parts, axis, split = _int(), _int(), _i64()
    v, c = (_int * 2)(), (_int * 2)()
    rc = load().gemm_f32_plan(M, N, K, lda, ldb, ldc, ctypes.byref(parts), ctypes.byref(axis),
                              ctypes.byref(split), v, c)
    if rc != GEMM_F32_OK:
        raise GemmError(rc, gemm_f32_last_error())
    return {"parts": parts.value, "axis": axis.value, "split": split.value,
            "configs": [(v[i], c[i]) for i in range(parts.value)]}


def gemm_f32_abi_version() -> int:
    return load().gemm_f32_abi_version()


def config_names(variant: int) -> list[str]:
    return [gemm_f32_config_name(variant, i) for i in range(gemm_f32_config_count(variant))]


def config_id(variant: int, name: str) -> int:
    names = config_names(variant)
    if name not in names:
        raise KeyError(f"variant {variant} has no configuration {name!r}; have {names}")
    return names.index(name)


# ---- tensor-level convenience ----------------------------------------------

def _operand(t, name: str, dims: int) -> tuple[int, int, int]:
    """(op, leading dimension, batch stride) of a float32 GPU tensor holding
    one (dims = 2) or a batch (dims = 3) of matrices.  A row-major matrix is
    OP_N with ld = stride of its rows; a transposed view of a row-major
    matrix (unit stride down the columns, e.g. ``X.T``) is OP_T with ld = the
    stored row stride.  A batch stride of 0 (expanded tensor) is allowed."""
    import torch

    if t.dtype != torch.float32 or t.dim() != dims or not t.is_cuda:
        raise TypeError(f"{name} must be a {dims}-D float32 GPU tensor")
    rows, cols = t.shape[-2], t.shape[-1]
    rs, cs = t.stride(-2), t.stride(-1)
    bs = t.stride(0) if dims == 3 else 0
    if cols <= 1 or cs == 1:
        return OP_N, (rs if rows > 1 else max(cols, 1)), bs
    if rows <= 1 or rs == 1:
        return OP_T, (cs if cols > 1 else max(rows, 1)), bs
    raise ValueError(f"{name} must be row-major or a transposed view of a row-major matrix")


def _marshal(A, B, out, variant, config, stream, batched: bool):
    """Checks the operands and returns (C entry point name, its arguments,
    out) for out = A @ B."""
    import torch

    dims = 3 if batched else 2
    nb = A.shape[0] if batched else 1
    M, K = A.shape[-2], A.shape[-1]
    K2, N = B.shape[-2], B.shape[-1]
    if K != K2 or (batched and B.shape[0] != nb):
        raise ValueError(f"shape mismatch {tuple(A.shape)} x {tuple(B.shape)}")
    opa, lda, sa = _operand(A, "A", dims)
    opb, ldb, sb = _operand(B, "B", dims)
    shape = (nb, M, N) if batched else (M, N)
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=A.device)
    if tuple(out.shape) != shape:
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {shape}")
    opc, ldc, sc = _operand(out, "out", dims)
    if opc != OP_N:
        raise ValueError("out must be row-major")
    sp = (stream if stream is not None else torch.cuda.current_stream(A.device)).cuda_stream
    if variant is None:
        v, c = -1, -1
    else:
        v = VARIANTS[variant] if isinstance(variant, str) else int(variant)
        c = config_id(v, config) if isinstance(config, str) else int(config)
    a, b, cp = A.data_ptr(), B.data_ptr(), out.data_ptr()
    if opa == OP_N and opb == OP_N and not batched:
        if v == -1:
            return "gemm_f32", (M, N, K, a, lda, b, ldb, cp, ldc, sp), out
        return "gemm_f32_variant", (v, c, M, N, K, a, lda, b, ldb, cp, ldc, sp), out
    if opa == OP_N and opb == OP_N:
        if v == -1:
            return ("gemm_f32_strided_batched",
                    (nb, M, N, K, a, lda, sa, b, ldb, sb, cp, ldc, sc, sp), out)
        return ("gemm_f32_strided_batched_variant",
                (v, c, nb, M, N, K, a, lda, sa, b, ldb, sb, cp, ldc, sc, sp), out)
    return ("gemm_f32_ex",
            (v, c, opa, opb, nb, M, N, K, a, lda, sa, b, ldb, sb, cp, ldc, sc, sp), out)


def _call(A, B, out, variant, config, stream, batched: bool):
    name, args, out = _marshal(A, B, out, variant, config, stream, batched)
    rc = getattr(load(), name)(*args)
    if rc != GEMM_F32_OK:
        raise GemmError(rc, gemm_f32_last_error())
    return out


def prepare(A, B, out, *, variant: int | str | None = None, config: int | str = -1,
            stream=None, batched: bool = False):
    """A callable with no arguments that enqueues ``out = A @ B`` (as gemm,
    or gemm_batched when ``batched``), with the operands checked and the C
    arguments built once: for launch loops, where the per-call checks of
    gemm would cost more host time than a small product takes on the GPU.
    The callable holds references to A, B and out, so their memory stays
    allocated while it exists; they must not be resized or re-strided."""
    name, args, _ = _marshal(A, B, out, variant, config, stream, batched)
    fn = getattr(load(), name)

    def launch():
        rc = fn(*args)
        if rc != GEMM_F32_OK:
            raise GemmError(rc, gemm_f32_last_error())

    launch.operands = (A, B, out)  # the raw addresses in args point into these
    return launch


def gemm(A, B, out=None, *, variant: int | str | None = None, config: int | str = -1,
         stream=None):
    """``out = A @ B`` for 2-D float32 GPU tensors through the C ABI.

    A and B may be row-major or transposed views of row-major matrices
    (``X.T``); ``out`` is row-major.  ``variant`` None lets the library
    choose; otherwise a variant id or name with an optional configuration
    id or name.  Enqueued on ``stream`` (a torch.cuda.Stream), default
    torch's current stream; returns ``out`` without synchronising.
    """
    return _call(A, B, out, variant, config, stream, batched=False)


def gemm_splitk(A, B, splits: int, out=None, workspace=None, *, variant: int | str | None = None,
                config: int | str = -1, stream=None, noalloc: bool = False):
    """``out = A @ B`` as `splits` partial products over K plus a fixed-order
    reduction (gemm_f32_splitk).  ``workspace`` is a float32 GPU tensor of at
    least gemm_f32_splitk_workspace_size bytes; allocated here when None.
    With ``noalloc`` the call goes to gemm_f32_splitk_noalloc, whose partial
    products use the library's static scratch (no workspace; ``out`` must be
    given, so that nothing is allocated)."""
    import torch

    if noalloc and (workspace is not None or out is None):
        raise ValueError("noalloc takes an out tensor and no workspace")

    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise ValueError(f"shape mismatch {tuple(A.shape)} x {tuple(B.shape)}")
    opa, lda, _ = _operand(A, "A", 2)
    opb, ldb, _ = _operand(B, "B", 2)
    if opa != OP_N or opb != OP_N:
        raise ValueError("gemm_splitk takes row-major operands")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    opc, ldc, _ = _operand(out, "out", 2)
    need = 0 if noalloc else gemm_f32_splitk_workspace_size(M, N, K, splits)
    if workspace is None and need:
        workspace = torch.empty(need // 4, dtype=torch.float32, device=A.device)
    wptr = workspace.data_ptr() if workspace is not None else None
    wbytes = workspace.numel() * 4 if workspace is not None else 0
    sp = (stream if stream is not None else torch.cuda.current_stream(A.device)).cuda_stream
    if variant is None:
        v, c = -1, -1
    else:
        v = VARIANTS[variant] if isinstance(variant, str) else int(variant)
        c = config_id(v, config) if isinstance(config, str) else int(config)
    if noalloc:
        rc = gemm_f32_splitk_noalloc(v, c, splits, M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb,
                                     out.data_ptr(), ldc, sp)
    else:
        rc = gemm_f32_splitk(v, c, splits, M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb,
                             out.data_ptr(), ldc, wptr, wbytes, sp)
    if rc != GEMM_F32_OK:
        raise GemmError(rc, gemm_f32_last_error())
    return out


def gemm_batched(A, B, out=None, *, variant: int | str | None = None, config: int | str = -1,
                 stream=None):
    """``out[b] = A[b] @ B[b]`` for 3-D float32 GPU tensors (strided batch;
    A or B may be an expanded tensor with batch stride 0, and either may be
    a batch of transposed views)."""
    return _call(A, B, out, variant, config, stream, batched=True)


# ---- microscaled 4-bit floating point (include/gemm_mxfp4.h) ----------------

MXFP4_BLOCK = 32  # values that share a scale


class Mxfp4Matrix(ctypes.Structure):
    """gemm_mxfp4_matrix of the C header."""

    _fields_ = [("codes", _vp), ("ld_codes", _i64), ("stride_codes", _i64),
                ("scales", _vp), ("ld_scales", _i64), ("stride_scales", _i64)]


def _matrix_arg(m):
    return None if m is None else ctypes.byref(m)


def gemm_mxfp4_quantize(batch, rows, cols, X, ldx, sX, Q, QT, stream=None) -> int:
    return load().gemm_mxfp4_quantize(batch, rows, cols, X, ldx, sX, _matrix_arg(Q),
                                      _matrix_arg(QT), stream)


def gemm_mxfp4_dequantize(batch, rows, cols, Q, Y, ldy, sY, stream=None) -> int:
    return load().gemm_mxfp4_dequantize(batch, rows, cols, _matrix_arg(Q), Y, ldy, sY, stream)


def gemm_mxfp4_product(batch, M, N, K, A, B, C, ldc, sC, workspace=None, workspace_bytes=0,
                       stream=None) -> int:
    """The C entry point gemm_mxfp4 (that name is the tensor-level call here)."""
    return load().gemm_mxfp4(batch, M, N, K, _matrix_arg(A), _matrix_arg(B), C, ldc, sC,
                             workspace, workspace_bytes, stream)


def gemm_mxfp4_workspace_size(batch, M, N, K) -> int:
    return load().gemm_mxfp4_workspace_size(batch, M, N, K)


def gemm_mxfp4_weight_product(opW, batch, M, N, K, A, lda, sA, W, C, ldc, sC, workspace=None,
                              workspace_bytes=0, stream=None) -> int:
    """The C entry point gemm_mxfp4_weight (that name is the tensor-level call here)."""
    return load().gemm_mxfp4_weight(opW, batch, M, N, K, A, lda, sA, _matrix_arg(W), C, ldc, sC,
                                    workspace, workspace_bytes, stream)


def gemm_mxfp4_weight_workspace_size(opW, batch, M, N, K) -> int:
    return load().gemm_mxfp4_weight_workspace_size(opW, batch, M, N, K)


def gemm_mxfp4_abi_version() -> int:
    return load().gemm_mxfp4_abi_version()


class Mxfp4:
    """A matrix (or a batch of them) in microscaled 4-bit floating point:
    ``codes`` (..., rows, >= 16 ceil(cols / 32)) and ``scales`` (..., rows,
    >= ceil(cols / 32)), uint8 tensors with unit stride along the last axis,
    in the layout of include/gemm_mxfp4.h, and the number of columns.  Codes
    past ``cols`` in a row's last block of 32 must be zero, which is not
    checked: the products add them to their sums.  It holds the tensors;
    their memory is not copied."""

    __slots__ = ("cols", "shape", "device", "_codes", "_scales", "_memory", "_c")

    def __init__(self, codes, scales, cols: int):
        load()
        if codes.dtype != _torch.uint8 or scales.dtype != _torch.uint8 or not codes.is_cuda:
            raise TypeError("codes and scales must be uint8 GPU tensors")
        if scales.device != codes.device:
            raise ValueError("codes and scales are on different devices")
        *lead, cb = codes.shape
        *lead_s, sb = scales.shape
        if len(lead) not in (1, 2) or lead_s != lead:
            raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scales.shape)} must be "
                             "2-D or 3-D with the same rows")
        cols = int(cols)
        nb = (cols + MXFP4_BLOCK - 1) // MXFP4_BLOCK
        words = (nb + 3) // 4 * 4
        if cols < 0 or cb < nb * 16 or sb < words:
            raise ValueError(f"{cols} columns need {nb * 16} bytes of codes and {words} of scales "
                             f"a row, not {cb} and {sb}")
        ct, st = codes.stride(), scales.stride()
        if (cb > 1 and ct[-1] != 1) or (sb > 1 and st[-1] != 1):
            raise ValueError("codes and scales must have unit stride along the last axis")
        self._codes, self._scales, self._memory = codes, scales, None
        self.cols, self.device = cols, codes.device
        #: (rows, columns) or (batch, rows, columns)
        self.shape = (*lead, cols)
        many, batched = lead[-1] > 1, len(lead) == 2 and lead[0] > 1
        self._c = Mxfp4Matrix(codes.data_ptr(), ct[-2] if many else cb // 16 * 16,
                              ct[0] if batched else 0,
                              scales.data_ptr(), st[-2] if many else sb // 4 * 4,
                              st[0] if batched else 0)

    @property
    def codes(self):
        if self._codes is None:
            self._split()
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            self._split()
        return self._scales

    def _split(self) -> None:
        """The tensors of an mxfp4_empty: its memory is one, codes first."""
        *lead, rows, _ = self.shape
        codes, words = self._c.ld_codes, self._c.ld_scales
        n = (lead[0] if lead else 1) * rows * codes
        self._codes = self._memory[:n].view(*lead, rows, codes)
        self._scales = self._memory[n:].view(*lead, rows, words)

    def __repr__(self) -> str:
        return f"Mxfp4(shape={self.shape}, device={self.device})"


def _empty(shape, strides, dtype, device, stream):
    """torch.empty (the quicker call) for memory that work on ``stream``
    (None: the current one) will use: taken from that stream's pool, so that
    nothing else still uses it, and nothing else gets it before that work is
    done."""
    if stream is None:
        return _torch.empty_strided(shape, strides, dtype=dtype, device=device)
    with _torch.cuda.stream(stream):
        return _torch.empty_strided(shape, strides, dtype=dtype, device=device)


def mxfp4_empty(shape, device="cuda", *, stream=None) -> Mxfp4:
    """An uninitialised Mxfp4 of ``shape`` (rows, cols) or (batch, rows, cols)."""
    load()
    if len(shape) not in (2, 3) or min(shape) < 0:
        raise ValueError(f"shape {tuple(shape)} must be (rows, cols) or (batch, rows, cols)")
    *lead, cols = shape
    nb = (cols + MXFP4_BLOCK - 1) // MXFP4_BLOCK
    words = (nb + 3) // 4 * 4
    rows = lead[-1]
    lines = rows if len(lead) == 1 else lead[0] * rows
    memory = _empty((lines * (nb * 16 + words),), (1,), _torch.uint8, device, stream)
    if not memory.is_cuda:
        raise TypeError(f"an Mxfp4 lies in GPU memory, not on {memory.device}")
    q = Mxfp4.__new__(Mxfp4)  # nothing else to check
    q._codes, q._scales, q._memory = None, None, memory
    q.cols, q.shape, q.device = cols, (*lead, cols), memory.device
    at = memory.data_ptr()
    q._c = Mxfp4Matrix(at, nb * 16, rows * nb * 16, at + lines * nb * 16, words, rows * words)
    return q


def _run_on(device, stream, fn, *args) -> None:
    """Calls a C entry point with the stream as its last argument, with the
    tensors' device current, and raises on an error."""
    index = device.index
    if stream is None:
        # (the raw handle: a torch.cuda.Stream object costs as much as a launch)
        sp = _torch._C._cuda_getCurrentRawStream(index)
    elif stream.device == device:
        sp = stream.cuda_stream
    else:
        raise ValueError(f"stream on {stream.device}, operands on {device}")
    if _torch._C._cuda_getDevice() == index:
        rc = fn(*args, sp)
    else:
        with _torch.cuda.device(device):
            rc = fn(*args, sp)
    if rc != GEMM_F32_OK:
        raise GemmError(rc, gemm_f32_last_error())


def _float_operand(t, name: str, device=None) -> tuple[int, int, int, int]:
    """(op, leading dimension, batch stride, batch) of a 2-D or 3-D tensor, as _operand."""
    dims = t.dim()
    if dims not in (2, 3):
        raise TypeError(f"{name} must be a 2-D or 3-D float32 GPU tensor")
    op, ld, bs = _operand(t, name, dims)
    if device is not None and t.device != device:
        raise ValueError(f"{name} on {t.device}, other operands on {device}")
    batch = t.shape[0] if dims == 3 else 1
    return op, ld, (bs if batch > 1 else 0), batch


def _quantize(X, want_rows: bool, want_cols: bool, stream, out, out_t):
    op, ld, bs, batch = _float_operand(X, "X")
    if op == OP_T:  # X is the transpose of what is stored: so are its blocks
        stored = X.transpose(-1, -2)
        q_cols, q_rows = _quantize(stored, want_cols, want_rows, stream, out_t, out)
        return q_rows, q_cols
    *lead, rows, cols = X.shape
    dev = X.device

    def target(q, shape):
        if q is None:
            return mxfp4_empty(shape, dev, stream=stream)
        if q.shape != shape or q.device != dev:
            raise ValueError(f"out is {q!r}, expected shape {shape} on {dev}")
        return q

    q = target(out, (*lead, rows, cols)) if want_rows else None
    qt = target(out_t, (*lead, cols, rows)) if want_cols else None
    _run_on(dev, stream, load().gemm_mxfp4_quantize, batch, rows, cols, X.data_ptr(), ld, bs,
            None if q is None else ctypes.byref(q._c), None if qt is None else ctypes.byref(qt._c))
    return q, qt


def mxfp4_quantize(X, out: Mxfp4 | None = None, *, stream=None) -> Mxfp4:
    """X (2-D or 3-D float32 GPU tensor, row-major or a transposed view of a
    row-major matrix) rounded to the format, with blocks along its last axis:
    ``mxfp4_quantize(X)`` for a product that sums over X's columns,
    ``mxfp4_quantize(X.T)`` for one that sums over its rows."""
    return _quantize(X, True, False, stream, out, None)[0]


def mxfp4_quantize_both(X, out: Mxfp4 | None = None, out_t: Mxfp4 | None = None, *,
                        stream=None) -> tuple[Mxfp4, Mxfp4]:
    """(mxfp4_quantize(X), mxfp4_quantize(X.transpose(-1, -2))) in one read of
    X, as a training step needs them."""
    return _quantize(X, True, True, stream, out, out_t)


def mxfp4_dequantize(q: Mxfp4, out=None, *, stream=None):
    """The float32 values of ``q``."""
    shape = q.shape
    device = q.device
    out, ld, bs, *_ = _mxfp4_out(out, shape, device, None, 0, stream)
    batch = shape[0] if len(shape) == 3 else 1
    _run_on(device, stream, load().gemm_mxfp4_dequantize, batch, shape[-2], shape[-1],
            ctypes.byref(q._c), out.data_ptr(), ld, bs)
    return out


def _mxfp4_out(out, shape, device, workspace, need: int, stream):
    """(out, its leading dimension and batch stride, workspace pointer and bytes)."""
    if out is None:
        ld = shape[-1] or 1
        bs = shape[-2] * ld
        out = _empty(shape, (ld, 1) if len(shape) == 2 else (bs, ld, 1), _torch.float32, device, stream)
    else:
        if tuple(out.shape) != shape:
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {shape}")
        op, ld, bs, _ = _float_operand(out, "out", device)
        if op != OP_N:
            raise ValueError("out must be row-major")
    if workspace is not None:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {device}")
        return out, ld, bs, workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if need:
        workspace = _empty((need // 4,), (1,), _torch.float32, device, stream)
        return out, ld, bs, workspace, workspace.data_ptr(), need
    return out, ld, bs, None, None, 0


def gemm_mxfp4(A: Mxfp4, B: Mxfp4, out=None, workspace=None, *, stream=None):
    """``out = A @ B.T`` (float32) with A (M x K) and B (N x K) both in the
    format, or a batch of such products (3-D; an expanded batch is allowed).
    ``workspace`` (a GPU tensor of at least gemm_mxfp4_workspace_size bytes)
    is allocated here when the sizes call for one and None is given.
    Enqueued on ``stream``, default torch's current stream."""
    sa, sb = A.shape, B.shape
    if len(sa) != len(sb) or sa[:-2] != sb[:-2] or sa[-1] != sb[-1]:
        raise ValueError(f"shape mismatch {sa} x {sb} transposed")
    device = A.device
    if B.device != device:
        raise ValueError(f"A on {device}, B on {B.device}")
    batch = sa[0] if len(sa) == 3 else 1
    M, N, K = sa[-2], sb[-2], sa[-1]
    lib = load()
    out, ldc, sc, workspace, wp, wb = _mxfp4_out(
        out, (*sa[:-1], N), device, workspace, lib.gemm_mxfp4_workspace_size(batch, M, N, K),
        stream)
    _run_on(device, stream, lib.gemm_mxfp4, batch, M, N, K, ctypes.byref(A._c),
            ctypes.byref(B._c), out.data_ptr(), ldc, sc, wp, wb)
    return out


def gemm_mxfp4_weight(A, W: Mxfp4, out=None, workspace=None, *, op: int = OP_T, stream=None):
    """``out = A @ W.T`` (op = OP_T: W is N x K, a stored layer) or ``A @ W``
    (op = OP_N: W is K x N; with A the gradient of the former's result, the
    gradient with respect to its activations).  A is a row-major float32 GPU
    tensor, 2-D, or 3-D with a batch of W; it is not rounded.  ``workspace``
    and ``stream`` as in gemm_mxfp4."""
    if op not in (OP_N, OP_T):
        raise ValueError("op must be OP_N or OP_T")
    device = W.device
    opa, lda, sa, batch = _float_operand(A, "A", device)
    if opa != OP_N:
        raise ValueError("A must be row-major")
    *lead, M, K = A.shape
    *lead_w, N, K2 = W.shape
    if op == OP_N:
        N, K2 = K2, N
    if K != K2 or lead != lead_w:
        raise ValueError(f"shape mismatch {tuple(A.shape)} x {W.shape}{' transposed' if op == OP_T else ''}")
    lib = load()
    out, ldc, sc, workspace, wp, wb = _mxfp4_out(
        out, (*lead, M, N), device, workspace,
        lib.gemm_mxfp4_weight_workspace_size(op, batch, M, N, K), stream)
    _run_on(device, stream, lib.gemm_mxfp4_weight, op, batch, M, N, K, A.data_ptr(), lda, sa,
            ctypes.byref(W._c), out.data_ptr(), ldc, sc, wp, wb)
    return out
