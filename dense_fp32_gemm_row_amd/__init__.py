"""Row-major FP32 GEMM (C = A x B) for AMD MI355X (gfx950).

The product is computed by hand-written HIP kernels behind the C-ABI library
``libgemm_f32.so`` (declared in ``include/gemm_f32.h``).  ``binding`` is the
thin ctypes layer over it; importing this package does not load the library,
so the seeded input generators in ``workloads`` stay usable without a GPU.
"""

from __future__ import annotations

__all__ = ["gemm", "gemm_f32", "gemm_f32_variant", "gemm_f32_strerror", "Mxfp4", "mxfp4_empty",
           "mxfp4_quantize", "mxfp4_quantize_both", "mxfp4_dequantize", "gemm_mxfp4", "gemm_mxfp4_weight", "OP_N",
           "OP_T", "workloads"]


def __getattr__(name):
    if name in __all__ and name != "workloads":
        from . import binding

        return getattr(binding, name)
    if name == "workloads":
        from importlib import import_module  # (a `from . import` would come back here)

        return import_module(".workloads", __name__)
    raise AttributeError(name)
