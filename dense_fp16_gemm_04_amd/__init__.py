"""fp16 C = A * B^T on AMD Instinct MI355X (gfx950).

The product runs in hand-written HIP kernels behind a C ABI
(``include/gemm_nt_f16.h``, built into ``libgemm_nt_f16.so`` in this
package).  The Python functions here only marshal arguments; the library is
loaded on first use and an error is raised if it is missing.

Beside it stand the operators of a linear layer's life, each with a library
and a C ABI of its own: the gated feed-forward layer and its gradients
(``gated_nt``, ``gated_nt_train``, ``gated_nt_backward``), the orthogonalised
update of a weight (``orthogonalize_ns``) and the product with 4-bit weights
(``gemv_w4``).
"""
from __future__ import annotations

__all__ = [
    "gemm_nt_f16",
    "gemm_nt_f16_ex",
    "gemm_nt_f16_config_name",
    "gemm_nt_f16_select",
    "gemm_nt_f16_version",
    "variants",
    "library_path",
    "load",
    "GemmError",
    "gated_nt",
    "gated_nt_train",
    "gated_nt_backward",
    "orthogonalize_ns",
    "gemv_w4",
]

_OPERATORS = ("gated_nt", "gated_nt_train", "gated_nt_backward", "orthogonalize_ns", "gemv_w4")


def __getattr__(name):
    if name in _OPERATORS:
        from . import operators
        return getattr(operators, name)
    if name in __all__:
        from . import binding
        return getattr(binding, name)
    raise AttributeError(name)
