"""fp16 C = A * B^T on AMD Instinct MI355X (gfx950).

The product runs in hand-written HIP kernels behind a C ABI
(``include/gemm_nt_f16.h``, built into ``libgemm_nt_f16.so`` in this
package).  The Python functions here only marshal arguments; the library is
loaded on first use and an error is raised if it is missing.

Beside it stand the operators of a linear layer's life, each with a library
and a C ABI of its own: the gated feed-forward layer and its gradients
(``gated_nt``, ``gated_nt_train``, ``gated_nt_backward``), the orthogonalised
update of a weight (``orthogonalize_ns``) and the product with 4-bit weights
(``gemv_w4``).  Around them stand those of a training step: the layer norm
(``layer_norm``, ``layer_norm_train``, ``layer_norm_backward``), dropout with
the sum of a residual (``dropout``, ``dropout_backward``) and the loss over a
vocabulary (``linear_cross_entropy``, ``linear_cross_entropy_train``,
``linear_cross_entropy_backward``).
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
    "layer_norm",
    "layer_norm_train",
    "layer_norm_backward",
    "dropout",
    "dropout_backward",
    "linear_cross_entropy",
    "linear_cross_entropy_train",
    "linear_cross_entropy_backward",
]

_OPERATORS = ("gated_nt", "gated_nt_train", "gated_nt_backward", "orthogonalize_ns", "gemv_w4")
_TRAINING = ("layer_norm", "layer_norm_train", "layer_norm_backward", "dropout", "dropout_backward", "linear_cross_entropy",
             "linear_cross_entropy_train", "linear_cross_entropy_backward")


def __getattr__(name):
    # (the first time; then it is the module's own)
    if name in _OPERATORS:
        from . import operators as module
    elif name in _TRAINING:
        from . import training as module
    elif name in __all__:
        from . import binding as module
    else:
        raise AttributeError(name)
    value = globals()[name] = getattr(module, name)
    return value
