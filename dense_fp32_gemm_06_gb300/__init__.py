"""GB300-native single-precision GEMM: C = alpha*A*B + beta*C (row-major FP32),
with the operators that train and serve low-rank adapters beside such a
product: ``lora_forward`` / ``lora_backward`` and the losses ``distill_topk``
and ``policy_loss``.

The compute path is the C-ABI CUDA library built from ``csrc/`` for sm_103a;
the functions below only marshal arguments to it.  Importing the package does
not load the library; the first call does, and raises if it is missing.
"""
from .binding import sgemm, sgemm_ex, SgemmError, PATH_AUTO, PATH_FFMA, PATH_TF32X3  # noqa: F401

__all__ = ["sgemm", "sgemm_ex", "SgemmError", "PATH_AUTO", "PATH_FFMA", "PATH_TF32X3",
           "lora_forward", "lora_backward", "distill_topk", "policy_loss"]

_OPERATORS = {"lora_forward": "adapters", "lora_backward": "adapters", "distill_topk": "losses", "policy_loss": "losses"}


def __getattr__(name):
    # these modules import torch: only once one of their functions is asked for
    if name in _OPERATORS:
        from importlib import import_module
        value = getattr(import_module("." + _OPERATORS[name], __name__), name)
        globals()[name] = value
        return value
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
