"""Matrices kept in 4 or 8 bits with a power of two per 32 values, and the
products that read them (argument marshalling only;
include/microscale_gb300.h states the format, the operations and the errors).

A coded matrix of rows x cols is two tensors, as ``mx_empty`` makes them:
``codes``, uint8 of rows x 16 ceil(cols / 32) (4 bits, two codes a byte) or
int8 of rows x 32 ceil(cols / 32) (8 bits), and ``scales``, uint8 of rows x
ceil(cols / 32); both start at multiples of 16 bytes, and so do their rows.
Real matrices are float32 or bfloat16, row-major, all of one type in a call.
Every call runs on ``stream`` (default: torch's current stream of the real
matrix's device).
"""
from __future__ import annotations

import torch

from . import _native
from ._native import SgemmError
from .adapters import run


def _check_status(status: int):
    if status:
        lib = _native.load()
        msg = lib.mx_status_string(status).decode()
        if status == 100:
            msg += f" (cudaError {lib.mx_last_cuda_error()})"
        raise SgemmError(status, msg)


def device_status(clear: bool = False) -> int:
    """The status word of these operators' bounded waits (0: none has run
    out); synchronises the device; resets it when `clear`."""
    import ctypes
    flag = ctypes.c_int(0)
    _check_status(_native.load().mx_device_status(ctypes.byref(flag), int(bool(clear))))
    return flag.value


def plan(call: str, t: int, k: int, n: int, dtype=torch.bfloat16, bits: int = 4) -> dict:
    """How the current device runs ``call`` ("linear", "grad_input" or
    "grad_weight") of these sizes: rows of a tile, CTAs that split its
    contraction, whether CTA pairs share tiles, and the most tiles that one of
    them takes."""
    p = _native.AdaptersPlan()
    kind = {"linear": 0, "grad_input": 1, "grad_weight": 2}.get(call, -1)
    _check_status(_native.load().mx_plan_for(kind, t, k, n, {torch.float32: 0, torch.bfloat16: 1}.get(dtype, -1), bits, p))
    return {name: getattr(p, name) for name, _ in p._fields_}


def mx_empty(rows: int, cols: int, bits: int, device="cuda"):
    """(codes, scales) for a rows x cols matrix in 4 or 8 bits, not written yet."""
    if bits not in (4, 8):
        raise SgemmError(-1, f"bits must be 4 or 8, not {bits}")
    if rows < 0 or cols < 0:
        raise SgemmError(-1, f"sizes must not be negative: {rows} x {cols}")
    blocks = (cols + 31) // 32
    codes = torch.empty(rows, blocks * bits * 4, dtype=torch.uint8 if bits == 4 else torch.int8, device=device)
    return codes, torch.empty(rows, (blocks + 15) // 16 * 16, dtype=torch.uint8, device=device)[:, :blocks]


def mx_quantize(X, codes, scales, *, stream=None):
    """X (rows x cols, row-major or a transposed view of a row-major matrix)
    into codes and scales, in the codes' number of bits, rounded to nearest.
    Returns (codes, scales)."""
    run("mx_quantize", X, stream, X, codes, scales, check=_check_status)
    return codes, scales


def mx_dequantize(codes, scales, Y, *, stream=None):
    """The values of codes and scales into Y (rows x cols).  Returns Y."""
    run("mx_dequantize", Y, stream, codes, scales, Y, check=_check_status)
    return Y


def mx4_linear(X, codes, scales, Y, *, stream=None):
    """Y = Q(X) @ W.T: X (T x K) rounded to 4 bits within the call as
    ``mx_quantize`` does, W (N x K) as codes and scales in 4 bits, on the
    tensor cores' 4-bit rate.  Returns Y (T x N)."""
    run("mx4_linear", Y, stream, X, codes, scales, Y, check=_check_status)
    return Y


def mx4_matmul(x_codes, x_scales, codes, scales, Y, *, stream=None):
    """Y = X @ W.T of two matrices in 4 bits, X (T x K) and W (N x K): for an
    X that several projections read.  Returns Y (T x N)."""
    run("mx4_matmul", Y, stream, x_codes, x_scales, codes, scales, Y, check=_check_status)
    return Y


def mx_grad_input(dY, codes, scales, dX, *, stream=None):
    """dX = dY @ W, the gradient of ``mx4_linear`` by X straight through its
    rounding; W (N x K) in 4 or 8 bits.  Returns dX (T x K)."""
    run("mx_grad_input", dY, stream, dY, codes, scales, dX, check=_check_status)
    return dX


def mx_grad_weight(dY, codes, scales, dW, *, accumulate=False, stream=None):
    """dW = dY.T @ X, or with ``accumulate`` added to dW, from a checkpoint of
    X (T x K) in 8 or 4 bits.  Returns dW (N x K)."""
    run("mx_grad_weight", dY, stream, dY, codes, scales, dW, accumulate, check=_check_status)
    return dW
