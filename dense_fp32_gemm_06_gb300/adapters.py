"""Low-rank adapters of many requests beside a shared projection (argument
marshalling only; include/adapters_gb300.h states the operation, the layout
and the errors).

    Y[t] = X[t] @ W + H[t] @ B[a],   H[t] = scale[a] * X[t] @ A[a].T,   a = ids[t]

X is T x K, W is K x N (row-major or a transposed view of a row-major N x K
matrix), A is L x R x K and B is L x R x N, both contiguous.  Rows of any
mixture of adapters may follow one another; a row whose id is outside
0 .. L-1 (say -1) has none.  Matrices are float32 or bfloat16, all of one
type; ids int32; scale and H float32.
"""
from __future__ import annotations

import torch

from . import _native
from ._native import SgemmError

F32, BF16, F16 = 0, 1, 2
DTYPES = {torch.float32: F32, torch.bfloat16: BF16}


def check_status(status: int):
    if status:
        lib = _native.load()
        msg = lib.adapters_status_string(status).decode()
        if status == 100:
            msg += f" (cudaError {lib.adapters_last_cuda_error()})"
        raise SgemmError(status, msg)


def device_status(clear: bool = False) -> int:
    """The status word of these operators' bounded waits (0: none has run
    out); synchronises the device; resets it when `clear`."""
    import ctypes
    flag = ctypes.c_int(0)
    check_status(_native.load().adapters_device_status(ctypes.byref(flag), int(bool(clear))))
    return flag.value


def need(ok, message):
    if not ok:
        raise SgemmError(-1, message)


def matrix(t, name, dtype, rows, cols, device):
    """Row pitch of a rows x cols row-major tensor of that type on that device."""
    need(t.is_cuda and t.dtype == dtype and t.device == device and t.dim() == 2,
         f"{name} must be a 2-D {dtype} CUDA tensor on the same device")
    need(t.shape[0] == rows and t.shape[1] == cols, f"shape mismatch: {name} is {tuple(t.shape)}, not {(rows, cols)}")
    need(cols <= 1 or t.stride(1) == 1, f"{name} must have unit column stride (row-major)")
    return max(t.stride(0) if rows > 1 else cols, cols, 1)


def vector(t, name, dtype, shape, device):
    """Pointer of a contiguous tensor of that shape, 0 for None."""
    if t is None:
        return 0
    need(t.is_cuda and t.dtype == dtype and t.device == device and t.is_contiguous(),
         f"{name} must be a contiguous {dtype} CUDA tensor on the same device")
    need(t.shape == shape, f"shape mismatch: {name} is {tuple(t.shape)}, not {tuple(shape)}")
    return t.data_ptr()


def _weight(W, dtype, device):
    """(op, ld) of W: row-major (0) or a transposed view of a row-major matrix (1)."""
    need(W.is_cuda and W.dtype == dtype and W.device == device and W.dim() == 2,
         f"W must be a 2-D {dtype} CUDA tensor on the same device")
    rows, cols = W.shape
    if cols <= 1 or W.stride(1) == 1:
        return 0, max(W.stride(0) if rows > 1 else cols, cols, 1)
    if rows <= 1 or W.stride(0) == 1:
        return 1, max(W.stride(1), rows, 1)
    raise SgemmError(-1, "W must be row-major or a transposed view of a row-major tensor")


def on_device(device, call, stream):
    """call(stream handle) with `device` current."""
    if stream is None:
        stream = torch.cuda.current_stream(device).cuda_stream
    if device.index == torch.cuda.current_device():
        check_status(call(stream))
    else:
        with torch.cuda.device(device):
            check_status(call(stream))


def _stacks(A, B, K, N, dtype, device):
    need(A.dim() == 3 and B.dim() == 3, "A and B must be 3-D: L x R x K and L x R x N")
    L, R = A.shape[0], A.shape[1]
    return L, R, vector(A, "A", dtype, (L, R, K), device), vector(B, "B", dtype, (L, R, N), device)


def lora_forward(X, W, A, B, ids, Y, scale=None, *, H=None, stream=None):
    """Y = X @ W + H @ B[ids] in place, H = scale[ids] * X @ A[ids].T; a training
    step passes H (T x R float32) to keep it for ``lora_backward``.  Runs on
    ``stream`` (default: torch's current stream of Y's device).  Returns Y."""
    need(X.dim() == 2 and W.dim() == 2, "X and W must be 2-D")
    device, dtype = Y.device, X.dtype
    need(dtype in DTYPES, "X must be float32 or bfloat16")
    T, K = X.shape
    N = W.shape[1]
    need(W.shape[0] == K, f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}")
    ldx, ldy = matrix(X, "X", dtype, T, K, device), matrix(Y, "Y", dtype, T, N, device)
    op, ldw = _weight(W, dtype, device)
    L, R, a, b = _stacks(A, B, K, N, dtype, device)
    i, s, h = (vector(ids, "ids", torch.int32, (T,), device), vector(scale, "scale", torch.float32, (L,), device),
               vector(H, "H", torch.float32, (T, R), device))
    lib = _native.load()
    on_device(device, lambda st: lib.lora_forward(T, K, N, L, R, DTYPES[dtype], X.data_ptr(), ldx, op, W.data_ptr(), ldw,
                                                  a, b, i, s, Y.data_ptr(), ldy, h, st), stream)
    return Y


def lora_backward(dY, X, W, A, B, ids, H, dX=None, dA=None, dB=None, scale=None, *, stream=None):
    """The gradients of ``lora_forward`` by X and the adapters (W is frozen),
    into those of dX (T x K), dA (L x R x K) and dB (L x R x N) that are given;
    H is the forward call's.  Returns (dX, dA, dB)."""
    need(dY.dim() == 2 and X.dim() == 2 and W.dim() == 2, "dY, X and W must be 2-D")
    device, dtype = dY.device, dY.dtype
    need(dtype in DTYPES, "dY must be float32 or bfloat16")
    T, K = X.shape
    N = W.shape[1]
    need(W.shape[0] == K, f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}")
    lddy, ldx = matrix(dY, "dY", dtype, T, N, device), matrix(X, "X", dtype, T, K, device)
    op, ldw = _weight(W, dtype, device)
    L, R, a, b = _stacks(A, B, K, N, dtype, device)
    i, s, h = (vector(ids, "ids", torch.int32, (T,), device), vector(scale, "scale", torch.float32, (L,), device),
               vector(H, "H", torch.float32, (T, R), device))
    lddx = matrix(dX, "dX", dtype, T, K, device) if dX is not None else max(K, 1)
    da, db = vector(dA, "dA", dtype, (L, R, K), device), vector(dB, "dB", dtype, (L, R, N), device)
    lib = _native.load()
    on_device(device, lambda st: lib.lora_backward(T, K, N, L, R, DTYPES[dtype], dY.data_ptr(), lddy, X.data_ptr(), ldx, op,
                                                   W.data_ptr(), ldw, a, b, i, s, h, dX.data_ptr() if dX is not None else 0,
                                                   lddx, da, db, st), stream)
    return dX, dA, dB
