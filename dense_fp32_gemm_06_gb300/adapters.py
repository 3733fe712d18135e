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


def refuse(message):
    raise SgemmError(-1, message)


MOST = 0x7FFFFFFF   # the C ABI's int

# The checks below run on every call, beside kernels of a few microseconds:
# they look at attributes only, and make a message once one has failed.
# `dev` is the index of the CUDA device.

def matrix(t, name, dtype, rows, cols, dev):
    """Row pitch of a rows x cols row-major tensor of that type on that device."""
    if t.dtype is not dtype or t.get_device() != dev or t.dim() != 2:
        refuse(f"{name} must be a 2-D {dtype} CUDA tensor on device {dev}")
    if t.shape != (rows, cols):
        refuse(f"shape mismatch: {name} is {tuple(t.shape)}, not {(rows, cols)}")
    pitch, one = t.stride()
    if one != 1 and cols > 1:
        refuse(f"{name} must have unit column stride (row-major)")
    if rows <= 1:
        pitch = cols or 1
    if pitch < cols or pitch > MOST or rows > MOST:
        refuse(f"{name} must have rows that do not overlap, of less than 2^31 elements")
    return pitch or 1


def vector(t, name, dtype, shape, dev):
    """Pointer of a contiguous tensor of that shape, 0 for None."""
    if t is None:
        return 0
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.shape == shape:
        return t.data_ptr()
    if t.shape != shape:
        refuse(f"shape mismatch: {name} is {tuple(t.shape)}, not {tuple(shape)}")
    refuse(f"{name} must be a contiguous {dtype} CUDA tensor on device {dev}")


def launch(fn, dev, stream, *args):
    """fn(*args, stream) with device `dev` current; the stream is torch's current one of it unless given."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    if dev == torch.cuda.current_device():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status:
        check_status(status)


def _problem(X, W, A, B, N, dev, dtype):
    """(T, K, L, R, op, ldw, pointers of the stacks) of the shared checks."""
    if X.dim() != 2 or W.dim() != 2 or A.dim() != 3 or B.dim() != 3:
        refuse("X and W must be 2-D, A (L x R x K) and B (L x R x N) 3-D")
    T, K = X.shape
    L, R, _ = A.shape
    if W.shape != (K, N):
        refuse(f"shape mismatch: W is {tuple(W.shape)}, not {(K, N)}")
    if dtype not in DTYPES or dev < 0:
        refuse("the matrices must be float32 or bfloat16 CUDA tensors")
    if W.dtype is not dtype or W.get_device() != dev:
        refuse(f"W must be a {dtype} CUDA tensor on device {dev}")
    s0, s1 = W.stride()
    if N <= 1 or s1 == 1:
        op, ldw, least = 0, s0 if K > 1 else N, N
    elif K <= 1 or s0 == 1:
        op, ldw, least = 1, s1, K
    else:
        refuse("W must be row-major or a transposed view of a row-major tensor")
    if ldw < least or ldw > MOST or L > MOST:
        refuse("W must have rows that do not overlap, of less than 2^31 elements")
    return T, K, L, R, op, ldw or 1, vector(A, "A", dtype, (L, R, K), dev), vector(B, "B", dtype, (L, R, N), dev)


def lora_forward(X, W, A, B, ids, Y, scale=None, *, H=None, stream=None):
    """Y = X @ W + H @ B[ids] in place, H = scale[ids] * X @ A[ids].T; a training
    step passes H (T x R float32) to keep it for ``lora_backward``.  Runs on
    ``stream`` (default: torch's current stream of Y's device).  Returns Y."""
    dev, dtype = Y.get_device(), Y.dtype
    N = Y.shape[-1]
    T, K, L, R, op, ldw, a, b = _problem(X, W, A, B, N, dev, dtype)
    launch(_native.load().lora_forward, dev, stream, T, K, N, L, R, DTYPES[dtype],
           X.data_ptr(), matrix(X, "X", dtype, T, K, dev), op, W.data_ptr(), ldw, a, b,
           vector(ids, "ids", torch.int32, (T,), dev), vector(scale, "scale", torch.float32, (L,), dev),
           Y.data_ptr(), matrix(Y, "Y", dtype, T, N, dev), vector(H, "H", torch.float32, (T, R), dev))
    return Y


def lora_backward(dY, X, W, A, B, ids, H, dX=None, dA=None, dB=None, scale=None, *, stream=None):
    """The gradients of ``lora_forward`` by X and the adapters (W is frozen),
    into those of dX (T x K), dA (L x R x K) and dB (L x R x N) that are given;
    H is the forward call's.  Returns (dX, dA, dB)."""
    dev, dtype = dY.get_device(), dY.dtype
    N = dY.shape[-1]
    T, K, L, R, op, ldw, a, b = _problem(X, W, A, B, N, dev, dtype)
    x_ptr, lddx = (dX.data_ptr(), matrix(dX, "dX", dtype, T, K, dev)) if dX is not None else (0, K or 1)
    launch(_native.load().lora_backward, dev, stream, T, K, N, L, R, DTYPES[dtype],
           dY.data_ptr(), matrix(dY, "dY", dtype, T, N, dev), X.data_ptr(), matrix(X, "X", dtype, T, K, dev),
           op, W.data_ptr(), ldw, a, b, vector(ids, "ids", torch.int32, (T,), dev),
           vector(scale, "scale", torch.float32, (L,), dev), vector(H, "H", torch.float32, (T, R), dev), x_ptr, lddx,
           vector(dA, "dA", dtype, (L, R, K), dev), vector(dB, "dB", dtype, (L, R, N), dev))
    return dX, dA, dB
