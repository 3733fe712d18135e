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


def plan(t: int, k: int, n: int) -> dict:
    """How the current device runs the bfloat16 projection of t rows from k to
    n features: rows of a tile, CTAs that split its contraction, whether CTA
    pairs share tiles, and the most tiles that one of them takes."""
    p = _native.AdaptersPlan()
    check_status(_native.load().adapters_plan_for(t, k, n, p))
    return {name: getattr(p, name) for name, _ in p._fields_}


MESSAGES = {
    "type": "{name} must be a {dtype} CUDA tensor on device {dev}",
    "contiguous": "{name} must be a contiguous {dtype} CUDA tensor on device {dev}",
    "shape": "shape mismatch: {name} is {shape}, which does not go with the other arguments",
    "one axis": "{name} must have one axis", "two axes": "{name} must be 2-D", "three axes": "{name} must be 3-D",
    "columns": "{name} must have unit column stride (row-major)",
    "transposed": "{name} must be row-major or a transposed view of a row-major tensor",
    "rows": "{name} must have rows that do not overlap, of less than 2^31 elements",
    "missing": "{name} is missing",
    "matrices": "the matrices must be float32 or bfloat16 CUDA tensors",
    "logits": "logits must be a 2-D float32, bfloat16 or float16 CUDA tensor",
    "kl_coef": "kl_coef needs ref",
    "codes": "{name} must be a CUDA tensor of uint8 (4 bits, two codes a byte) or int8 (8 bits)",
    "codes of 4 bits": "{name} must be a CUDA tensor of uint8 (4 bits, two codes a byte)",
    "sixteen": "{name} must start at a multiple of 16 bytes, and its rows be multiples of 16 bytes apart",
}


def _refuse(what, name, t, dtype, dev):
    raise SgemmError(-1, MESSAGES[what].format(name=name, dtype=dtype, dev=dev, shape=tuple(t.shape) if t is not None else None))


_operands = None
# (looked up once: each call asks both, and a torch without CUDA has neither)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _load_operands():
    global _operands
    _operands = _native.load_operands(lambda m: m.setup(_refuse, torch.float32, torch.bfloat16, torch.float16, torch.int32, torch.uint8, torch.int8))
    return _operands


def run(name, main, stream, *args, check=check_status):
    """The C ABI's `name` on the device of tensor `main`, on its current torch
    stream unless one is given; the extension module looks `args` over."""
    dev = -1 if main is None else main.get_device()
    call = getattr(_operands or _load_operands(), name)
    address = _native.load().address[name]
    if dev < 0:
        status = call(address, dev, 0, *args)   # refused
    else:
        if stream is None:
            stream = _raw_stream(dev)
        if dev == _current_device():   # (a CUDA tensor is there: CUDA is initialised)
            status = call(address, dev, stream, *args)
        else:
            with torch.cuda.device(dev):
                status = call(address, dev, stream, *args)
    if status:
        check(status)


def lora_forward(X, W, A, B, ids, Y, scale=None, *, H=None, stream=None):
    """Y = X @ W + H @ B[ids] in place, H = scale[ids] * X @ A[ids].T; a training
    step passes H (T x R float32) to keep it for ``lora_backward``.  Runs on
    ``stream`` (default: torch's current stream of Y's device).  Returns Y."""
    run("lora_forward", Y, stream, X, W, A, B, ids, Y, scale, H)
    return Y


def lora_backward(dY, X, W, A, B, ids, H, dX=None, dA=None, dB=None, scale=None, *, stream=None):
    """The gradients of ``lora_forward`` by X and the adapters (W is frozen),
    into those of dX (T x K), dA (L x R x K) and dB (L x R x N) that are given;
    H is the forward call's.  What those do not need may be None: H without dB,
    X without dA, W and A without dX, B with dB alone.  Returns (dX, dA, dB)."""
    run("lora_backward", dY, stream, dY, X, W, A, B, ids, H, dX, dA, dB, scale)
    return dX, dA, dB
