"""The microscaled operators without a GPU: the header's functions are the
exported ones, every invalid argument is refused by its position before any
CUDA call, the binding refuses tensors that do not go together, and the 64-bit
forms that the GPU tests compare with round to the nearest code and have the
gradients that differences show."""
import os
import re

import numpy as np
import pytest
import torch

import dense_fp32_gemm_06_gb300 as lib
import mx_oracle as mo
from dense_fp32_gemm_06_gb300 import _native

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 4096   # a pointer that is aligned and never read: every call below ends before any CUDA call


def test_header_and_exports():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "microscale_gb300.h")).read(), flags=re.S)
    names = re.findall(r"^\s*(?:int|const\s+char\s*\*)\s*(\w+)\s*\(", text, flags=re.M)
    assert set(names) == set(_native.MX_EXPORTS)
    for checked in (False, True):
        so = _native.load(checked=checked)
        for name in names:
            assert hasattr(so, name), name


def test_status_strings():
    so = _native.load()
    for st in range(1, 15):
        assert so.mx_status_string(st).decode().startswith(f"invalid argument {st}")
    assert b"unknown" not in so.mx_status_string(100)
    assert so.mx_status_string(12345) == b"unknown status"


QUANTIZE = dict(rows=4, cols=40, dtype=0, op=0, X=P, ldx=40, bits=4, codes=P, ldc=32, scales=P, lds=16, stream=0)
DEQUANTIZE = dict(rows=4, cols=40, dtype=0, bits=8, codes=P, ldc=64, scales=P, lds=16, Y=P, ldy=40, stream=0)
LINEAR = dict(t=3, k=40, n=5, dtype=0, X=P, ldx=40, W=P, ldw=32, ws=P, ldws=16, Y=P, ldy=5, stream=0)
MATMUL = dict(t=3, k=40, n=5, dtype=1, X=P, ldx=32, xs=P, ldxs=16, W=P, ldw=32, ws=P, ldws=16, Y=P, ldy=5, stream=0)
GRAD_INPUT = dict(t=3, k=40, n=5, dtype=0, dY=P, lddy=5, bits=4, W=P, ldw=32, ws=P, ldws=16, dX=P, lddx=40, stream=0)
GRAD_WEIGHT = dict(t=3, k=40, n=5, dtype=0, dY=P, lddy=5, bits=8, X=P, ldx=64, xs=P, ldxs=16, accumulate=0, dW=P, lddw=40, stream=0)


def call(name, base, over):
    return getattr(_native.load(), name)(*{**base, **over}.values())


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), 1), (dict(cols=-1), 2), (dict(dtype=2), 3), (dict(op=2), 4), (dict(X=0), 5), (dict(X=P + 2), 5), (dict(ldx=39), 6),
    (dict(op=1, ldx=3), 6), (dict(bits=5), 7), (dict(codes=0), 8), (dict(codes=P + 8), 8), (dict(ldc=16), 9), (dict(ldc=40), 9),
    (dict(bits=8, ldc=48), 9), (dict(scales=0), 10), (dict(scales=P + 1), 10), (dict(lds=8), 11), (dict(cols=544, ldx=544, ldc=272, lds=16), 11),
])
def test_quantize_refusals(over, status):
    assert call("mx_quantize", QUANTIZE, over) == status


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), 1), (dict(cols=-1), 2), (dict(dtype=-1), 3), (dict(bits=0), 4), (dict(codes=0), 5), (dict(ldc=48), 6), (dict(scales=P + 4), 7),
    (dict(lds=17), 8), (dict(Y=0), 9), (dict(Y=P + 1), 9), (dict(ldy=39), 10),
])
def test_dequantize_refusals(over, status):
    assert call("mx_dequantize", DEQUANTIZE, over) == status


@pytest.mark.parametrize("over,status", [
    (dict(t=-1), 1), (dict(k=-1), 2), (dict(n=-1), 3), (dict(dtype=2), 4), (dict(X=0), 5), (dict(X=P + 1), 5), (dict(ldx=39), 6), (dict(W=0), 7),
    (dict(W=P + 8), 7), (dict(ldw=16), 8), (dict(ldw=33), 8), (dict(ws=P + 8), 9), (dict(ldws=0), 10), (dict(Y=0), 11), (dict(ldy=4), 12),
])
def test_linear_refusals(over, status):
    assert call("mx4_linear", LINEAR, over) == status


@pytest.mark.parametrize("over,status", [
    (dict(t=-1), 1), (dict(k=-1), 2), (dict(n=-1), 3), (dict(dtype=2), 4), (dict(X=P + 8), 5), (dict(ldx=16), 6), (dict(xs=0), 7), (dict(ldxs=20), 8),
    (dict(W=0), 9), (dict(ldw=31), 10), (dict(ws=P + 2), 11), (dict(ldws=15), 12), (dict(Y=P + 1), 13), (dict(ldy=4), 14),
])
def test_matmul_refusals(over, status):
    assert call("mx4_matmul", MATMUL, over) == status


@pytest.mark.parametrize("over,status", [
    (dict(t=-1), 1), (dict(k=-1), 2), (dict(n=-1), 3), (dict(dtype=2), 4), (dict(dY=0), 5), (dict(lddy=4), 6), (dict(bits=6), 7), (dict(W=0), 8),
    (dict(ldw=16), 9), (dict(ws=0), 10), (dict(ldws=8), 11), (dict(dX=0), 12), (dict(lddx=39), 13),
])
def test_grad_input_refusals(over, status):
    assert call("mx_grad_input", GRAD_INPUT, over) == status


@pytest.mark.parametrize("over,status", [
    (dict(t=-1), 1), (dict(k=-1), 2), (dict(n=-1), 3), (dict(dtype=2), 4), (dict(dY=P + 2), 5), (dict(lddy=4), 6), (dict(bits=16), 7), (dict(X=P + 4), 8),
    (dict(ldx=32), 9), (dict(xs=0), 10), (dict(ldxs=12), 11), (dict(dW=0), 13), (dict(lddw=39), 14),
])
def test_grad_weight_refusals(over, status):
    assert call("mx_grad_weight", GRAD_WEIGHT, over) == status


@pytest.mark.parametrize("args,status", [((-1, 1, 1, 1, 0, 4), 1), ((3, 1, 1, 1, 0, 4), 1), ((0, 0, 1, 1, 0, 4), 2), ((1, 1, 0, 1, 0, 4), 3), ((1, 1, 1, 0, 0, 4), 4),
                                         ((0, 1, 1, 1, 2, 4), 5), ((1, 1, 1, 1, 0, 5), 6), ((2, 1, 1, 1, 1, 0), 6), ((0, 1, 1, 1, 0, 4), 7)])
def test_plan_refusals(args, status):
    assert _native.load().mx_plan_for(*args, None) == status


@pytest.mark.parametrize("name,base,over", [
    ("mx_quantize", QUANTIZE, dict(rows=0, X=0, codes=0, scales=0)), ("mx_quantize", QUANTIZE, dict(cols=0, X=0, codes=0, scales=0)),
    ("mx_dequantize", DEQUANTIZE, dict(rows=0, codes=0, scales=0, Y=0)), ("mx4_linear", LINEAR, dict(t=0, X=0, Y=0)),
    ("mx4_linear", LINEAR, dict(n=0, X=0, W=0, ws=0, Y=0)), ("mx4_matmul", MATMUL, dict(n=0, W=0, ws=0, Y=0)),
    ("mx_grad_input", GRAD_INPUT, dict(t=0, dY=0, dX=0)), ("mx_grad_input", GRAD_INPUT, dict(k=0, W=0, ws=0, dX=0)),
    ("mx_grad_weight", GRAD_WEIGHT, dict(n=0, dY=0, dW=0)), ("mx_grad_weight", GRAD_WEIGHT, dict(t=0, dY=0, X=0, xs=0, accumulate=1)),
])
def test_calls_of_nothing(name, base, over):
    assert call(name, base, over) == 0


def test_the_binding_refuses_cpu_tensors_and_missing_ones():
    x, (c, s) = torch.zeros(3, 40), lib.mx_empty(3, 40, 4, device="cpu")
    for f, args in ((lib.mx_quantize, (x, c, s)), (lib.mx_dequantize, (c, s, x)), (lib.mx4_linear, (x, c, s, x)), (lib.mx4_matmul, (c, s, c, s, x)),
                    (lib.mx_grad_input, (x, c, s, x)), (lib.mx_grad_weight, (x, c, s, x))):
        with pytest.raises(lib.SgemmError):
            f(*args)
        for i in range(len(args)):
            with pytest.raises(lib.SgemmError):
                f(*args[:i], None, *args[i + 1:])


@pytest.mark.parametrize("rows,cols,bits,codes,scales", [(3, 40, 4, (3, 32), 16), (1, 1, 8, (1, 32), 16), (5, 544, 8, (5, 544), 32), (0, 64, 4, (0, 32), 16)])
def test_buffers(rows, cols, bits, codes, scales):
    c, s = lib.mx_empty(rows, cols, bits, device="cpu")
    assert tuple(c.shape) == codes and c.dtype == (torch.uint8 if bits == 4 else torch.int8)
    assert tuple(s.shape) == (rows, (cols + 31) // 32) and s.dtype == torch.uint8
    assert s.stride(0) == scales or rows <= 1


@pytest.mark.parametrize("bad", [(2, 2, 5), (-1, 2, 4), (2, -1, 8)])
def test_buffers_refused(bad):
    with pytest.raises(lib.SgemmError):
        lib.mx_empty(*bad, device="cpu")


# ---- the 64-bit forms themselves


@pytest.mark.parametrize("bits,most,half", [(4, 6, 0.25), (8, 127, 0.5)])
def test_rounding_is_to_the_nearest_of_all_codes(bits, most, half):
    g = torch.Generator().manual_seed(bits)
    x = torch.randn(40, 70, generator=g) * torch.exp2(torch.randint(-20, 20, (40, 1), generator=g).float())
    codes, scales = mo.quantize(x, bits)
    y = mo.values(torch.from_numpy(codes), torch.from_numpy(scales), 70)
    power = torch.from_numpy(2.0 ** (scales.astype(np.float64) - 127)).repeat_interleave(32, 1)[:, :70]
    grid = torch.from_numpy(np.concatenate([-mo.GRID4, mo.GRID4]) if bits == 4 else np.arange(-127.0, 128)) if bits else None
    # no code of the block's scale is nearer than the one taken
    best = (grid[None, None, :] * power[:, :, None] - x.double()[:, :, None]).abs().amin(2)
    assert torch.equal((y - x.double()).abs(), best)
    # and half the scale would not have held the block
    top = torch.nn.functional.pad(x.abs(), (0, 26)).reshape(40, 3, 32).amax(2).double()
    s = power[:, ::32]
    assert (top <= most * s).all() and (top > most * s / 2).all()


def test_rounding_of_ties_and_borders():
    # a block whose scale is 1: 6 is there, and every half-way point
    x = torch.tensor([[6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -5.0, 0.0, -0.0, 4.9999, 5.0001, 0.2501]])
    codes, scales = mo.quantize(x, 4)
    assert scales.tolist() == [[127]]
    got = mo.values(torch.from_numpy(codes), torch.from_numpy(scales), 16)[0].tolist()
    assert got == [6, 0, 1, 1, 2, 2, 4, 4, -0.0, -1, -4, 0, -0.0, 4, 6, 0.5]
    assert codes[0, 6] & 15 == 8   # -0.0 keeps its sign
    x = torch.tensor([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5]])
    codes, scales = mo.quantize(x, 8)
    assert scales.tolist() == [[127]] and codes[0, :6].tolist() == [127, 0, 2, 2, 0, -2]


def test_rounding_at_the_ends_of_the_range():
    tiny, huge = 2.0 ** -149, 3.4028234663852886e38
    for bits, last in ((4, 252), (8, 248)):
        codes, scales = mo.quantize(torch.tensor([[tiny] * 32 + [huge] * 32 + [float("inf")] + [1.0] * 31 + [0.0] * 32]), bits)
        assert scales.tolist() == [[0, last, 255, 0]]
        y = mo.values(torch.from_numpy(codes), torch.from_numpy(scales), 128)[0]
        assert (y[:32] == 0).all() and y[64:96].isnan().all() and (y[96:] == 0).all()
        assert torch.isfinite(y[32:64].float()).all() and (y[32:64] > 0.7 * huge).all()


def test_gradients_against_differences():
    """loss = sum(C * (X W^T)) of coded X and W: its gradients by the values of X and of W, against differences."""
    g = torch.Generator().manual_seed(3)
    T, K, N = 3, 40, 5
    X = mo.values(*(torch.from_numpy(v) for v in mo.quantize(torch.randn(T, K, generator=g), 8)), K)
    W = mo.values(*(torch.from_numpy(v) for v in mo.quantize(torch.randn(N, K, generator=g), 4)), K)
    C = torch.randn(T, N, generator=g).double()
    dX, _ = mo.product(C, W, torch.float32)
    dW, _ = mo.product(C.t(), X, torch.float32)
    h = 2.0 ** -10
    for M, D in ((X, dX), (W, dW)):
        for i in range(M.shape[0]):
            for j in range(0, K, 7):
                keep = M[i, j].item()
                M[i, j] = keep + h
                up = (C * (X @ W.t())).sum()
                M[i, j] = keep - h
                down = (C * (X @ W.t())).sum()
                M[i, j] = keep
                # linear in each value: the difference is the gradient but for 64-bit roundings
                assert abs((up - down) / (2 * h) - D[i, j]) <= 1e-9
