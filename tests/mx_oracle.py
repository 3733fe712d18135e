"""Plain 64-bit forms of the microscaled operators, with the bounds that the
kernels' arithmetic has to meet.  The rounding is written as a search over the
grid of codes, apart from the library's formulas."""
import numpy as np
import torch

GRID4 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
OUT_U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def blocks(cols):
    return (cols + 31) // 32


def quantize(X, bits):
    """(codes as the library stores them, scale bytes) of a matrix, numpy uint8 / int8."""
    x = X.detach().cpu().to(torch.float64).numpy()
    rows, cols = x.shape
    nb = blocks(cols)
    x = np.pad(x, ((0, 0), (0, nb * 32 - cols))).reshape(rows, nb, 32)
    top = np.abs(x).max(axis=2) if x.size else np.zeros((rows, nb))
    bad = ~np.isfinite(top)
    most, last = (6.0, 125) if bits == 4 else (127.0, 121)
    # the least of all exponents that holds the block
    e = np.full((rows, nb), last)
    for k in range(last, -128, -1):
        e = np.where(np.where(bad, 0.0, top) <= most * 2.0 ** k, k, e)
    y = np.where(bad[:, :, None], 0.0, x) / 2.0 ** e[:, :, None].astype(np.float64)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    if bits == 8:
        grid = np.arange(0, 128, dtype=np.float64)
    else:
        grid = GRID4
    a = np.minimum(np.abs(y), grid[-1])
    up = np.searchsorted(grid, a).clip(0, len(grid) - 1)
    down = np.maximum(up - 1, 0)
    to_up, to_down = grid[up] - a, a - grid[down]
    code = np.where((to_up < to_down) | ((to_up == to_down) & (up % 2 == 0)), up, down)
    if bits == 8:
        return np.where(np.signbit(y), -code, code).astype(np.int8).reshape(rows, nb * 32), scales
    code = code + 8 * (np.signbit(y) & ~bad[:, :, None])
    code = code.reshape(rows, nb * 16, 2)
    return (code[:, :, 0] + 16 * code[:, :, 1]).astype(np.uint8), scales


def values(codes, scales, cols):
    """What codes and scales stand for, float64 on the CPU."""
    c, s = codes.detach().cpu().numpy(), scales.detach().cpu().numpy()
    rows = c.shape[0]
    if c.dtype == np.int8:
        q = c.astype(np.float64)
    else:
        pair = np.stack([c & 15, c >> 4], axis=2).reshape(rows, -1)
        q = np.where(pair & 8, -1.0, 1.0) * GRID4[pair & 7]
    power = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))
    return torch.from_numpy((q.reshape(rows, -1, 32) * power[:, :, None]).reshape(rows, -1)[:, :cols].copy())


def product(A, B, dtype, parts=1):
    """(A B, the bound of a kernel's distance from it): exact products; the
    tensor core rounds its FP32 sum towards zero once per 16 of the depth, at
    most 2^-22 of it, for each of an FP32 operand's three parts; joined sums
    and the output's rounding come on top."""
    A, B = A.double().cpu(), B.double().cpu()
    Y, E = A @ B, A.abs() @ B.abs()
    bound = (parts * A.shape[1] / 16 + 12) * 2.0 ** -22 * E
    return Y, bound + OUT_U[dtype] * (Y.abs() + bound) + 2.0 ** -126


def close(got, want, bound, what):
    got = got.detach().double().cpu()
    assert got.shape == want.shape, what
    nan = want.isnan()
    assert torch.equal(got.isnan(), nan), f"{what}: not a number in other places"
    inf = want.isinf()
    assert torch.equal(got[inf], want[inf]), what
    d = ((got - want).abs() / bound)[~nan & ~inf]
    assert d.numel() == 0 or d.max() <= 1, f"{what}: {d.max():.3g} of the bound"
