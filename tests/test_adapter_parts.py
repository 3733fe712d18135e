"""H and U in bfloat16 calls: the projection and the gradients take them as
two bfloat16 parts, so what they lose is 2^-16 of each value, not the 2^-8 of
one bfloat16.  Bounds as in adapter_oracle with that in the place of the
bfloat16 roundoff; elements whose terms cancel tell the two apart, which a
test on the CPU shows with the arithmetic of either kind."""
import pytest
import torch

import adapter_oracle as ao
import dense_fp32_gemm_06_gb300 as lib
import test_lora_gpu as lora
from dense_fp32_gemm_06_gb300 import adapters

BF16 = torch.bfloat16
PARTS = 2.0 ** -16   # 2^-8 of the rest that the high part (within 2^-8) leaves


def outer_bound(P, X, up, extra=0.0):
    """|sum of products| of P held in parts with X, `up` additions in a chain; plus the rounding to bfloat16 of a value of that error."""
    return (ao.gamma(ao.chain(up)) + PARTS + extra) * (P.abs() @ X.abs())


def forward(X, W, A, B, ids, scale=None):
    """(Y, its bound, H, its bound) in float64 on the CPU."""
    _, _, H, HB = ao.lora_forward(X, W, A, B, ids, scale, BF16)
    X, W, A, B, ids, s = ao.lora_parts(X, W, A, B, ids, scale)
    K, R = X.shape[1], A.shape[1]
    Y, bound = X @ W, ao.product_bound(K + R, BF16) * (X.abs() @ W.abs())
    for a in range(A.shape[0]):
        rows = torch.nonzero(ids == a)[:, 0]
        Y[rows] += H[rows] @ B[a]
        bound[rows] += (ao.gamma(R + 8) + PARTS + ao.product_bound(R, BF16)) * (H[rows].abs() @ B[a].abs()) + HB[rows] @ B[a].abs() * 1.01
    return Y, bound + ao.OUT_U[BF16] * (Y.abs() + bound) + 1e-30, H, HB


def backward(dY, X, W, A, B, ids, H, scale=None):
    """{name: (gradient, bound)}."""
    dX, bx, U, UB = forward(dY, W.t(), B, A, ids, scale)
    dY, H = dY.detach().cpu().double(), H.detach().cpu().double()
    X, W, A, B, ids, s = ao.lora_parts(X, W, A, B, ids, scale)
    out = {"dX": (dX, bx)}
    for name, P, PB, V, like in (("dA", U, UB, X, A), ("dB", H, torch.zeros_like(H), dY, B)):
        G, b = torch.zeros_like(like), torch.zeros_like(like)
        for a in range(A.shape[0]):
            rows = torch.nonzero(ids == a)[:, 0]
            G[a] = P[rows].t() @ V[rows]
            b[a] = outer_bound(P[rows].t(), V[rows], rows.numel()) + PB[rows].t() @ V[rows].abs() * 1.01
        out[name] = (G, b + ao.OUT_U[BF16] * (G.abs() + b) + 1e-30)
    return out


def check(T, K, N, L, R, mix, w_t=False, pad=0, off=0, seed=0, std_w=1.0):
    c = lora.make(T, K, N, L, R, BF16, mix, w_t, pad, off, seed)
    c["W"].mul_(std_w)
    o = lora.outputs(c, BF16, pad, off)
    lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], o["Y"], c["scale"], H=o["H"])
    Y, yb, _, _ = forward(c["X"], c["W"], c["A"], c["B"], c["ids"], c["scale"])
    ao.close(o["Y"], Y, yb, "Y")
    lib.lora_backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], o["H"], o["dX"], o["dA"], o["dB"], c["scale"])
    for name, (want, bound) in backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], o["H"], c["scale"]).items():
        ao.close(o[name], want, bound, name)
    assert adapters.device_status(clear=True) == 0
    return c, o


@pytest.mark.gpu
@pytest.mark.parametrize("std_w", [0.0, 1.0], ids=["adapters alone", "beside a projection"])
@pytest.mark.parametrize("T", [1, 40, 150, 700, 2100])   # single rows, few, the tensor-core shrink, rows cut into parts
@pytest.mark.parametrize("R", [8, 16, 32, 40, 64, 100])
def test_products_of_h(R, T, std_w):
    check(T, 128, 264, 2, R, "runs" if T > 1 else "one", seed=R + T, std_w=std_w)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N,L,R,mix", [(64, 1024, 256, 64, 16, "rows"), (64, 1024, 128, 9, 100, "rows"), (300, 1100, 136, 40, 33, "rows"),
                                           (17, 257, 131, 5, 7, "rows"), (260, 200, 264, 3, 256, "runs")])
def test_products_of_h_of_many_adapters(T, K, N, L, R, mix):
    check(T, K, N, L, R, mix, True, seed=7, std_w=0.1)


@pytest.mark.gpu
@pytest.mark.parametrize("R", [8, 32, 40, 64, 100])
@pytest.mark.parametrize("T", [96, 160, 1800])
def test_what_the_high_parts_leave(T, R):
    """Rows in pairs: dY and X change sign, H and U by a step far below their bfloat16 spacing.  The gradients are what the low parts give."""
    K, N, L = 136, 200, 2
    c = lora.make(T, K, N, L, R, BF16, "one", seed=R)
    c["ids"][: T // 2] = 0
    c["X"][1::2] = -c["X"][0::2]
    c["dY"][1::2] = -c["dY"][0::2]
    H = torch.randn(T, R, device="cuda", generator=torch.Generator(device="cuda").manual_seed(T)) + 4
    H[1::2] = H[0::2] * (1 + 2.0 ** -10)
    dA, dB = torch.empty_like(c["A"]), torch.empty_like(c["B"])
    lib.lora_backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], H, None, dA, dB, c["scale"])
    for name, got in (("dA", dA), ("dB", dB)):
        ao.close(got, *backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], H, c["scale"])[name], name)


def split(v, parts):
    hi = v.float().to(BF16).double()
    return hi if parts == 1 else hi + (v.float() - hi.float()).to(BF16).double()


@pytest.mark.parametrize("R", [8, 16, 100])
def test_the_bound_tells_one_part_from_two(R):
    g = torch.Generator().manual_seed(R)
    T, K, N, L = 40, 128, 264, 2
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(BF16)  # noqa: E731
    X, W, A, B, dY = rnd(T, K), rnd(K, N, std=K ** -0.5), rnd(L, R, K, std=K ** -0.5), rnd(L, R, N, std=0.1), rnd(T, N)
    ids = torch.arange(T) % 2
    Y, yb, H, _ = forward(X, W, A, B, ids)
    want, gb = backward(dY, X, W, A, B, ids, H.float())["dB"]
    for parts in (1, 2):
        h = split(H, parts)
        got = X.double() @ W.double() + (h[:, None, :] @ B.double()[ids])[:, 0]
        dB = torch.stack([h[ids == a].t() @ dY.double()[ids == a] for a in range(L)])
        if parts == 2:
            ao.close(got.to(BF16), Y, yb, "Y")
            ao.close(dB.to(BF16), want, gb, "dB")
        else:
            for bad, ref, bound in ((got, Y, yb), (dB, want, gb)):
                with pytest.raises(AssertionError):
                    ao.close(bad.to(BF16), ref, bound)
