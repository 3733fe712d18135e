"""What makes the FP32 results of the microscaled products FP32: every bit of a
gradient enters, and the tensor core's truncating accumulators are taken out
after 128 (gradients) or 1024 (products of 4-bit matrices) values.  The inputs
are such that the results are known to the last bit, or to what one
accumulator may lose, at each plan (split contractions, CTA pairs, one CTA)."""
import pytest
import torch

import dense_fp32_gemm_06_gb300 as lib
from dense_fp32_gemm_06_gb300 import microscale

pytestmark = pytest.mark.gpu

F32 = torch.float32
BITS = pytest.mark.parametrize("bits", [4, 8])
# (T, K, N): split contractions, CTA pairs and a CTA a tile (`kind`)
PLANS = [(200, 300, 1000), (100, 70, 65), (2048, 2048, 2048), (700, 4000, 500), (4100, 130, 600), (60, 6000, 9000)]


@pytest.fixture(autouse=True)
def _waits():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    assert microscale.device_status(clear=True) == 0


def kind(call, T, K, N, bits=4):
    p = microscale.plan(call, T, K, N, F32, bits)
    return "pair" if p["pair"] else "split" if p["split"] > 1 else "one"


@BITS
def test_the_plans_differ(bits):
    for call in ("grad_input", "grad_weight"):
        assert {kind(call, *p, bits) for p in PLANS} >= {"pair", "split"}


def powers(rows, cols, bits, seed):
    """A coded matrix of values +-2^e, and these values."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes, scales = lib.mx_empty(rows, cols, bits)
    scales.copy_(torch.randint(117, 138, scales.shape, device="cuda", generator=g))
    if bits == 4:
        table = torch.tensor([1, 2, 4, 6, 9, 10, 12, 14], device="cuda")       # 0.5, 1, 2, 4 and below zero
        value = torch.tensor([0.5, 1, 2, 4, -0.5, -1, -2, -4], device="cuda")
    else:
        value = torch.tensor([1, 2, 4, 8, 16, 32, 64, -1, -2, -64], device="cuda").float()
        table = value.long()
    pick = torch.randint(len(table), (rows, scales.shape[1] * 32), device="cuda", generator=g)
    if bits == 4:
        c = table[pick].view(rows, -1, 2)
        codes.copy_(c[:, :, 0] | c[:, :, 1] << 4)
    else:
        codes.copy_(table[pick])
    v = value[pick] * torch.exp2(scales.float() - 127).repeat_interleave(32, 1)
    return (codes, scales), v[:, :cols]


def wide(n, seed):
    """Values of all 24 bits, of 2^-20 to 2^20."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    m = torch.randint(2 ** 23, 2 ** 24, (n,), device="cuda", generator=g).float()
    return m * torch.exp2(torch.randint(-43, -3, (n,), device="cuda", generator=g).float()) * (1 - 2 * torch.randint(2, (n,), device="cuda", generator=g))


@BITS
@pytest.mark.parametrize("T,K,N", PLANS)
def test_input_gradients_of_one_term_are_exact(T, K, N, bits):
    """A value of dY a row, times powers of two.  Its bfloat16 parts' sums are leading bits of it: nothing is cut off."""
    m, W = powers(N, K, bits, seed=1)
    at = torch.arange(T, device="cuda") * 37 % N
    dY = torch.zeros(T, N, device="cuda")
    dY[torch.arange(T), at] = wide(T, seed=2)
    dX = torch.empty(T, K, device="cuda")
    lib.mx_grad_input(dY, *m, dX)
    assert torch.equal(dX, dY.sum(1, keepdim=True) * W[at])


@BITS
@pytest.mark.parametrize("T,K,N", PLANS)
def test_weight_gradients_of_one_term_are_exact(T, K, N, bits):
    m, X = powers(T, K, bits, seed=3)
    at = torch.arange(N, device="cuda") * 37 % T
    dY = torch.zeros(T, N, device="cuda")
    dY[at, torch.arange(N)] = wide(N, seed=4)
    dW = torch.empty(N, K, device="cuda")
    lib.mx_grad_weight(dY, *m, dW)
    want = dY.sum(0)[:, None] * X[at]
    assert torch.equal(dW, want)
    lib.mx_grad_weight(dY, *m, dW, accumulate=True)
    assert torch.equal(dW, 2 * want)


# 2^24 and then terms of which each MMA's add up to 1, half a unit in 2^24's last place.  An accumulator that had 2^24 in it
# from first to last would lose them all: 1 an MMA.  Taken out after `taken` values, it loses those beside 2^24 alone; the others'
# sums and their FP32 sum are even whole numbers, exact.  (One more: where the first accumulator's own sum is odd, it is
# rounded by 1.)


@BITS
@pytest.mark.parametrize("T,K", [(70, 200), (300, 2048), (2048, 2048)])
def test_sums_of_input_gradients_are_taken_out(T, K, bits):
    N = 16384
    c, s = lib.mx_quantize(torch.ones(1, K, device="cuda"), *lib.mx_empty(1, K, bits))
    codes, scales = lib.mx_empty(N, K, bits)
    codes.copy_(c.expand(N, -1)), scales.copy_(s.expand(N, -1))
    dY = torch.full((T, N), 1 / 16, device="cuda")
    dY[:, 0] = 2.0 ** 24
    dX = torch.empty(T, K, device="cuda")
    lib.mx_grad_input(dY, codes, scales, dX)
    assert N / microscale.plan("grad_input", T, K, N, F32, bits)["split"] / 16 > 100
    assert (dX.double() - (2.0 ** 24 + (N - 1) / 16)).abs().max() <= 127 / 16 + 1


@BITS
@pytest.mark.parametrize("N,K", [(70, 200), (300, 2048), (2048, 2048)])
def test_sums_of_weight_gradients_are_taken_out(N, K, bits):
    T = 16384
    c, s = lib.mx_quantize(torch.ones(1, K, device="cuda"), *lib.mx_empty(1, K, bits))
    codes, scales = lib.mx_empty(T, K, bits)
    codes.copy_(c.expand(T, -1)), scales.copy_(s.expand(T, -1))
    dY = torch.full((T, N), 1 / 16, device="cuda")
    dY[0] = 2.0 ** 24
    dW = torch.empty(N, K, device="cuda")
    lib.mx_grad_weight(dY, codes, scales, dW)
    assert T / microscale.plan("grad_weight", T, K, N, F32, bits)["split"] / 16 > 100
    assert (dW.double() - (2.0 ** 24 + (T - 1) / 16)).abs().max() <= 127 / 16 + 1


@pytest.mark.parametrize("T,N", [(3, 200), (16, 9000), (40, 200), (70, 9000), (300, 2900), (2600, 2900)])
def test_sums_of_linear_are_taken_out(T, N):
    K = 32768
    x = torch.full((T, K), 1 / 64, device="cuda")
    x[:, :32] = 0
    x[:, 0] = 2.0 ** 24
    w = lib.mx_quantize(torch.ones(N, K, device="cuda"), *lib.mx_empty(N, K, 4))
    assert K / microscale.plan("linear", T, K, N, F32)["split"] / 64 > 60
    want = 2.0 ** 24 + (K - 32) / 64
    Y = torch.empty(T, N, device="cuda")
    lib.mx4_linear(x, *w, Y)
    assert (Y.double() - want).abs().max() <= (1024 - 32) / 64 + 1
    lib.mx4_matmul(*lib.mx_quantize(x, *lib.mx_empty(T, K, 4)), *w, Y.zero_())
    assert (Y.double() - want).abs().max() <= (1024 - 32) / 64 + 1
