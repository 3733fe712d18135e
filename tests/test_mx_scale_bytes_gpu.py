"""Codes and scales made elsewhere: every scale byte, those above the ones
that mx_quantize writes among them, beside all codes whose values have
magnitudes below 2^128, and what becomes of the others."""
import pytest
import torch

import dense_fp32_gemm_06_gb300 as lib
import mx_oracle as mo
from dense_fp32_gemm_06_gb300 import microscale

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
BITS = pytest.mark.parametrize("bits", [4, 8])


@pytest.fixture(autouse=True)
def _waits():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    assert microscale.device_status(clear=True) == 0


def every_byte(cols, bits, seed=0, finite=True):
    """A row for each byte 0 .. 254, random codes; where `finite`, none of a magnitude of 2^128 or more (those are 0)."""
    g = torch.Generator().manual_seed(seed)
    nb = mo.blocks(cols)
    scales = torch.arange(255, dtype=torch.uint8)[:, None].repeat(1, nb)
    codes = torch.randint(0, 256, (255, nb * bits * 4), generator=g).to(torch.uint8)
    if bits == 8:
        codes = codes.view(torch.int8)
    if finite:
        large = mo.values(codes, scales, nb * 32).abs() >= 2.0 ** 128
        if bits == 8:
            codes = torch.where(large, torch.zeros_like(codes), codes)
        else:
            pair = large.view(255, -1, 2)
            codes = codes & (torch.where(pair[:, :, 0], 0xF0, 0xFF) & torch.where(pair[:, :, 1], 0x0F, 0xFF)).to(torch.uint8)
    c, s = lib.mx_empty(255, cols, bits)
    c.copy_(codes)
    s.copy_(scales)
    return c, s


@TYPES
@BITS
@pytest.mark.parametrize("cols", [96, 1024])
def test_reading_every_byte(cols, bits, dtype):
    """The value rounded to the type: from 2^128 on an infinity."""
    c, s = every_byte(cols, bits, finite=False)
    Y = torch.empty(255, cols, device="cuda", dtype=dtype)
    lib.mx_dequantize(c, s, Y)
    assert torch.equal(Y.cpu(), mo.values(c, s, cols).float().to(dtype))


def of_16_bits(n, exponent, dtype, seed):
    """Values of 16 (bfloat16: 8) bits, of those powers of two."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    top = 2 ** 16 if dtype == F32 else 2 ** 8
    m = torch.randint(top // 2, top, (n,), device="cuda", generator=g).double() / (top // 2)
    return (m * torch.exp2(exponent.double())).to(dtype)


@TYPES
@BITS
@pytest.mark.parametrize("T,K", [(255, 160), (510, 4096)])
def test_gradients_beside_every_byte(T, K, bits, dtype):
    """One value of dY a sum, of 16 bits beside codes of 7: a bfloat16 part's products, and their sums, are exact in FP32."""
    N = 255
    m = every_byte(K, bits, seed=1)
    W = mo.values(*m, K).cuda()
    at = torch.arange(T, device="cuda") % N
    v = of_16_bits(T, (147 - at).clamp(max=120), dtype, seed=2)
    dY = torch.zeros(T, N, device="cuda", dtype=dtype)
    dY[torch.arange(T), at] = v
    dX = torch.empty(T, K, device="cuda", dtype=dtype)
    lib.mx_grad_input(dY, *m, dX)
    assert torch.equal(dX, (v.double()[:, None] * W[at]).float().to(dtype))
    dW = torch.empty(T, K, device="cuda", dtype=dtype)
    lib.mx_grad_weight(dY.t().contiguous(), *m, dW)   # (255 tokens, T features)
    assert torch.equal(dW, dX)


@TYPES
@BITS
def test_gradients_beside_values_past_the_range(bits, dtype):
    """Such a value counts as an infinity: the sums that it is in are not finite, the others are as without it."""
    T, N, K = 70, 200, 300
    g = torch.Generator(device="cuda").manual_seed(1)
    dY = torch.randn(T, N, device="cuda", generator=g).to(dtype)
    c, s = lib.mx_quantize(torch.randn(N, K, device="cuda", generator=g).to(dtype), *lib.mx_empty(N, K, bits))
    outs = []
    for large in (False, True):
        if large:
            c[17, 40 * bits // 8] = 0x77 if bits == 4 else 127   # column 40, in 4 bits also 41
            keep = c[17, 32 * bits // 8:64 * bits // 8].clone()
            s[17, 1] = 254
            c[17, 32 * bits // 8:64 * bits // 8] = 0             # (the block's others stay in range)
            c[17, 40 * bits // 8] = keep[8 * bits // 8]
        dX = torch.empty(T, K, device="cuda", dtype=dtype)
        lib.mx_grad_input(dY, c, s, dX)
        outs.append(dX)
    cols = [40, 41] if bits == 4 else [40]
    rest = [k for k in range(K) if not 32 <= k < 64]
    assert not outs[1][:, cols].isfinite().any()
    assert torch.equal(outs[0][:, rest], outs[1][:, rest])
    assert outs[1][:, [k for k in range(32, 64) if k not in cols]].isfinite().all()


@TYPES
@pytest.mark.parametrize("T,N", [(3, 40), (40, 255), (255, 510)])
def test_products_of_every_byte(T, N, dtype):
    """A block a row of X beside W's of any byte; all other blocks of X are zeros, of any byte too (0 times 2^254 is 0)."""
    K = 4096
    g = torch.Generator().manual_seed(T)
    xc, xs = lib.mx_empty(T, K, 4)
    wc, ws = lib.mx_empty(N, K, 4)
    byte = torch.randint(0, 255, (T,), generator=g)
    at = torch.randint(0, K // 32, (T,), generator=g)
    xs.copy_(torch.randint(0, 255, xs.shape, generator=g))
    xc.zero_()
    xs[torch.arange(T), at.cuda()] = byte.to(torch.uint8).cuda()
    blocks = xc.view(T, K // 32, 16)
    blocks[torch.arange(T), at.cuda()] = torch.randint(0, 256, (T, 16), generator=g).to(torch.uint8).cuda()
    # W's scales make each row's product with that row's block something in range: 2^-60 .. 2^60
    ws.copy_(torch.randint(0, 255, ws.shape, generator=g))
    for t in range(T):
        low, high = max(0, 194 - int(byte[t])), min(254, 314 - int(byte[t]))
        ws[:, at[t]] = torch.randint(low, high + 1, (N,), generator=g).to(torch.uint8).cuda() if (at[:t] != at[t]).all() else ws[:, at[t]]
    wc.copy_(torch.randint(0, 256, wc.shape, generator=g))
    want, bound = mo.product(mo.values(xc, xs, K), mo.values(wc, ws, K).t(), dtype)
    Y = torch.empty(T, N, device="cuda", dtype=dtype)
    lib.mx4_matmul(xc, xs, wc, ws, Y)
    most = torch.finfo(dtype).max
    fine = want.abs() < most / 4   # (rows that share a block may pass the range: infinities of their sign)
    assert fine.float().mean() > 0.5
    got = Y.double().cpu()
    assert ((got - want).abs() <= bound)[fine].all()
    past = want.abs() > 2 * most
    assert torch.equal(got[past], want[past].sign() * float("inf"))
