"""The microscaled operators against their 64-bit forms: codes and scales to
the bit, products within their bounds; one row to many, odd sizes, strides,
unaligned matrices, both types and numbers of bits, blocks that are not finite,
the ends of the range, what must not be written, streams and graphs."""
import pytest
import torch

import dense_fp32_gemm_06_gb300 as lib
import mx_oracle as mo
from dense_fp32_gemm_06_gb300 import _native, microscale

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
BITS = pytest.mark.parametrize("bits", [4, 8])
GUARD = 0xA5


@pytest.fixture(autouse=True)
def _waits():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    assert microscale.device_status(clear=True) == 0


def normal(*shape, dtype=F32, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)


class Framed:
    """A rows x cols matrix of that pitch, `off` elements behind an aligned address, among elements that must stay."""

    def __init__(self, rows, cols, dtype, pad=0, off=0, pitch=None):
        self.pitch = cols + pad if pitch is None else pitch
        self.at, self.n = 64 + off, max(rows, 1) * self.pitch
        self.buf = torch.full((self.at + self.n + 64,), GUARD if dtype in (torch.uint8,) else 77, device="cuda", dtype=dtype)
        self.view = self.buf.as_strided((rows, cols), (self.pitch, 1), self.at)
        self.before = self.buf.clone()

    def check(self):
        now = self.buf.clone()
        now.as_strided(self.view.shape, self.view.stride(), self.at).copy_(self.before.as_strided(self.view.shape, self.view.stride(), self.at))
        assert torch.equal(now, self.before), "written outside the matrix"


def framed(x, pad=0, off=0):
    f = Framed(*x.shape, x.dtype, pad, off)
    f.view.copy_(x)
    f.before = f.buf.clone()
    return f


def coded_buffers(rows, cols, bits, pad=0):
    nb = mo.blocks(cols)
    codes = Framed(rows, nb * bits * 4, torch.uint8 if bits == 4 else torch.int8, pitch=nb * bits * 4 + 16 * pad)
    scales = Framed(rows, nb, torch.uint8, pitch=(nb + 15) // 16 * 16 + 16 * pad)
    return codes, scales


def coded(x, bits, pad=0):
    """A matrix as the oracle codes it, in framed buffers."""
    c, s = (torch.from_numpy(v).cuda() for v in mo.quantize(x, bits))
    codes, scales = coded_buffers(*x.shape, bits, pad)
    codes.view.copy_(c)
    scales.view.copy_(s)
    codes.before, scales.before = codes.buf.clone(), scales.buf.clone()
    return codes.view, scales.view


def check_store(x, bits, pad=0, off=0, transposed=False):
    f = framed(x.t().contiguous() if transposed else x, pad, off)
    X = f.view.t() if transposed else f.view
    codes, scales = coded_buffers(*x.shape, bits, pad)
    lib.mx_quantize(X, codes.view, scales.view)
    want_c, want_s = mo.quantize(x, bits)
    assert torch.equal(scales.view.cpu(), torch.from_numpy(want_s))
    assert torch.equal(codes.view.cpu(), torch.from_numpy(want_c))
    codes.check()
    scales.check()
    Y = Framed(*x.shape, x.dtype, pad, off)
    lib.mx_dequantize(codes.view, scales.view, Y.view)
    want = mo.values(codes.view, scales.view, x.shape[1])
    got = Y.view.double().cpu()
    assert torch.equal(got.nan_to_num(nan=12345.0), want.nan_to_num(nan=12345.0))
    Y.check()


STORES = [(1, 1), (1, 31), (1, 32), (2, 33), (7, 255), (5, 257), (33, 1000), (64, 544), (129, 777), (1, 8200), (300, 2048)]


@TYPES
@BITS
@pytest.mark.parametrize("rows,cols", STORES)
def test_store(rows, cols, bits, dtype):
    check_store(normal(rows, cols, dtype=dtype, seed=rows + cols), bits)


@TYPES
@BITS
@pytest.mark.parametrize("rows,cols", STORES)
def test_store_of_a_transposed_view(rows, cols, bits, dtype):
    check_store(normal(rows, cols, dtype=dtype, seed=rows + cols), bits, transposed=True)


@TYPES
@BITS
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("pad,off", [(1, 0), (3, 1), (8, 8), (5, 3)])
def test_store_with_strides(pad, off, transposed, bits, dtype):
    check_store(normal(37, 300, dtype=dtype, seed=pad), bits, pad, off, transposed)


@TYPES
@BITS
@pytest.mark.parametrize("transposed", [False, True])
def test_store_of_every_magnitude(transposed, bits, dtype):
    """Blocks from subnormal to the largest magnitudes, with ties, zeros of both signs, and some not finite."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(64, 320, device="cuda", generator=g)
    x = x * torch.exp2(torch.randint(-150, 128, (64, 10), device="cuda", generator=g).float()).repeat_interleave(32, 1)
    top = torch.finfo(dtype).max
    x = x.nan_to_num(posinf=top, neginf=-top).clamp(-top, top).to(dtype)
    x[0, :32] = 0.0
    x[1, :32] = -0.0
    x[2, 5], x[3, 40], x[4, 70] = float("inf"), float("-inf"), float("nan")
    x[5, :32] = torch.finfo(dtype).max
    x[6, :32] = -torch.finfo(dtype).max
    x[7, :32] = torch.arange(32, device="cuda") * 0.25 - 2   # ties
    x[7, 0] = 6
    x[8, :32] = torch.arange(32, device="cuda") * 0.5 - 8
    x[8, 0] = 127
    x[9, :64] = 2.0 ** -126
    x[10, :64] = torch.finfo(dtype).tiny * torch.finfo(dtype).eps   # the least subnormal
    check_store(x, bits, transposed=transposed)


@TYPES
@BITS
def test_store_of_every_fraction(bits, dtype):
    """The largest magnitude's fraction decides the scale: every one of its upper eight bits, and the values next to them."""
    f = (torch.arange(256, device="cuda", dtype=torch.int32) << 15) + (127 << 23)
    x = torch.stack([f, f + 1, f - 1, f + (8 << 23)]).view(F32).reshape(-1, 1).to(dtype)
    x = torch.cat([x, normal(x.shape[0], 31, dtype=dtype)], 1)
    check_store(x, bits)


def check_linear(T, K, N, dtype, pad=0, off=0, seed=0, x=None, w=None, std=1.0):
    X = framed(normal(T, K, dtype=dtype, seed=seed) if x is None else x, pad, off)
    wc, ws = coded(normal(N, K, dtype=dtype, seed=seed + 1, std=std) if w is None else w, 4, pad)
    xc, xs = coded(X.view, 4, pad)
    want, bound = mo.product(mo.values(xc, xs, K), mo.values(wc, ws, K).t(), dtype)
    for call in (lambda y: lib.mx4_linear(X.view, wc, ws, y), lambda y: lib.mx4_matmul(xc, xs, wc, ws, y)):
        Y = Framed(T, N, dtype, pad, off)
        assert call(Y.view) is Y.view
        mo.close(Y.view, want, bound, f"Y of {T} x {K} x {N}")
        Y.check()


PRODUCTS = [(1, 1, 1), (1, 32, 16), (1, 4096, 256), (2, 33, 5), (3, 64, 130), (5, 100, 128), (8, 512, 257), (16, 545, 300), (17, 257, 131), (33, 1000, 100),
            (64, 2048, 512), (65, 1024, 129), (100, 96, 1), (128, 128, 128), (129, 777, 300), (200, 8192, 150), (257, 1000, 1500), (300, 300, 260),
            (520, 512, 640), (1, 8, 5000), (1000, 777, 1500)]


@TYPES
@pytest.mark.parametrize("T,K,N", PRODUCTS)
def test_linear(T, K, N, dtype):
    check_linear(T, K, N, dtype, seed=T + K)


@TYPES
@pytest.mark.parametrize("T,K,N,pad,off", [(1, 100, 70, 1, 1), (40, 256, 200, 8, 0), (130, 520, 260, 3, 5), (300, 513, 300, 5, 1)])
def test_linear_with_strides(T, K, N, pad, off, dtype):
    check_linear(T, K, N, dtype, pad, off)


@TYPES
@pytest.mark.parametrize("T", [3, 150])
def test_linear_of_blocks_that_are_not_finite(T, dtype):
    """A row of X with a NaN or an infinity in some block is NaN, the others are as they were; so are features of W."""
    K, N = 300, 140
    x, w = normal(T, K, dtype=dtype, seed=1), normal(N, K, dtype=dtype, seed=2)
    x[1, 70], x[2, 299], w[3, 0], w[N - 1, 290] = float("nan"), float("inf"), float("-inf"), float("nan")
    check_linear(T, K, N, dtype, x=x, w=w)


@TYPES
def test_linear_of_small_and_large_magnitudes(dtype):
    K, N, T = 200, 64, 20
    for sx, sw in ((2.0 ** -60, 2.0 ** -40), (2.0 ** 60, 2.0 ** 50), (2.0 ** 100, 2.0 ** -110), (0.0, 1.0)):
        check_linear(T, K, N, dtype, x=normal(T, K, dtype=dtype) * sx, w=normal(N, K, dtype=dtype, seed=1) * sw)


def check_grads(T, K, N, bits, dtype, pad=0, off=0, seed=0, dy=None, m=None):
    dY = framed(normal(T, N, dtype=dtype, seed=seed) if dy is None else dy, pad, off)
    parts = 3 if dtype == F32 else 1
    wc, ws = coded(normal(N, K, dtype=dtype, seed=seed + 1) if m is None else m, bits, pad)
    want, bound = mo.product(dY.view, mo.values(wc, ws, K), dtype, parts)
    dX = Framed(T, K, dtype, pad, off)
    assert lib.mx_grad_input(dY.view, wc, ws, dX.view) is dX.view
    mo.close(dX.view, want, bound, f"dX of {T} x {K} x {N}")
    dX.check()
    xc, xs = coded(normal(T, K, dtype=dtype, seed=seed + 2), bits, pad)
    want, bound = mo.product(dY.view.t(), mo.values(xc, xs, K), dtype, parts)
    dW = Framed(N, K, dtype, pad, off)
    assert lib.mx_grad_weight(dY.view, xc, xs, dW.view) is dW.view
    mo.close(dW.view, want, bound, f"dW of {T} x {K} x {N}")
    dW.check()
    # added to what is there: one more FP32 addition and the output's rounding
    first = dW.view.clone()
    lib.mx_grad_weight(dY.view, xc, xs, dW.view, accumulate=True)
    twice = first.double().cpu() + want
    mo.close(dW.view, twice, bound + (2.0 ** -24 + mo.OUT_U[dtype]) * (twice.abs() + bound), "dW added")
    dW.check()


@TYPES
@BITS
@pytest.mark.parametrize("T,K,N", [p for p in PRODUCTS if p != (1000, 777, 1500)] + [(4096, 64, 96), (300, 2100, 40)])
def test_gradients(T, K, N, bits, dtype):
    check_grads(T, K, N, bits, dtype, seed=T + N)


@TYPES
@BITS
@pytest.mark.parametrize("T,K,N,pad,off", [(1, 100, 70, 1, 1), (40, 256, 200, 8, 0), (130, 520, 260, 3, 5), (300, 513, 300, 5, 1)])
def test_gradients_with_strides(T, K, N, pad, off, bits, dtype):
    check_grads(T, K, N, bits, dtype, pad, off)


@TYPES
@BITS
def test_gradients_of_blocks_that_are_not_finite(bits, dtype):
    T, K, N = 70, 200, 90
    m = normal(N, K, dtype=dtype, seed=2)
    m[3, 40] = float("nan")
    dy = normal(T, N, dtype=dtype)
    dy[5, 7], dy[6, 8] = float("inf"), float("nan")
    dY = dy
    wc, ws = coded(m, bits)
    want, bound = mo.product(dY, mo.values(wc, ws, K), dtype, 3)
    dX = torch.empty(T, K, device="cuda", dtype=dtype)
    lib.mx_grad_input(dY, wc, ws, dX)
    mo.close(dX, want, bound, "dX")


@TYPES
def test_linear_past_the_range(dtype):
    """Sums above 2^128 are infinities of their sign, sums below 2^-126 are within it of 0."""
    T, K, N = 20, 96, 40
    one = torch.ones(T, K, device="cuda", dtype=dtype)
    w = torch.where(torch.arange(N, device="cuda")[:, None] % 2 == 0, 1.0, -1.0).expand(N, K).to(dtype)
    Y = torch.empty(T, N, device="cuda", dtype=dtype)
    lib.mx4_linear(one * 2.0 ** 70, *lib.mx_quantize(w * 2.0 ** 70, *lib.mx_empty(N, K, 4)), Y)
    assert torch.equal(Y.float(), w[:, :1].t().float().expand(T, N) * float("inf"))
    lib.mx4_linear(one * 2.0 ** -80, *lib.mx_quantize(w * 2.0 ** -80, *lib.mx_empty(N, K, 4)), Y)
    assert (Y.float().abs() <= 2.0 ** -126).all()


# several tiles for each cluster, last ones ragged: what the plan says, and the values
@TYPES
@pytest.mark.parametrize("T,K,N", [(2600, 520, 2900), (8200, 300, 200), (70, 8000, 1000), (16, 4100, 9000), (13, 200, 90000), (5, 700, 60000)])
def test_linear_of_many_tiles(T, K, N, dtype):
    p = microscale.plan("linear", T, K, N, dtype)
    if T == 2600:
        assert p["tiles"] >= 2 and p["pair"]
    assert T != 70 or p["split"] > 1
    check_linear(T, K, N, dtype, pad=3, seed=T)


@TYPES
@BITS
@pytest.mark.parametrize("T,K,N", [(2500, 3800, 1500), (8200, 300, 700), (1500, 3800, 2500)])
def test_gradients_of_many_tiles(T, K, N, bits, dtype):
    p = [microscale.plan(call, T, K, N, dtype, bits) for call in ("grad_input", "grad_weight")]
    if T == 2500:
        assert p[0]["pair"] and p[0]["tiles"] >= 2
    elif T == 1500:
        assert p[1]["pair"] and p[1]["tiles"] >= 2
    else:
        assert p[1]["split"] > 1 or p[1]["pair"]
    check_grads(T, K, N, bits, dtype, pad=8, seed=T)


@BITS
@pytest.mark.parametrize("T,K,N", [(190, 4000, 500), (250, 2601, 700), (256, 3000, 63), (129, 4864, 130)])
def test_float32_gradients_of_a_few_rows_in_pairs(T, K, N, bits):
    """Tiles of 64 rows by 256 columns, the last ones ragged both ways."""
    if N >= 500:
        p = microscale.plan("grad_input", T, K, N, torch.float32, bits)
        assert p["pair"] and p["rows"] == 64
    check_grads(T, K, N, bits, torch.float32, pad=3, seed=N)


@TYPES
@BITS
def test_gradients_of_extreme_scales(bits, dtype):
    """Scales far from 1, and values of dY of every size: FP32 ones keep all of their 24 bits."""
    for s_dy, s_m in ((2.0 ** 90, 2.0 ** -80), (2.0 ** -70, 2.0 ** 60), (2.0 ** 20, 2.0 ** 100), (2.0 ** -20, 2.0 ** -100),
                       (2.0 ** 60, 2.0 ** -124), (2.0 ** -60, 2.0 ** 123)):
        check_grads(33, 100, 65, bits, dtype, dy=normal(33, 65, dtype=dtype) * s_dy, m=normal(65, 100, dtype=dtype, seed=4) * s_m)


def test_float32_gradients_keep_their_bits():
    """One value of dY a row: dX is that value times the codes, to the last bit."""
    T = N = 64
    dy = torch.zeros(T, N, device="cuda")
    dy[torch.arange(T), torch.arange(N)] = normal(T) * torch.exp2(torch.arange(T, device="cuda") - 32.0)
    for bits in (4, 8):
        wc, ws = coded(torch.ones(N, 32, device="cuda"), bits)   # codes that stand for 1
        dX = torch.empty(T, 32, device="cuda")
        lib.mx_grad_input(dy, wc, ws, dX)
        assert torch.equal(dX, dy.sum(1, keepdim=True).expand(T, 32))


def far(x, pitch):
    """x with rows that far apart: the last ones start past 2^32 bytes."""
    v = torch.empty((x.shape[0] - 1) * pitch + x.shape[1], device="cuda", dtype=x.dtype).as_strided(x.shape, (pitch, 1))
    v.copy_(x)
    return v


@TYPES
@BITS
def test_offsets_past_32_bits(bits, dtype):
    rows, K, N = 4, 100, 70
    real, byte = 2 ** 30 + (8 if dtype == BF16 else 4), 2 ** 31 - 16
    x = normal(rows, K, dtype=dtype)
    c, s = (far(v, byte) for v in lib.mx_empty(rows, K, bits))
    lib.mx_quantize(far(x, real), c, s)
    want_c, want_s = mo.quantize(x, bits)
    assert torch.equal(c.cpu(), torch.from_numpy(want_c)) and torch.equal(s.cpu(), torch.from_numpy(want_s))
    y = far(torch.zeros_like(x), real)
    lib.mx_dequantize(c, s, y)
    assert torch.equal(y.double().cpu(), mo.values(c, s, K))
    del y
    dy, parts = normal(rows, N, dtype=dtype, seed=1), 3 if dtype == F32 else 1
    dW = far(torch.zeros(N, K, device="cuda", dtype=dtype), 2 ** 26 + 8)   # (70 rows)
    lib.mx_grad_weight(far(dy, real), c, s, dW)
    mo.close(dW, *mo.product(dy.t(), mo.values(c, s, K), dtype, parts), "dW")
    del dW
    dX = far(torch.zeros_like(x), real)
    lib.mx_grad_input(far(normal(rows, rows, dtype=dtype, seed=2), real), c, s, dX)
    mo.close(dX, *mo.product(normal(rows, rows, dtype=dtype, seed=2), mo.values(c, s, K), dtype, parts), "dX")
    del dX
    if bits == 4:
        wc, ws = coded(normal(N, K, dtype=dtype, seed=3), 4)
        want, bound = mo.product(mo.values(c, s, K), mo.values(wc, ws, K).t(), dtype)
        Y = far(torch.zeros(rows, N, device="cuda", dtype=dtype), real)
        lib.mx4_matmul(c, s, wc, ws, Y)
        mo.close(Y, want, bound, "Y")
        lib.mx4_linear(far(x, real), wc, ws, Y.zero_())
        mo.close(Y, want, bound, "Y")
        Z = torch.zeros(N, rows, device="cuda", dtype=dtype)
        lib.mx4_matmul(wc, ws, c, s, Z)
        mo.close(Z, want.t(), bound.t(), "Y of far weights")


@BITS
def test_more_columns_than_2_to_28(bits):
    """A row's byte offsets pass 2^31 when counted in bits: the last columns against the form of those alone."""
    T, N, K, last = 2, 3, 2 ** 28 + 160, 4096 + 160
    x = torch.empty(N, K, device="cuda", dtype=BF16).normal_()
    c, s = lib.mx_quantize(x, *lib.mx_empty(N, K, bits))
    tail_c, tail_s = (torch.from_numpy(v) for v in mo.quantize(x[:, -last:], bits))
    assert torch.equal(c[:, -tail_c.shape[1]:].cpu(), tail_c) and torch.equal(s[:, -tail_s.shape[1]:].cpu(), tail_s)
    back = torch.empty_like(x)
    lib.mx_dequantize(c, s, back)
    assert torch.equal(back[:, -last:].double().cpu(), mo.values(tail_c, tail_s, last))
    del back, x
    dy, dX = normal(T, N, dtype=BF16), torch.empty(T, K, device="cuda", dtype=BF16)
    lib.mx_grad_input(dy, c, s, dX)
    mo.close(dX[:, -last:], *mo.product(dy, mo.values(tail_c, tail_s, last), BF16), "dX")
    dy, dW = normal(N, 5, dtype=BF16), torch.empty(5, K, device="cuda", dtype=BF16)
    lib.mx_grad_weight(dy, c, s, dW)
    mo.close(dW[:, -last:], *mo.product(dy.t(), mo.values(tail_c, tail_s, last), BF16), "dW")
    if bits == 4:
        Y, w = torch.empty(T, N, device="cuda", dtype=F32), torch.zeros(T, K, device="cuda", dtype=BF16)
        w[:, -last:] = normal(T, last, dtype=BF16, seed=4)
        want, bound = mo.product(mo.values(*(torch.from_numpy(v) for v in mo.quantize(w[:, -last:], 4)), last), mo.values(tail_c, tail_s, last).t(), F32)
        # (a sum over all of k, all but the last columns' terms zero: the accumulator is rounded once per promotion too)
        lib.mx4_linear(w.float(), c, s, Y)
        mo.close(Y, want, bound, "Y")


@TYPES
def test_nothing_to_contract(dtype):
    e = lambda *s: torch.empty(*s, device="cuda", dtype=dtype)  # noqa: E731
    ones = lambda *s: torch.ones(*s, device="cuda", dtype=dtype)  # noqa: E731
    c0, s0 = lib.mx_empty(5, 0, 4)
    assert (lib.mx4_linear(e(3, 0), c0, s0, ones(3, 5)) == 0).all()
    assert (lib.mx4_matmul(*lib.mx_empty(3, 0, 4), c0, s0, ones(3, 5)) == 0).all()
    c, s = lib.mx_empty(0, 40, 8)
    assert (lib.mx_grad_input(e(3, 0), c, s, ones(3, 40)) == 0).all()
    assert (lib.mx_grad_weight(e(0, 6), c, s, ones(6, 40)) == 0).all()
    assert (lib.mx_grad_weight(e(0, 6), c, s, ones(6, 40), accumulate=True) == 1).all()
    for rows, cols in ((0, 40), (3, 0), (0, 0)):
        c, s = lib.mx_empty(rows, cols, 8)
        lib.mx_quantize(e(rows, cols), c, s)
        lib.mx_dequantize(c, s, e(rows, cols))
    assert lib.mx4_linear(e(0, 40), *lib.mx_empty(5, 40, 4), e(0, 5)).shape == (0, 5)


@pytest.mark.parametrize("what", ["codes' type", "columns", "rows", "pitch", "start", "types", "dY"])
def test_refusals(what):
    X, Y = normal(4, 64), torch.empty(4, 6, device="cuda")
    c, s = lib.mx_empty(6, 64, 4)
    if what == "codes' type":
        c = lib.mx_empty(6, 64, 8)[0]
    elif what == "columns":
        X = normal(4, 65)
    elif what == "rows":
        Y = torch.empty(4, 7, device="cuda")
    elif what == "pitch":
        s = torch.zeros(6, 2, device="cuda", dtype=torch.uint8)
    elif what == "start":
        c = torch.zeros(6 * 32 + 8, device="cuda", dtype=torch.uint8)[8:].view(6, 32)
    elif what == "types":
        X = X.bfloat16()
    elif what == "dY":
        X, Y = X.half(), Y.half()
    with pytest.raises(lib.SgemmError):
        lib.mx4_linear(X, c, s, Y)


@TYPES
def test_streams_and_graphs(dtype):
    """On another stream, and captured and replayed on new inputs: the eager calls' bits."""
    T, K, N = 130, 300, 200

    def step(x, dy, out):
        lib.mx_quantize(x, *out["ck"])
        lib.mx4_linear(x, *out["w"], out["y"])
        lib.mx_grad_input(dy, *out["w"], out["dx"])
        lib.mx_grad_weight(dy, *out["ck"], out["dw"])

    def buffers():
        w = lib.mx_quantize(normal(N, K, dtype=dtype, seed=9), *lib.mx_empty(N, K, 4))
        e = lambda *s: torch.empty(*s, device="cuda", dtype=dtype)  # noqa: E731
        return dict(w=w, ck=lib.mx_empty(T, K, 8), y=e(T, N), dx=e(T, K), dw=e(N, K))

    x, dy = torch.empty(T, K, device="cuda", dtype=dtype), torch.empty(T, N, device="cuda", dtype=dtype)
    eager, other, graphed = buffers(), buffers(), buffers()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    step(x.fill_(0), dy.fill_(0), graphed)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(x, dy, graphed)
    for seed in (1, 2, 3):
        x.copy_(normal(T, K, dtype=dtype, seed=seed))
        dy.copy_(normal(T, N, dtype=dtype, seed=seed + 10))
        step(x, dy, eager)
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            step(x, dy, other)
        graph.replay()
        torch.cuda.synchronize()
        for k in ("y", "dx", "dw"):
            assert torch.equal(eager[k], other[k]) and torch.equal(eager[k], graphed[k]), k
        want, bound = mo.product(mo.values(*(torch.from_numpy(v) for v in mo.quantize(x, 4)), K), mo.values(*eager["w"], K).t(), dtype)
        mo.close(eager["y"], want, bound, "Y")


@TYPES
@BITS
@pytest.mark.parametrize("T,K,N", [(2048, 2048, 2048), (777, 1000, 1500), (300, 2900, 2600)])
def test_calls_back_to_back_have_the_same_bits(T, K, N, bits, dtype):
    """Calls that follow one another without a wait, on changing inputs, against each by itself: no slot of a ring, no
    scratch and no barrier may let one call's (or stage's) data into another's."""
    def calls(seed):
        m, x = (lib.mx_quantize(normal(r, K, dtype=dtype, seed=seed + i), *lib.mx_empty(r, K, bits)) for i, r in enumerate((N, T)))
        w4, x4 = (lib.mx_quantize(normal(r, K, dtype=dtype, seed=seed + 5 + i), *lib.mx_empty(r, K, 4)) for i, r in enumerate((N, T)))
        dy, X = normal(T, N, dtype=dtype, seed=seed + 7), normal(T, K, dtype=dtype, seed=seed + 8)
        out = [torch.empty(*s, device="cuda", dtype=dtype) for s in ((T, K), (N, K), (T, N), (T, N))]
        return out, [lambda: lib.mx_grad_input(dy, *m, out[0]), lambda: lib.mx_grad_weight(dy, *x, out[1]),
                     lambda: lib.mx4_matmul(*x4, *w4, out[2]), lambda: lib.mx4_linear(X, *w4, out[3])]

    sets = [calls(10 * i) for i in range(3)]
    want = []
    for out, fs in sets:
        for f in fs:
            f()
            torch.cuda.synchronize()
        want.append([o.clone() for o in out])
    for i in range(4):
        for _ in range(8):
            for _, fs in sets:
                fs[i]()
        torch.cuda.synchronize()
        for (out, _), w in zip(sets, want):
            assert torch.equal(out[i], w[i]), f"call {i}: {(out[i] != w[i]).sum()} values differ"


def test_calls_on_several_streams_and_threads():
    """Four threads, a stream each, differently planned calls at once: each call's own bits."""
    import threading
    shapes = [(1, 1024, 700, F32), (70, 4096, 512, BF16), (1500, 777, 900, F32), (2048, 1024, 2048, BF16)]

    def calls(T, K, N, dtype):
        w = lib.mx_quantize(normal(N, K, dtype=dtype, seed=1), *lib.mx_empty(N, K, 4))
        x, dy, ck = normal(T, K, dtype=dtype, seed=2), normal(T, N, dtype=dtype, seed=3), lib.mx_empty(T, K, 8)
        out = [torch.empty(*s, device="cuda", dtype=dtype) for s in ((T, N), (T, K), (N, K))]

        def step(stream=None):
            lib.mx_quantize(x, *ck, stream=stream)
            lib.mx4_linear(x, *w, out[0], stream=stream)
            lib.mx_grad_input(dy, *w, out[1], stream=stream)
            lib.mx_grad_weight(dy, *ck, out[2], stream=stream)
        return out, step

    sets = [calls(*s) for s in shapes]
    want = []
    for out, step in sets:
        step()
        torch.cuda.synchronize()
        want.append([o.clone() for o in out])
        for o in out:
            o.zero_()
    torch.cuda.synchronize()
    errors = []

    def work(step, stream):
        try:
            for _ in range(20):
                step(stream.cuda_stream)
        except BaseException as e:   # noqa: BLE001
            errors.append(e)

    streams = [torch.cuda.Stream() for _ in sets]
    threads = [threading.Thread(target=work, args=(step, stream)) for (_, step), stream in zip(sets, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for (out, _), w in zip(sets, want):
        for a, b in zip(out, w):
            assert torch.equal(a, b)


@TYPES
def test_two_graphs_replayed_together(dtype):
    """Two captured calls that need scratch, replayed at once on two streams, again and again: neither has the other's."""
    T, K, N = 700, 520, 390
    graphs, outs, want = [], [], []
    for i in range(2):
        w = lib.mx_quantize(normal(N, K, dtype=dtype, seed=i), *lib.mx_empty(N, K, 4))
        x, dy = normal(T, K, dtype=dtype, seed=5 + i), normal(T, N + 1, dtype=dtype, seed=7 + i)[:, :N]   # (rows that TMA cannot read)
        y, dx = torch.empty(T, N, device="cuda", dtype=dtype), torch.empty(T, K, device="cuda", dtype=dtype)
        run = lambda x=x, w=w, y=y, dy=dy, dx=dx: (lib.mx4_linear(x, *w, y), lib.mx_grad_input(dy, *w, dx))  # noqa: E731
        run()
        torch.cuda.synchronize()
        want.append((y.clone(), dx.clone()))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append((g, (x, w, dy)))
        outs.append((y, dx))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for (g, _), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


@TYPES
def test_a_training_step(dtype):
    """The operators as they are used together, against the same step in 64 bits."""
    T, K, N = 200, 320, 170
    X, W, dY = normal(T, K, dtype=dtype), normal(N, K, dtype=dtype, seed=1, std=K ** -0.5), normal(T, N, dtype=dtype, seed=2)
    w, ck = lib.mx_quantize(W, *lib.mx_empty(N, K, 4)), lib.mx_quantize(X, *lib.mx_empty(T, K, 8))
    Y, dX, dW = (torch.empty(*s, device="cuda", dtype=dtype) for s in ((T, N), (T, K), (N, K)))
    lib.mx4_linear(X, *w, Y)
    lib.mx_grad_input(dY, *w, dX)
    lib.mx_grad_weight(dY, *ck, dW)
    q = lambda x, b: mo.values(*(torch.from_numpy(v) for v in mo.quantize(x, b)), x.shape[1])  # noqa: E731
    parts = 3 if dtype == F32 else 1
    mo.close(Y, *mo.product(q(X, 4), q(W, 4).t(), dtype), "Y")
    mo.close(dX, *mo.product(dY, q(W, 4), dtype, parts), "dX")
    mo.close(dW, *mo.product(dY.t(), q(X, 8), dtype, parts), "dW")
    # a block's rounding: half a step of the scale at most, which is at most amax / 64 (8 bits: 127 s / 2 < amax)
    amax = X.abs().float().reshape(T, -1, 32).amax(2).repeat_interleave(32, 1).cpu().double()
    assert ((q(X, 8) - X.double().cpu()).abs() <= amax / 127 + 1e-30).all()


def test_a_failed_allocation_leaves_the_output(monkeypatch):
    X, (c, s) = normal(70, 64), lib.mx_quantize(normal(40, 64, seed=1), *lib.mx_empty(40, 64, 4))
    Y = torch.full((70, 40), 3.0, device="cuda")
    monkeypatch.setenv("SGEMM_GB300_FAIL_ALLOC", "1")
    with pytest.raises(lib.SgemmError):
        lib.mx4_linear(X, c, s, Y)
    monkeypatch.delenv("SGEMM_GB300_FAIL_ALLOC")
    assert (Y == 3).all()
    lib.mx4_linear(X, c, s, Y)
    assert torch.isfinite(Y).all() and not (Y == 3).all()


@pytest.fixture
def checked(monkeypatch):
    so = _native.load(checked=True)
    monkeypatch.setattr(_native, "load", lambda *a, **k: so)
    microscale.device_status(clear=True)
    yield so
    assert microscale.device_status(clear=True) == 0, "an index was out of its buffer (0x208) or a wait ran out"


@TYPES
@BITS
@pytest.mark.parametrize("T,K,N,pad,off", [(1, 70, 33, 0, 0), (33, 257, 129, 0, 0), (150, 520, 300, 3, 1), (260, 1024, 600, 8, 0)])
def test_every_index_tested(checked, T, K, N, pad, off, bits, dtype):
    check_store(normal(T, K, dtype=dtype), bits, pad, off)
    check_store(normal(T, K, dtype=dtype), bits, pad, off, transposed=True)
    check_grads(T, K, N, bits, dtype, pad, off)
    if bits == 4:
        check_linear(T, K, N, dtype, pad, off)
