"""Long contractions of the microscaled products with bfloat16 results: the
tensor core truncates its sum once per MMA, which all of one sign add up to a
loss in proportion to the depth.  No accumulator may take more than 1024 MMAs."""
import pytest
import torch

import dense_fp32_gemm_06_gb300 as lib
import mx_oracle as mo
from dense_fp32_gemm_06_gb300 import _native, microscale

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _waits():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()   # (matrices of gigabytes)
    assert microscale.device_status(clear=True) == 0


def positive(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g).abs().to(BF16)


def coded(x, bits, down=1, right=1):
    """x's codes and scales, both repeated that often (x has whole blocks)."""
    c, s = lib.mx_quantize(x, *lib.mx_empty(*x.shape, bits))
    want = mo.values(c, s, x.shape[1])
    codes, scales = lib.mx_empty(x.shape[0] * down, x.shape[1] * right, bits, device="cuda")
    codes.view(down, x.shape[0], right, -1).copy_(c.view(1, x.shape[0], 1, -1))
    scales.copy_(s.repeat(down, right))
    return (codes, scales), want


def check(got, want, depth, mmas, what, first=None):
    """Sums of positive terms: an accumulator of 1024 MMAs is off by at most 2^-22 of itself in each; then FP32 additions
    of the accumulators and of up to eight CTAs' parts (and of what was there), and the result's rounding."""
    off = (1024 * 2.0 ** -22 + (depth / mmas / 1024 + 10) * 2.0 ** -24) * want
    if first is not None:
        want = want + first
    bound = off + 2.0 ** -8 * (want.abs() + off)
    rows, cols = want.shape
    for r in range(0, got.shape[0], rows):
        mo.close(got[r:r + rows, :cols][:want.shape[0]], want[:got.shape[0] - r], bound[:got.shape[0] - r], what)
    for c in range(0, got.shape[1], cols):
        assert torch.equal(got[:, c:c + cols], got[:, :cols]), what


# (tokens, features of dY and of X: in 64s and 128s, so that tiles are CTA pairs' or split)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,N,K", [(2 ** 19, 2048, 2048), (2 ** 22, 64, 128)])
def test_weight_gradients_of_many_tokens(T, N, K, bits):
    P = 2048
    p = microscale.plan("grad_weight", T, K, N, BF16, bits)
    assert p["split"] == 1 and p["pair"] if N > 64 else p["split"] > 1
    y, x = positive(P, 64, seed=1), positive(P, 128, seed=2)
    m, X = coded(x, bits, T // P, K // 128)
    want = y.double().cpu().t() @ X * (T // P)
    dY = y.repeat(T // P, N // 64)
    dW = torch.empty(N, K, device="cuda", dtype=BF16)
    lib.mx_grad_weight(dY, *m, dW)
    check(dW, want, T, 16, "dW")
    first = (torch.randn(64, 128, generator=torch.Generator().manual_seed(3)) * T).to(BF16)
    dW.copy_(first.cuda().repeat(N // 64, K // 128))
    lib.mx_grad_weight(dY, *m, dW, accumulate=True)
    check(dW, want, T, 16, "dW added", first.double())


@pytest.mark.parametrize("bits", [4, 8])
def test_input_gradients_of_many_features(bits):
    T, N, K, P = 260, 2 ** 19, 2048, 2048
    y, w = positive(20, P, seed=1), positive(P, 128, seed=2)
    m, W = coded(w, bits, N // P, K // 128)
    dX = torch.empty(T, K, device="cuda", dtype=BF16)
    lib.mx_grad_input(y.repeat(T // 20, N // P), *m, dX)
    check(dX, y.double().cpu() @ W * (N // P), N, 16, "dX")


@pytest.mark.parametrize("T,N", [(5, 512), (40, 512), (260, 1024)])
def test_linear_of_many_features(T, N):
    K, P = 2 ** 23, 8192
    x, w = positive(T, P, seed=1), positive(64, P, seed=2)
    m, W = coded(w, 4, N // 64, K // P)
    q, X = coded(x, 4, 1, K // P)
    want = X @ W.t() * (K // P)
    Y = torch.empty(T, N, device="cuda", dtype=BF16)
    lib.mx4_matmul(*q, *m, Y)
    check(Y, want, K, 64, "Y of codes")
    Y.zero_()
    lib.mx4_linear(x.repeat(1, K // P), *m, Y)
    check(Y, want, K, 64, "Y")


def test_a_failed_allocation_of_the_sums_leaves_the_output(monkeypatch):
    T, N, K = 2 ** 18, 64, 128
    dY, (c, s) = torch.ones(T, N, device="cuda", dtype=BF16), lib.mx_empty(T, K, 8)
    c.fill_(1), s.fill_(127)
    dW = torch.full((N, K), 3.0, device="cuda", dtype=BF16)
    assert T // microscale.plan("grad_weight", T, K, N, BF16, 8)["split"] > 16384
    monkeypatch.setenv("SGEMM_GB300_FAIL_ALLOC", "1")
    with pytest.raises(lib.SgemmError):
        lib.mx_grad_weight(dY, c, s, dW)
    monkeypatch.delenv("SGEMM_GB300_FAIL_ALLOC")
    assert (dW == 3).all()
    lib.mx_grad_weight(dY, c, s, dW)
    assert (dW == T).all()


def test_graphs_replayed_together_have_sums_of_their_own():
    """Two captured calls on two streams at once, beside eager ones on a third: each keeps its accumulators' sums to itself."""
    T, N, K = 2 ** 18, 64, 128
    sets = []
    for i in range(3):
        y, x = positive(T, N, seed=i), positive(T, K, seed=10 + i)
        m = lib.mx_quantize(x, *lib.mx_empty(T, K, 8))
        out = torch.empty(N, K, device="cuda", dtype=BF16)
        run = lambda y=y, m=m, out=out: lib.mx_grad_weight(y, *m, out)  # noqa: E731
        run()
        torch.cuda.synchronize()
        want, graph = out.clone(), None
        if i < 2:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                run()
        out.zero_()
        # (a graph does not hold what it was captured on: y and m have to stay as long as it)
        sets.append((graph.replay if graph else run, out, want, torch.cuda.Stream(), (graph, y, m)))
    torch.cuda.synchronize()
    assert len({tuple(s[2].flatten()[:50].tolist()) for s in sets}) == 3
    for _ in range(10):
        for call, _, _, stream, _ in sets:
            with torch.cuda.stream(stream):
                call()
    torch.cuda.synchronize()
    for _, out, want, _, _ in sets:
        assert torch.equal(out, want)


@pytest.mark.parametrize("bits", [4, 8])
def test_every_index_tested(bits, monkeypatch):
    """Through the bounds-checking library: split, pairs, odd sizes."""
    so = _native.load(checked=True)
    monkeypatch.setattr(_native, "load", lambda *a, **k: so)
    microscale.device_status(clear=True)
    test_weight_gradients_of_many_tokens(2 ** 18, 64, 128, bits)
    for T, N, K in ((2 ** 18 + 5, 65, 129), (2 ** 15 + 7, 2050, 2049)):
        p = microscale.plan("grad_weight", T, K, N, BF16, bits)
        assert T / p["split"] > 16384
        dY, (c, s) = torch.ones(T, N, device="cuda", dtype=BF16), lib.mx_empty(T, K, bits)
        c.fill_(0x22 if bits == 4 else 1), s.fill_(127)
        dW = torch.empty(N, K, device="cuda", dtype=BF16)
        lib.mx_grad_weight(dY, c, s, dW)
        assert (dW == torch.tensor(float(T)).to(BF16).cuda()).all()   # (whole numbers below 2^24: no step rounds)
    assert microscale.device_status(clear=True) == 0
