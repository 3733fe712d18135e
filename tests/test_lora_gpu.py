"""lora_forward and lora_backward against their 64-bit forms: one row to many,
odd sizes, ranks and strides, mixed and missing adapters, both types and both
layouts of W, what must not be read or written, streams and graphs."""
import pytest
import torch

import adapter_oracle as ao
import dense_fp32_gemm_06_gb300 as lib
from dense_fp32_gemm_06_gb300 import adapters

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
GUARD = 61


@pytest.fixture(autouse=True)
def _waits():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    assert adapters.device_status(clear=True) == 0


def strided(rows, cols, pitch, dtype, off=0, fill=None):
    """A rows x cols view with that pitch that starts `off` elements behind an aligned address, between guards."""
    buf = torch.full((GUARD + 3 + off + max(rows, 1) * pitch + GUARD,), float("nan") if fill is None else fill, device="cuda", dtype=dtype)
    return buf, buf[64 + off: 64 + off + max(rows, 1) * pitch].as_strided((rows, cols), (pitch, 1), 64 + off)


def make_ids(mix, T, L, seed):
    g = torch.Generator().manual_seed(seed)
    if mix == "one":
        return torch.full((T,), L - 1, dtype=torch.int32)
    if mix == "none":
        return torch.full((T,), -1, dtype=torch.int32)
    if mix == "rows":      # any adapter in any row, some rows without, some ids out of range
        return torch.randint(-1, L + 1, (T,), generator=g, dtype=torch.int32)
    cuts = torch.sort(torch.randint(0, T + 1, (max(1, min(T, 6)),), generator=g)).values
    which = torch.randint(-1, L, (cuts.numel() + 1,), generator=g, dtype=torch.int32)
    return which[torch.searchsorted(cuts, torch.arange(T), right=True)]


def make(T, K, N, L, R, dtype, mix, w_t=False, pad=0, off=0, seed=0, scale=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s, std=1.0: torch.randn(*s, device="cuda", generator=g).mul_(std).to(dtype)  # noqa: E731
    c = {}
    _, c["X"] = strided(T, K, K + pad, dtype, off)
    c["X"].copy_(rnd(T, K))
    _, c["dY"] = strided(T, N, N + pad, dtype, off)
    c["dY"].copy_(rnd(T, N, std=N ** -0.5))
    shape = (N, K) if w_t else (K, N)
    _, W = strided(*shape, shape[1] + pad, dtype, off)
    W.copy_(rnd(*shape, std=max(K, 1) ** -0.5))
    c["W"] = W.t() if w_t else W
    c["A"], c["B"] = rnd(L, R, K, std=max(K, 1) ** -0.5), rnd(L, R, N, std=0.1)
    c["ids"] = make_ids(mix, T, L, seed).cuda()
    c["scale"] = 0.5 + torch.rand(L, device="cuda", generator=g) if scale else None
    return c


def outputs(c, dtype, pad, off):
    T, K = c["X"].shape
    N = c["W"].shape[1]
    L, R = c["A"].shape[:2]
    yb, Y = strided(T, N, N + pad, dtype, off, 7.0)
    xb, dX = strided(T, K, K + pad, dtype, off, 7.0)
    return dict(Y=Y, yb=yb, dX=dX, xb=xb, H=torch.full((T, R), 7.0, device="cuda"), dA=torch.full_like(c["A"], 7.0), dB=torch.full_like(c["B"], 7.0))


def untouched(buf, view):
    m = torch.ones_like(buf, dtype=torch.bool)
    m.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(False)
    return bool((buf[m] == 7.0).all())


def check(T, K, N, L, R, dtype, mix, w_t=False, pad=0, off=0, seed=0, scale=True):
    c = make(T, K, N, L, R, dtype, mix, w_t, pad, off, seed, scale)
    o = outputs(c, dtype, pad, off)
    lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], o["Y"], c["scale"], H=o["H"])
    Y, yb, H, hb = ao.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], c["scale"], dtype)
    ao.close(o["H"], H, hb, "H")
    ao.close(o["Y"], Y, yb, "Y")
    assert untouched(o["yb"], o["Y"])
    Y2 = torch.empty(T, N, device="cuda", dtype=dtype)
    lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], Y2, c["scale"])
    ao.close(Y2, Y, yb, "Y with H in scratch")
    lib.lora_backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], o["H"], o["dX"], o["dA"], o["dB"], c["scale"])
    for name, (want, bound) in ao.lora_backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], o["H"], c["scale"], dtype).items():
        ao.close(o[name], want, bound, name)
    assert untouched(o["xb"], o["dX"])
    return c, o


TYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])


@TYPES
@pytest.mark.parametrize("w_t", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("T", [1, 2, 7, 16, 17, 64, 129, 300])
def test_rows(T, w_t, dtype):
    check(T, 256, 320, 5, 16, dtype, "rows", w_t, seed=T)


@TYPES
@pytest.mark.parametrize("mix", ["one", "none", "runs", "rows"])
def test_mixes(mix, dtype):
    check(333, 264, 200, 9, 8, dtype, mix, seed=3)
    check(40, 520, 136, 33, 4, dtype, mix, True, seed=4)


@TYPES
@pytest.mark.parametrize("R", [1, 3, 4, 8, 15, 16, 17, 32, 33, 64, 65, 100, 128, 200, 256])
def test_ranks(R, dtype):
    check(150, 192, 264, 3, R, dtype, "runs", seed=R)


@TYPES
@pytest.mark.parametrize("T,K,N", [(1, 1, 1), (3, 5, 7), (1, 1000, 1), (1, 1, 1000), (129, 127, 257), (257, 1000, 1500), (100, 777, 333),
                                   (64, 4096, 64), (130, 72, 2056), (513, 65, 63), (1030, 136, 120)])
@pytest.mark.parametrize("w_t", [False, True], ids=["kn", "nk"])
def test_odd_sizes(T, K, N, w_t, dtype):
    check(T, K, N, 4, 8, dtype, "runs", w_t, seed=T + K)


@TYPES
@pytest.mark.parametrize("pad,off", [(8, 0), (3, 0), (0, 1), (5, 3), (8, 4)])
@pytest.mark.parametrize("w_t", [False, True], ids=["kn", "nk"])
def test_strides(pad, off, w_t, dtype):
    check(140, 200, 136, 4, 12, dtype, "rows", w_t, pad, off, seed=pad)


@TYPES
def test_long_rows_and_many_adapters(dtype):
    check(70, 8192, 256, 64, 16, dtype, "rows", seed=8)
    check(24, 256, 8192, 300, 8, dtype, "rows", True, seed=9)


@TYPES
@pytest.mark.parametrize("T,K,N,L,R", [(64, 4096, 512, 64, 16), (64, 3000, 512, 64, 64), (256, 2048, 256, 100, 33), (200, 1536, 136, 50, 100)])
def test_adapters_of_many_stages_behind_a_long_contraction(T, K, N, L, R, dtype):
    c, o = check(T, K, N, L, R, dtype, "rows", True, seed=12)
    for _ in range(30):   # back to back
        lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], Y := torch.empty_like(o["Y"]), c["scale"])
    assert torch.equal(Y, o["Y"])


@TYPES
def test_many_rows(dtype):
    check(4100, 128, 192, 2, 16, dtype, "runs", seed=10)
    check(2500, 192, 128, 40, 8, dtype, "rows", True, seed=11, scale=False)


@TYPES
def test_pitches_past_32_bits(dtype):
    """Rows of X, dY, Y and dX 2^31 - 8 elements apart."""
    T, K, N, L, R = 3, 72, 88, 2, 8
    c = make(T, K, N, L, R, dtype, "rows", seed=71)
    c["ids"] = torch.tensor([1, -1, 0], dtype=torch.int32, device="cuda")
    far = (1 << 31) - 8
    buf = torch.empty((T - 1) * far + 4096, device="cuda", dtype=dtype)
    X, dY, Y, dX = (buf.as_strided((T, n), (far, 1), at) for n, at in ((K, 0), (N, 1024), (N, 2048), (K, 3072)))
    X.copy_(c["X"])
    dY.copy_(c["dY"])
    H, dA, dB = torch.empty(T, R, device="cuda"), torch.empty_like(c["A"]), torch.empty_like(c["B"])
    lib.lora_forward(X, c["W"], c["A"], c["B"], c["ids"], Y, c["scale"], H=H)
    want, bound, _, _ = ao.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], c["scale"], dtype)
    ao.close(Y, want, bound, "Y")
    lib.lora_backward(dY, X, c["W"], c["A"], c["B"], c["ids"], H, dX, dA, dB, c["scale"])
    grads = ao.lora_backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], H, c["scale"], dtype)
    for name, got in (("dX", dX), ("dA", dA), ("dB", dB)):
        ao.close(got, *grads[name], name)


@TYPES
def test_calls_that_follow_one_another(dtype):
    """Each call's input is the output of the call before it, without a wait in between: 40 of them give what waits give."""
    T, K, L, R = 70, 256, 5, 16
    c = make(T, K, K, L, R, dtype, "rows", seed=72)
    ends = []
    for wait in (True, False):
        x = [c["X"].clone().contiguous(), torch.empty(T, K, device="cuda", dtype=dtype)]
        for i in range(40):
            lib.lora_forward(x[i % 2], c["W"], c["A"], c["B"], c["ids"], x[(i + 1) % 2], c["scale"])
            x[(i + 1) % 2].clamp_(-3, 3)
            if wait:
                torch.cuda.synchronize()
        for i in range(40):
            lib.lora_forward(x[i % 2], c["W"], c["A"], c["B"], c["ids"], x[(i + 1) % 2], c["scale"])
            if wait:
                torch.cuda.synchronize()
            if i % 4 == 3:
                x[(i + 1) % 2].mul_(0.01)
        ends.append(x[0].clone())
    assert torch.equal(*ends) and torch.isfinite(ends[0]).all()


@TYPES
def test_no_adapters_and_empty_sizes(dtype):
    c = make(33, 64, 40, 2, 4, dtype, "rows")
    want = c["X"].cpu().double() @ c["W"].cpu().double()
    bound = ao.product_bound(64, dtype) * (c["X"].cpu().double().abs() @ c["W"].cpu().double().abs()) + ao.OUT_U[dtype] * want.abs() + 1e-30
    for L, R in ((0, 4), (2, 0)):
        Y = torch.full((33, 40), 7.0, device="cuda", dtype=dtype)
        lib.lora_forward(c["X"], c["W"], torch.empty(L, R, 64, device="cuda", dtype=dtype), torch.empty(L, R, 40, device="cuda", dtype=dtype), c["ids"], Y)
        ao.close(Y, want, bound * 1.01, "Y")
    e = lambda *s: torch.empty(*s, device="cuda", dtype=dtype)  # noqa: E731
    Y = torch.full((33, 40), 7.0, device="cuda", dtype=dtype)
    lib.lora_forward(e(33, 0), e(0, 40), e(2, 4, 0), c["B"], c["ids"], Y)      # k = 0: H is zero, and Y
    assert not Y.any()
    H = torch.full((33, 4), 7.0, device="cuda")
    lib.lora_forward(c["X"], e(64, 0), c["A"], e(2, 4, 0), c["ids"], e(33, 0), H=H)   # n = 0: H alone
    ao.close(H, *ao.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], None, dtype)[2:], "H")
    dA, dB = torch.full_like(c["A"], 7.0), torch.full_like(c["B"], 7.0)
    lib.lora_backward(e(0, 40), e(0, 64), c["W"], c["A"], c["B"], c["ids"][:0], H[:0], e(0, 64), dA, dB)
    assert not dA.any() and not dB.any()
    dX = torch.full((33, 64), 7.0, device="cuda", dtype=dtype)
    lib.lora_backward(e(33, 0), c["X"], e(64, 0), c["A"], e(2, 4, 0), c["ids"], H, dX, dA, e(2, 4, 0))   # n = 0
    assert not dX.any() and not dA.any()


@TYPES
def test_each_gradient_alone(dtype):
    c = make(200, 136, 264, 4, 8, dtype, "runs", seed=21)
    o = outputs(c, dtype, 0, 0)
    lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], o["Y"], c["scale"], H=o["H"])
    lib.lora_backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], o["H"], o["dX"], o["dA"], o["dB"], c["scale"])
    for name in ("dX", "dA", "dB"):
        one = torch.full_like(o[name], 7.0)
        lib.lora_backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], o["H"], scale=c["scale"], **{name: one})
        assert torch.equal(one, o[name]), name


@TYPES
def test_an_adapter_that_no_row_has_is_not_read(dtype):
    """NaN in the adapters of absent ids, in H of rows without an adapter, and in the scale."""
    T, K, N, L, R = 260, 128, 192, 6, 16
    c = make(T, K, N, L, R, dtype, "runs", seed=31)
    c["ids"] = torch.where(torch.arange(T, device="cuda") < 100, 1, 4).int()
    c["ids"][50:60] = -1
    clean = {k: (v.clone() if v is not None else None) for k, v in c.items()}
    for name in ("A", "B", "scale"):
        for a in (0, 2, 3, 5):
            c[name][a] = float("nan")
            clean[name][a] = 0
    o = outputs(c, dtype, 0, 0)
    lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], o["Y"], c["scale"], H=o["H"])
    assert not o["H"][50:60].any()
    Y, yb, _, _ = ao.lora_forward(c["X"], c["W"], clean["A"], clean["B"], c["ids"], clean["scale"], dtype)
    ao.close(o["Y"], Y, yb, "Y")
    H = o["H"].clone()
    H[50:60] = float("nan")
    lib.lora_backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], H, o["dX"], o["dA"], o["dB"], c["scale"])
    for name, (want, bound) in ao.lora_backward(c["dY"], c["X"], c["W"], clean["A"], clean["B"], c["ids"], o["H"], clean["scale"], dtype).items():
        ao.close(o[name], want, bound, name)
    assert not o["dA"][0].any() and not o["dB"][5].any()


@TYPES
def test_a_row_that_is_not_finite_stays_alone(dtype):
    """NaN or infinity in one row of X reaches its own row of Y (and its adapter's gradient), no other."""
    T, K, N, L, R = 300, 128, 136, 3, 8
    c = make(T, K, N, L, R, dtype, "one", seed=33)
    c["ids"][:150] = 0
    c["ids"][150:] = 2
    want = torch.empty(T, N, device="cuda", dtype=dtype)
    lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], want, c["scale"])
    c["X"][17, 5], c["X"][140, 100] = float("nan"), float("inf")
    Y = torch.empty_like(want)
    lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], Y, c["scale"])
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[17] = keep[140] = False
    assert torch.equal(Y[keep], want[keep])
    assert torch.isnan(Y[17]).all() and not torch.isfinite(Y[140]).any()


@TYPES
@pytest.mark.parametrize("T,N", [(40, 256), (300, 200), (1500, 1024)])
def test_an_adapter_that_is_not_finite_stays_with_its_rows(T, N, dtype):
    """NaN and infinities in one adapter, among rows of others and rows without one."""
    K, L, R = 136, 5, 16
    c = make(T, K, N, L, R, dtype, "rows", seed=34)
    want = torch.empty(T, N, device="cuda", dtype=dtype)
    lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], want, c["scale"])
    c["B"][3, 2, 7], c["B"][3, 0, 100], c["B"][1, 5, N - 1] = float("nan"), float("inf"), -float("inf")
    Y = torch.empty_like(want)
    lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], Y, c["scale"])
    others = (c["ids"] != 3) & (c["ids"] != 1)
    ref, bound, _, _ = ao.lora_forward(c["X"], c["W"], torch.nan_to_num(c["A"], 0, 0, 0), torch.nan_to_num(c["B"], 0, 0, 0), c["ids"], c["scale"], dtype)
    ao.close(Y[others], ref[others.cpu()], bound[others.cpu()], "rows of other adapters")
    rows = c["ids"] == 3
    assert torch.isnan(Y[rows, 7]).all() and not torch.isfinite(Y[rows, 100]).any()
    rows = c["ids"] == 1
    assert not torch.isfinite(Y[rows, N - 1]).any() and torch.isfinite(Y[rows, 7]).all() and torch.isfinite(Y[rows, 100]).all()


@TYPES
@pytest.mark.parametrize("T,L", [(64, 64), (700, 3)])
def test_the_same_call_gives_the_same_bits(T, L, dtype):
    c = make(T, 1000, 520, L, 16, dtype, "rows", seed=41)
    got = []
    for _ in range(3):
        o = outputs(c, dtype, 0, 0)
        lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], o["Y"], c["scale"], H=o["H"])
        lib.lora_backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], o["H"], o["dX"], o["dA"], o["dB"], c["scale"])
        got.append([o[k].clone() for k in ("Y", "H", "dX", "dA", "dB")])
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


@TYPES
def test_streams_and_graphs(dtype):
    """Calls on several streams at once, and captured and replayed on other inputs, give what calls alone give."""
    cs = [make(T, 512, 384, 6, 16, dtype, "rows", seed=50 + T) for T in (5, 200, 1000)]
    alone = []
    for c in cs:
        o = outputs(c, dtype, 0, 0)
        lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], o["Y"], c["scale"], H=o["H"])
        lib.lora_backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], o["H"], o["dX"], o["dA"], o["dB"], c["scale"])
        alone.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    both = [outputs(c, dtype, 0, 0) for c in cs]
    torch.cuda.synchronize()
    for _ in range(4):
        for c, o, s in zip(cs, both, streams):
            lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], o["Y"], c["scale"], H=o["H"], stream=s.cuda_stream)
            lib.lora_backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], o["H"], o["dX"], o["dA"], o["dB"], c["scale"], stream=s.cuda_stream)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert all(torch.equal(a[k], b[k]) for k in ("Y", "H", "dX", "dA", "dB"))
    c, o = cs[1], outputs(cs[1], dtype, 0, 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], o["Y"], c["scale"], H=o["H"])
        lib.lora_backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], o["H"], o["dX"], o["dA"], o["dB"], c["scale"])
    c["X"].mul_(0.5)
    c["ids"].copy_(c["ids"].flip(0))
    want = outputs(c, dtype, 0, 0)
    lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], want["Y"], c["scale"], H=want["H"])
    lib.lora_backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], want["H"], want["dX"], want["dA"], want["dB"], c["scale"])
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o[k], want[k]) for k in ("Y", "H", "dX", "dA", "dB"))


def test_failed_allocation_leaves_the_outputs(monkeypatch):
    c = make(40, 64, 72, 3, 8, BF16, "rows")
    Y = torch.full((40, 72), 7.0, device="cuda", dtype=BF16)
    monkeypatch.setenv("SGEMM_GB300_FAIL_ALLOC", "1")
    with pytest.raises(lib.SgemmError) as err:
        lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], Y, c["scale"])
    assert err.value.status == 100 and "cudaError 2" in str(err.value)
    monkeypatch.delenv("SGEMM_GB300_FAIL_ALLOC")
    torch.cuda.synchronize()
    assert (Y == 7.0).all()
    lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], Y, c["scale"])
    ao.close(Y, *ao.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], c["scale"], BF16)[:2], "Y")


def test_gradients_against_differences_of_the_kernel():
    """FP32: a step h along a direction changes <Y, dY> by the gradient times h."""
    c = make(60, 96, 80, 3, 8, F32, "runs", seed=61)
    o = outputs(c, F32, 0, 0)
    lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], o["Y"], c["scale"], H=o["H"])
    lib.lora_backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], o["H"], o["dX"], o["dA"], o["dB"], c["scale"])
    g = torch.Generator(device="cuda").manual_seed(5)
    for name, grad in (("X", "dX"), ("A", "dA"), ("B", "dB")):
        step = torch.randn(c[name].shape, device="cuda", generator=g) * 2.0 ** -4
        side = []
        for sign in (1, -1):
            moved = {**c, name: c[name] + sign * step}
            Y = torch.empty_like(o["Y"])
            lib.lora_forward(moved["X"], moved["W"], moved["A"], moved["B"], moved["ids"], Y, moved["scale"])
            side.append(float((Y.double() * c["dY"].double()).sum()))
        want = float((o[grad].double() * step.double()).sum())
        # <Y, dY> is linear in each of the three: only rounding separates the two, 1e-5 of the sums of magnitudes (~60 * 80 * 0.1)
        assert abs((side[0] - side[1]) / 2 - want) < 1e-5 * 500, name


def test_binding_refusals_on_the_gpu():
    c = make(8, 16, 24, 2, 4, F32, "rows")
    Y = torch.empty(8, 24, device="cuda")
    for over in (dict(ids=c["ids"].long()), dict(ids=c["ids"][:4]), dict(A=c["A"].to(BF16)), dict(A=c["A"].transpose(1, 2)), dict(B=c["B"][:, :, :5]),
                 dict(scale=c["scale"].double()), dict(Y=torch.empty(8, 24, device="cuda", dtype=BF16)), dict(Y=torch.empty(24, 8, device="cuda").t()),
                 dict(X=c["X"].t()), dict(W=torch.empty(16, 48, device="cuda")[:, ::2]), dict(X=c["X"][:1].expand(8, 16)),
                 dict(W=c["W"][:1].expand(16, 24)), dict(Y=torch.empty(1, 24, device="cuda").expand(8, 24))):
        a = {**c, "Y": Y, **over}
        with pytest.raises(lib.SgemmError) as err:
            lib.lora_forward(a["X"], a["W"], a["A"], a["B"], a["ids"], a["Y"], a["scale"])
        assert err.value.status == -1, over
