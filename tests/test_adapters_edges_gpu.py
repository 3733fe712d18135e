"""What the adapter calls do at the edges: infinities in H, an adapter that is
not finite at all beside other requests', no contraction, a failed allocation
of the product under them, gradients of very wide matrices, operands that a
call does not need."""
import pytest
import torch

import adapter_oracle as ao
import dense_fp32_gemm_06_gb300 as lib
import test_lora_gpu as lora
from dense_fp32_gemm_06_gb300 import adapters

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
INF = float("inf")


@pytest.fixture(autouse=True)
def _waits():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    assert adapters.device_status(clear=True) == 0


def same(got, want):
    """Equal infinities and NaN, whatever is finite."""
    got, want = got.detach().cpu().double(), want.cpu().double()
    return bool((torch.isnan(got) == torch.isnan(want)).all() and (torch.isposinf(got) == torch.isposinf(want)).all()
                and (torch.isneginf(got) == torch.isneginf(want)).all())


# ---------------------------------------------------------------- infinities

@TYPES
@pytest.mark.parametrize("T", [40, 300, 1500])
def test_infinities_in_h_and_its_gradient(T, dtype):
    """dB = H^T dY: an infinite H gives infinities of its sign times dY's, not NaN; so does the largest FP32 H with a small dY."""
    K, N, L, R = 64, 136, 2, 16
    c = lora.make(T, K, N, L, R, dtype, "one", seed=T)
    c["ids"][: T // 2] = 0
    H = torch.randn(T, R, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    H[3, 2], H[T - 1, 5], H[T - 2, 7] = INF, -INF, float("nan")
    dB = torch.empty_like(c["B"])
    lib.lora_backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], H, None, None, dB, c["scale"])
    want = torch.stack([H[c["ids"] == a].cpu().double().t() @ c["dY"][c["ids"] == a].cpu().double() for a in range(L)])
    assert torch.isinf(want).sum() >= 2 * N - 8 and same(dB, want)


@TYPES
@pytest.mark.parametrize("T", [40, 300])
def test_the_largest_h(T, dtype):
    K, N, L, R = 64, 136, 1, 8
    c = lora.make(T, K, N, L, R, dtype, "one", seed=T)
    H = torch.ones(T, R, device="cuda")
    H[5, 3] = torch.finfo(F32).max            # above bfloat16's largest value
    c["dY"][5] = torch.where(c["dY"][5] < 0, -0.25, 0.25)
    dB = torch.empty_like(c["B"])
    lib.lora_backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], H, None, None, dB, c["scale"])
    want, bound = ao.lora_backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], H, c["scale"], dtype)["dB"]
    ao.close(dB, want, bound, "dB")


# ---------------------------------------------------------------- infinities in the projection

@TYPES
@pytest.mark.parametrize("T", [1, 40, 300])
def test_infinities_of_a_rows_own_adapter(T, dtype):
    """Y = X W + H B with an infinity or NaN in B: in the rows of that adapter what H and the sum make of it, elsewhere nothing."""
    K, N, L, R = 128, 136, 3, 16
    c = lora.make(T, K, N, L, R, dtype, "one", seed=T)
    if T > 1:
        c["ids"][: T // 2] = 0
        c["ids"][1] = -1
    b = c["B"][L - 1]
    b[2, 7], b[0, 100], b[3, N - 1], b[5, N - 1] = INF, -INF, INF, -INF
    c["B"][0, 4, 9] = float("nan")
    Y, H = torch.empty(T, N, device="cuda", dtype=dtype), torch.empty(T, R, device="cuda")
    lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], Y, c["scale"], H=H)
    X, W, _, B, ids, _ = ao.lora_parts(c["X"], c["W"], c["A"], c["B"], c["ids"], c["scale"])
    want = X @ W
    for a in range(L):
        want[ids == a] += H.cpu().double()[ids == a] @ B[a]
    assert same(Y, want)
    assert torch.isinf(want).any()


@TYPES
def test_an_infinite_h_in_the_projection(dtype):
    T, K, N, L, R = 300, 128, 264, 3, 16
    c = lora.make(T, K, N, L, R, dtype, "runs", seed=5)
    c["ids"][:20] = 1
    c["scale"][1] = INF                                # H of adapter 1: infinities
    Y, H = torch.empty(T, N, device="cuda", dtype=dtype), torch.empty(T, R, device="cuda")
    lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], Y, c["scale"], H=H)
    assert torch.isinf(H[:20]).all()
    X, W, _, B, ids, _ = ao.lora_parts(c["X"], c["W"], c["A"], c["B"], c["ids"], c["scale"])
    want = X @ W
    for a in range(L):
        want[ids == a] += H.cpu().double()[ids == a] @ B[a]
    assert same(Y, want)


# ---------------------------------------------------------------- a diverged adapter

def microseconds(call, n=5):
    call()
    torch.cuda.synchronize()
    best = INF
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3)
    return best


@TYPES
@pytest.mark.parametrize("T,K,N,R,mix", [(64, 1024, 512, 16, "rows"), (256, 512, 1024, 16, "rows"), (300, 264, 200, 80, "rows"), (2100, 256, 1300, 8, "runs"),
                                         (1, 512, 264, 16, "one")])
def test_a_diverged_adapter(T, K, N, R, mix, dtype):
    """An adapter of nothing but NaN (infinities, in a second call): the other rows' results are theirs, and the call is about as quick."""
    L = 8
    c = lora.make(T, K, N, L, R, dtype, mix, True, seed=T)
    if T > 1:
        c["ids"][::9] = 2
    Y = torch.empty(T, N, device="cuda", dtype=dtype)
    call = lambda: lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], Y, c["scale"])  # noqa: E731
    sound = microseconds(call)
    others = ((c["ids"] != 2) & (c["ids"] != 7)).cpu()
    want, bound, _, _ = ao.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], c["scale"], dtype)
    for value in (float("nan"), INF):
        c["B"][2], c["B"][7] = value, value
        diverged = microseconds(call)
        ao.close(Y.cpu()[others], want[others], bound[others], "rows of other adapters")
        assert not torch.isfinite(Y.cpu()[~others & (c["ids"].cpu() >= 0) & (c["ids"].cpu() < L)]).any()
        # the diverged rows' own terms are added beside the tile's product
        assert diverged <= 4 * sound + 20, (diverged, sound)


@TYPES
@pytest.mark.parametrize("T", [7, 40, 300, 1500])
@pytest.mark.parametrize("R", [16, 80])
def test_what_is_not_finite_on_both_sides(R, T, dtype):
    """Infinite H (an infinite scale) and NaN H (NaN in A) beside infinities in B, of the same rows and of others: every term as IEEE has it."""
    K, N, L = 136, 264, 5
    c = lora.make(T, K, N, L, R, dtype, "rows", seed=T)
    c["ids"][:4] = torch.tensor([1, 2, 3, 0], device="cuda")
    c["scale"][1] = INF
    c["A"][2, 1, 5] = float("nan")
    c["B"][1, 3, 5], c["B"][1, 0, 6], c["B"][1, 1, 6], c["B"][3, R - 1, 9], c["B"][3, 2, 200] = INF, INF, -INF, -INF, INF
    c["B"][1, :, 11] = 0                       # an infinite H times zeros
    Y, H = torch.empty(T, N, device="cuda", dtype=dtype), torch.empty(T, R, device="cuda")
    lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], Y, c["scale"], H=H)
    X, W, _, B, ids, _ = ao.lora_parts(c["X"], c["W"], c["A"], c["B"], c["ids"], c["scale"])
    want = X @ W
    for a in range(L):
        want[ids == a] += H.cpu().double()[ids == a] @ B[a]
    assert same(Y, want)
    assert torch.isnan(want[0, 11]) and torch.isinf(want[2, 9]) and torch.isfinite(want[3]).all()


# ---------------------------------------------------------------- no contraction

@TYPES
@pytest.mark.parametrize("T", [5, 40])
def test_no_contraction_is_zero_whatever_the_adapter_holds(T, dtype):
    """K = 0: Y = 0 (and N = 0: dX = 0), as the header says, beside an adapter that is not finite."""
    N, L, R = 72, 2, 4
    e = lambda *s: torch.empty(*s, device="cuda", dtype=dtype)  # noqa: E731
    B = torch.full((L, R, N), INF, device="cuda", dtype=dtype)
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    Y, H = torch.full((T, N), 7.0, device="cuda", dtype=dtype), torch.full((T, R), 7.0, device="cuda")
    lib.lora_forward(e(T, 0), e(0, N), e(L, R, 0), B, ids, Y, H=H)
    assert not Y.any() and not H.any()
    dX = torch.full((T, N), 7.0, device="cuda", dtype=dtype)
    lib.lora_backward(e(T, 0), torch.ones(T, N, device="cuda", dtype=dtype), e(N, 0), B, e(L, R, 0), ids, H, dX)
    assert not dX.any()


# ---------------------------------------------------------------- failed allocations

@pytest.mark.parametrize("T,K,N", [(400, 1000, 1001)])
def test_a_failed_allocation_of_the_product_leaves_the_outputs(T, K, N, monkeypatch):
    """FP32, where the projection is sgemm's: its scratch is asked for before anything of the call is enqueued."""
    c = lora.make(T, K, N, 3, 8, F32, "rows")
    Y, H, dX = (torch.full(s, 7.0, device="cuda") for s in ((T, N), (T, 8), (T, K)))
    dA, dB = torch.full_like(c["A"], 7.0), torch.full_like(c["B"], 7.0)
    forward = lambda: lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], Y, c["scale"], H=H)  # noqa: E731
    backward = lambda: lib.lora_backward(c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], Hs, dX, dA, dB, c["scale"])  # noqa: E731
    Hs = torch.zeros(T, 8, device="cuda")
    for what in ("1", "sgemm"):              # every allocation, and sgemm's alone
        monkeypatch.setenv("SGEMM_GB300_FAIL_ALLOC", what)
        for call in (forward, backward):
            with pytest.raises(lib.SgemmError) as err:
                call()
            assert err.value.status == 100 and "cudaError 2" in str(err.value)
        torch.cuda.synchronize()
        assert all((v == 7.0).all() for v in (Y, H, dX, dA, dB)), what
    monkeypatch.delenv("SGEMM_GB300_FAIL_ALLOC")
    forward()
    want, bound, h, hb = ao.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], c["scale"], F32)
    ao.close(Y, want, bound, "Y")
    ao.close(H, h, hb, "H")


# ---------------------------------------------------------------- very wide matrices

@pytest.mark.parametrize("dtype,K", [(F32, 64 * 65536 + 70), (BF16, 128 * 65536 + 136)], ids=["f32", "bf16"])
def test_gradients_of_more_columns_than_a_grid_axis_has_blocks(dtype, K):
    T, N, L, R = 3, 8, 1, 1
    g = torch.Generator(device="cuda").manual_seed(3)
    X = torch.randn(T, K, device="cuda", generator=g).to(dtype)
    dY = torch.randn(T, N, device="cuda", generator=g).to(dtype)
    B = torch.randn(L, R, N, device="cuda", generator=g).to(dtype)
    A, W = torch.zeros(L, R, K, device="cuda", dtype=dtype), torch.zeros(K, N, device="cuda", dtype=dtype)
    ids = torch.tensor([0, -1, 0], dtype=torch.int32, device="cuda")
    H = torch.randn(T, R, device="cuda", generator=g)
    dA, dB = torch.empty_like(A), torch.empty_like(B)
    lib.lora_backward(dY, X, W, A, B, ids, H, None, dA, dB)
    grads = ao.lora_backward(dY, X[:, :64], W[:64], A[:, :, :64], B, ids, H, None, dtype)
    ao.close(dB, *grads["dB"], "dB")
    U = dY.cpu().double() @ B[0].cpu().double().t()
    want = (U[[0, 2]].t() @ X.cpu()[[0, 2]].double())[None]
    size = (U[[0, 2]].abs().t() @ X.cpu()[[0, 2]].double().abs())[None]
    ao.close(dA, want, (2.0 ** -20 + (2.0 ** -16 if dtype == BF16 else 0)) * size + ao.OUT_U[dtype] * want.abs() + 1e-30, "dA")


# ---------------------------------------------------------------- what a call does not need

@TYPES
def test_operands_that_a_gradient_does_not_need_may_be_missing(dtype):
    c = lora.make(70, 136, 264, 4, 8, dtype, "runs", seed=21)
    o = lora.outputs(c, dtype, 0, 0)
    lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], o["Y"], c["scale"], H=o["H"])
    every = (c["dY"], c["X"], c["W"], c["A"], c["B"], c["ids"], o["H"])
    lib.lora_backward(*every, o["dX"], o["dA"], o["dB"], c["scale"])
    for name, missing in (("dX", (1, 6)), ("dA", (2, 3, 6)), ("dB", (1, 2, 3, 4))):
        one = torch.full_like(o[name], 7.0)
        lib.lora_backward(*(None if i in missing else v for i, v in enumerate(every)), scale=c["scale"], **{name: one})
        assert torch.equal(one, o[name]), name
    # one that is needed is refused by its position in the C call
    for name, gone, status in (("dX", 2, 12), ("dX", 3, 14), ("dX", 4, 15), ("dA", 1, 9), ("dB", 6, 18), ("dB", 5, 16)):
        with pytest.raises(lib.SgemmError) as err:
            lib.lora_backward(*(None if i == gone else v for i, v in enumerate(every)), scale=c["scale"], **{name: torch.empty_like(o[name])})
        assert err.value.status == status, (name, gone)
    with pytest.raises(lib.SgemmError):
        lib.lora_backward(None, *every[1:], o["dX"])
    for gone in range(5):
        a = [c["X"], c["W"], c["A"], c["B"], c["ids"], o["Y"]]
        a[gone] = None
        with pytest.raises(lib.SgemmError):
            lib.lora_forward(*a, c["scale"])
    with pytest.raises(lib.SgemmError):
        lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], None, c["scale"])
