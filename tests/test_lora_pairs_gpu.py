"""The bfloat16 projection of many rows, whose tiles CTA pairs take in turn,
three and more each: barriers across the two CTAs, W and X and the adapters
loaded by halves, H written by halves, both accumulators and lists over again,
rings whose phases carry across tiles.  Each test asserts by the plan that it
gets there; single CTAs that take tiles in turn, and clusters along the
contraction, are asserted once each too."""
import pytest
import torch

import adapter_oracle as ao
import dense_fp32_gemm_06_gb300 as lib
import test_adapter_parts as parts
import test_lora_gpu as lora
from dense_fp32_gemm_06_gb300 import _native, adapters

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _waits():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    assert adapters.device_status(clear=True) == 0


def in_pairs(t, k, n):
    p = adapters.plan(t, k, n)
    return p["pair"] == 1 and p["rows"] == 256 and p["tiles"] >= 3


def check(T, K, N, L, R, mix, w_t, pad=0, off=0, seed=0, backward=False):
    assert in_pairs(T, K, N), adapters.plan(T, K, N)
    if not backward:
        c = lora.make(T, K, N, L, R, BF16, mix, w_t, pad, off, seed)
        o = lora.outputs(c, BF16, pad, off)
        lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], o["Y"], c["scale"], H=o["H"])
        Y, yb, _, _ = parts.forward(c["X"], c["W"], c["A"], c["B"], c["ids"], c["scale"])
        ao.close(o["Y"], Y, yb, "Y")
        assert lora.untouched(o["yb"], o["Y"])
        return c, o
    assert in_pairs(T, N, K), adapters.plan(T, N, K)
    return parts.check(T, K, N, L, R, mix, w_t, pad, off, seed)


@pytest.mark.parametrize("w_t", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("T,K,N,L,R,mix", [
    (4096, 200, 4096, 5, 16, "runs"),
    (4100, 72, 4104, 9, 48, "rows"),         # tails of t, n and k; ranks past a stage's half
    (5000, 136, 3500, 6, 80, "runs"),
    (4333, 264, 4001, 7, 130, "rows"),       # an odd n: copies of W and B, Y stored element by element
    (4096, 72, 4096, 300, 8, "rows"),        # as many adapters as a tile has rows: more ring phases than tiles
    (6000, 65, 3400, 4, 16, "none"),     # no row has an adapter
    (4096, 128, 4096, 3, 16, "one"),
])
def test_forward(T, K, N, L, R, mix, w_t):
    check(T, K, N, L, R, mix, w_t, seed=T)


@pytest.mark.parametrize("w_t", [False, True], ids=["kn", "nk"])
@pytest.mark.parametrize("T,K,N,L,R,mix", [(12000, 1000, 1100, 5, 16, "runs"), (15000, 520, 777, 6, 40, "rows")])
def test_with_the_gradients(T, K, N, L, R, mix, w_t):
    check(T, K, N, L, R, mix, w_t, seed=T, backward=True)


@pytest.mark.parametrize("pad,off", [(8, 0), (3, 1)])
def test_strides(pad, off):
    check(4100, 136, 4100, 4, 12, "rows", False, pad, off)


@pytest.mark.parametrize("w_t", [False, True], ids=["kn", "nk"])
def test_tiles_without_an_adapter_and_a_diverged_one(w_t):
    """Rows of whole tiles without an adapter between others; then NaN in all of one adapter, infinities in some of another."""
    T, K, N, L, R = 4864, 200, 4096, 6, 48
    assert in_pairs(T, K, N)
    c = lora.make(T, K, N, L, R, BF16, "rows", w_t, seed=6)
    t = torch.arange(T, device="cuda")
    c["ids"][(t >= 512) & (t < 1280) | (t >= 4000)] = -1
    c["ids"][:256] = 3
    Y = torch.empty(T, N, device="cuda", dtype=BF16)
    lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], Y, c["scale"])
    want, bound, H, _ = parts.forward(c["X"], c["W"], c["A"], c["B"], c["ids"], c["scale"])
    ao.close(Y, want, bound, "Y")
    c["B"][2] = float("nan")
    c["B"][4, 33, 1000], c["B"][4, 47, N - 1], c["B"][4, 0, N - 1] = float("inf"), -float("inf"), float("inf")
    lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], Y, c["scale"])
    ids = c["ids"].cpu()
    others = (ids != 2) & (ids != 4)
    ao.close(Y.cpu()[others], want[others], bound[others], "rows of other adapters")
    assert torch.isnan(Y.cpu()[ids == 2]).all()
    got, h = Y.cpu().double()[ids == 4], H[ids == 4]
    assert torch.equal(got[:, 1000], torch.where(h[:, 33] > 0, 1.0, -1.0) * float("inf"))
    assert torch.equal(torch.isnan(got[:, N - 1]), h[:, 0] * h[:, 47] > 0) and not torch.isfinite(got[:, N - 1]).any()
    clean = torch.ones(N, dtype=torch.bool)
    clean[[1000, N - 1]] = False
    ao.close(got[:, clean], want[ids == 4][:, clean], bound[ids == 4][:, clean], "an adapter's features that are finite")


def test_the_same_bits_back_to_back():
    c, o = check(4100, 264, 4104, 40, 48, "rows", True, seed=9)
    Y = [torch.empty_like(o["Y"]) for _ in range(8)]
    for y in Y:
        lib.lora_forward(c["X"], c["W"], c["A"], c["B"], c["ids"], y, c["scale"])
    assert all(torch.equal(y, o["Y"]) for y in Y)


def test_with_every_index_tested(monkeypatch):
    so = _native.load(checked=True)
    monkeypatch.setattr(_native, "load", lambda *a, **k: so)
    check(4333, 136, 4001, 5, 48, "rows", False, seed=3)
    check(4096, 72, 4096, 4, 16, "runs", True, 3, 1, seed=4)
    assert adapters.device_status(clear=True) == 0, "an index was out of its buffer (0x208) or a wait ran out"


@pytest.mark.parametrize("T,K,N,want", [
    (4000, 64, 1500, dict(pair=0, split=1)), (64, 4096, 512, dict(pair=0)), (1, 4096, 4096, dict(rows=16, pair=0)),
])
def test_other_plans(T, K, N, want):
    p = adapters.plan(T, K, N)
    assert all(p[k] == v for k, v in want.items()), p
    assert p["tiles"] >= 2 if T == 4000 else p["split"] >= 2, p
    for w_t in (False, True):
        parts.check(T, K, N, 5, 16, "rows" if T > 1 else "one", w_t, seed=T)
