"""What the adapter calls do at the edges: infinities in H."""
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
