"""mx4_linear of a few rows: X is rounded within the product's launch where
that is the shorter way, and by a launch in front of it (which needs scratch,
by which the tests tell the two) where every CTA would round too much of it.
Either way the values are the same."""
import pytest
import torch

import dense_fp32_gemm_06_gb300 as lib
import mx_oracle as mo
from dense_fp32_gemm_06_gb300 import microscale

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _waits():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    assert microscale.device_status(clear=True) == 0


# sizes at which both ways were timed, and the shorter one by 5 % or more
@pytest.mark.parametrize("T,K,N,dtype,fused", [
    (1, 4096, 4096, BF16, True), (16, 4096, 4096, BF16, True), (1, 8192, 8192, BF16, True), (8, 8192, 8192, BF16, True), (16, 8192, 8192, BF16, False),
    (16, 16384, 8192, BF16, False), (8, 16384, 2048, BF16, True), (4, 16384, 8192, F32, True), (12, 8192, 8192, F32, False), (16, 4096, 16384, F32, False),
    (16, 2048, 2048, F32, True)])
def test_the_shorter_way_is_taken(T, K, N, dtype, fused, monkeypatch):
    g = torch.Generator(device="cuda").manual_seed(T + K)
    x = torch.randn(T, K, device="cuda", generator=g).to(dtype)
    w = lib.mx_quantize(torch.randn(N, K, device="cuda", generator=g).to(dtype), *lib.mx_empty(N, K, 4))
    Y = torch.empty(T, N, device="cuda", dtype=dtype)
    lib.mx4_linear(x, *w, Y)
    some = slice(0, 200)
    want, bound = mo.product(mo.values(*(torch.from_numpy(v) for v in mo.quantize(x, 4)), K), mo.values(w[0][some], w[1][some], K).t(), dtype)
    mo.close(Y[:, some], want, bound, "Y")
    codes = lib.mx_quantize(x, *lib.mx_empty(T, K, 4))
    same = lib.mx4_matmul(*codes, *w, torch.empty_like(Y))
    assert torch.equal(Y, same)   # (the same plan, and the same codes)
    monkeypatch.setenv("SGEMM_GB300_FAIL_ALLOC", "1")
    if fused:
        lib.mx4_linear(x, *w, Y.zero_())
        assert torch.equal(Y, same)
    else:
        with pytest.raises(lib.SgemmError):
            lib.mx4_linear(x, *w, Y)
