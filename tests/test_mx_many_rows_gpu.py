"""The quantiser and the reader of almost 2^31 rows: the numbers of rows and of
tiles of them do not fit a sum in 32 bits."""
import pytest
import torch

import dense_fp32_gemm_06_gb300 as lib
import mx_oracle as mo
from dense_fp32_gemm_06_gb300 import microscale

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _waits():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.empty_cache()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()   # (77 GB)
    assert microscale.device_status(clear=True) == 0


# pairs of rows by 64 and single ones by 32 (transposed), and rows that start anywhere
@pytest.mark.parametrize("rows,transposed", [(2 ** 31 - 6, True), (2 ** 31 - 5, True), (2 ** 31 - 1, False)])
def test_as_many_rows_as_there_may_be(rows, transposed):
    x = torch.empty((2, rows) if transposed else (rows, 2), device="cuda", dtype=torch.bfloat16)
    # a pattern of 4099 rows, so that every row's codes are known
    pattern = torch.randn(4099, 2, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    X, whole = x.t() if transposed else x, rows // 4099 * 4099
    for c in range(2):
        X[:whole, c].view(-1, 4099).copy_(pattern[:, c].expand(whole // 4099, -1))
        X[whole:, c].copy_(pattern[:rows - whole, c])
    codes, scales = lib.mx_empty(rows, 2, 4)
    codes.fill_(0xA5), scales.fill_(0xA5)
    lib.mx_quantize(X, codes, scales)
    want = [torch.from_numpy(v).cuda() for v in mo.quantize(pattern, 4)]
    for got, w in ((codes, want[0]), (scales, want[1])):
        for at in range(0, whole, 4099 * 4096):   # (65 MB at a time)
            part = got[at:min(at + 4099 * 4096, whole)]
            assert (part.reshape(-1, 4099, w.shape[1]) == w).all(), at
        assert torch.equal(got[whole:], w[:rows - whole])
    y = x.view(rows, 2).fill_(0)
    lib.mx_dequantize(codes, scales, y)
    w = mo.values(want[0], want[1], 2).bfloat16().cuda()
    for at in range(0, whole, 4099 * 4096):
        assert (y[at:min(at + 4099 * 4096, whole)].view(-1, 4099, 2) == w).all(), at
    assert torch.equal(y[whole:], w[:rows - whole])
