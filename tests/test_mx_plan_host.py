"""microscale.plan without a GPU: a type or call that it does not know is
refused by the C ABI, before any CUDA call."""
import pytest
import torch

import dense_fp32_gemm_06_gb300 as lib
from dense_fp32_gemm_06_gb300 import microscale


@pytest.mark.parametrize("args,status", [(("linear", 8, 64, 8, torch.float16), 5), (("grad_input", 8, 64, 8, torch.float64, 8), 5), (("product", 8, 64, 8), 1),
                                         (("grad_weight", 8, 64, 8, torch.bfloat16, 5), 6), (("linear", 0, 64, 8), 2)])
def test_refusals(args, status):
    with pytest.raises(lib.SgemmError) as e:
        microscale.plan(*args)
    assert e.value.status == status
