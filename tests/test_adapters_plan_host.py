"""adapters_plan_for without a GPU: refusals by position, before any CUDA call."""
import pytest

from dense_fp32_gemm_06_gb300 import _native


@pytest.mark.parametrize("args,status", [((0, 8, 8), 1), ((-3, 8, 8), 1), ((8, 0, 8), 2), ((8, 8, 0), 3), ((8, 8, 8, None), 4)])
def test_refusals(args, status):
    plan = _native.AdaptersPlan() if len(args) == 3 else None
    assert _native.load().adapters_plan_for(*args[:3], plan) == status
