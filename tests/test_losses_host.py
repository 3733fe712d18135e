"""The losses without a GPU: refusals beside those of their positions."""
from dense_fp32_gemm_06_gb300 import _native


def test_a_temperature_whose_reciprocal_is_infinite_is_refused():
    P, so = 4096, _native.load()
    args = [4, 9, 3, 0, P, 9, P, P, P, 2.0, P, P, 9, 0]
    for tau in (1e-39, 4e-39, 1e-45):
        args[9] = tau
        assert so.distill_topk(*args) == 10, tau
