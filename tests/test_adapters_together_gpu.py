"""The operators together: the example's training step and decoding step, and
every kernel through the bounds-checking library (each global index tested
before its access) with no test failed."""
import importlib.util
import os

import pytest
import torch

import adapter_oracle as ao
import dense_fp32_gemm_06_gb300 as lib
from dense_fp32_gemm_06_gb300 import _native, adapters
import test_lora_gpu as lora
import test_row_losses_gpu as losses

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def test_example():
    spec = importlib.util.spec_from_file_location("example_adapters", os.path.join(ROOT, "examples", "adapters.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    distil, reward, (tokens, W, A, B, scale, served) = example.main(steps=60, vocab=1024, width=256, quiet=True)
    # by construction both improve: the teacher is the projection plus a matrix of rank 8 <= 16, and one token in eight is rewarded
    assert distil[1] < 0.8 * distil[0], distil
    assert reward[1] > reward[0], reward
    ids = torch.tensor([0, 1, -1, 1, 0, -1])
    want, bound, _, _ = ao.lora_forward(tokens, W, A.to(BF16), B.to(BF16), ids, scale, BF16)
    ao.close(served, want, bound, "served")
    assert adapters.device_status() == 0


@pytest.fixture
def checked(monkeypatch):
    so = _native.load(checked=True)
    assert so.sgemm_version().endswith(b"checked)")
    monkeypatch.setattr(_native, "load", lambda *a, **k: so)
    adapters.device_status(clear=True)
    yield so
    assert adapters.device_status(clear=True) == 0, "an index was out of its buffer (0x208) or a wait ran out"


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,K,N,L,R,mix,w_t,pad,off", [
    (1, 256, 320, 2, 16, "one", True, 0, 0),          # few rows
    (17, 257, 131, 5, 7, "rows", False, 0, 0),        # odd everything: copies of every operand
    (300, 200, 264, 6, 16, "runs", True, 5, 3),       # strides
    (300, 136, 520, 6, 80, "rows", False, 0, 0),      # ranks past a stage
    (1100, 512, 640, 3, 130, "runs", True, 8, 0),     # ranks past a pass of the shrink; CTA pairs
])
def test_adapters_with_every_index_tested(checked, dtype, T, K, N, L, R, mix, w_t, pad, off):
    lora.check(T, K, N, L, R, dtype, mix, w_t, pad, off, seed=T)


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,V", [(3, 7), (5, 1003), (400, 5001), (330, 33000), (3, 262151)])
def test_losses_with_every_index_tested(checked, dtype, T, V):
    z, g = losses.logits(T, V, dtype, seed=V)
    losses.check_distill(z, *losses.distill_inputs(z, g, 20), 2.0)
    losses.check_policy(z, *losses.policy_inputs(z, g))
