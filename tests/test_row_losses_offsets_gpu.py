"""Losses over rows whose logits, divided by the temperature, share a large
offset: p and the gradient depend on differences only, so the bounds of
adapter_oracle hold as they are.  Logits are whole steps of the type at that
offset, some of them tied at the maximum.  And losses that are not a number."""
import pytest
import torch

import dense_fp32_gemm_06_gb300 as lib
import test_row_losses_gpu as losses

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def rows(T, V, dtype, top, step, levels, seed=0):
    """Logits top - step * (0 .. levels - 1), several at the top of each row."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    down = torch.randint(0, levels, (T, V), device="cuda", generator=g)
    down[:, V // 3] = 0
    down[:, ::7] = 0
    return (top - step * down.double()).to(dtype), g


CASES = [  # type, maximum, step, levels, temperature of distill
    (F16, 3.0e4, 16.0, 3, 1.0), (F16, 3.0e4, 16.0, 40, 10.0), (F16, -2.0e4, 16.0, 40, 10.0), (F16, 2000.0, 1.0, 12, 0.1), (F16, 100.0, 0.0625, 8, 1e-4),
    (BF16, 1.0e6, 4096.0, 3, 1.0), (BF16, 1.0e6, 4096.0, 30, 2048.0), (BF16, 5.0e6, 32768.0, 3, 1.0), (BF16, -1.0e6, 4096.0, 30, 2048.0),
    (BF16, 100.0, 0.5, 8, 1e-4), (BF16, 100.0, 0.5, 8, 1e-5), (BF16, 300.0, 2.0, 12, 1.0), (BF16, 60.0, 0.25, 60, 0.25),
    (F32, 1.0e5, 2.0 ** -7, 900, 1.0), (F32, 4.0e6, 0.5, 16, 1.0), (F32, -1.0e5, 2.0 ** -7, 900, 0.5), (F32, 1000.0, 2.0 ** -13, 60000, 0.01), (F32, 90.0, 2.0 ** -10, 9000, 1.0),
]
SHAPES = [(3, 1000), (5, 4099), (2, 40001), (300, 8192), (1, 131072)]


@pytest.mark.parametrize("dtype,top,step,levels,tau", CASES)
@pytest.mark.parametrize("T,V", SHAPES)
def test_distill(T, V, dtype, top, step, levels, tau):
    z, g = rows(T, V, dtype, top, step, levels, seed=V)
    teacher, index, w = losses.distill_inputs(z, g, 16)
    losses.check_distill(z, teacher * tau, index, w, tau)


@pytest.mark.parametrize("dtype,top,step,levels,tau", [c for c in CASES if c[4] == 1.0])
@pytest.mark.parametrize("T,V", SHAPES)
def test_policy(T, V, dtype, top, step, levels, tau):
    z, g = rows(T, V, dtype, top, step, levels, seed=V)
    losses.check_policy(z, *losses.policy_inputs(z, g))


def test_a_row_longer_than_a_cluster_holds():
    z, g = rows(2, 600_001, F32, 4.0e6, 0.5, 16, seed=1)
    losses.check_distill(z, *losses.distill_inputs(z, g, 16), 1.0)
    losses.check_policy(z, *losses.policy_inputs(z, g))
    z, g = rows(2, 300_001, BF16, 1.0e6, 4096.0, 30, seed=2)
    losses.check_distill(z, *losses.distill_inputs(z, g, 16), 2048.0)


@pytest.mark.parametrize("dtype,top,step,tau", [(F16, 3.0e4, 16.0, 10.0), (BF16, 1.0e6, 4096.0, 2048.0)])
def test_on_other_boundaries_and_in_place(dtype, top, step, tau):
    z, g = rows(9, 3001, dtype, top, step, 30, seed=3)
    teacher, index, w = losses.distill_inputs(z, g, 16)
    losses.check_distill(z, teacher * tau, index, w, tau, *reversed(losses.like(z, off=1)))   # stored element by element
    losses.check_distill(z, teacher * tau, index, w, tau, grad=z)


@pytest.mark.parametrize("dtype,top,step", [(F16, 3.0e4, 16.0), (F16, 20.0, 0.125), (BF16, 1.0e6, 4096.0), (BF16, 20.0, 0.125), (F32, 1.0e5, 2.0 ** -7)])
@pytest.mark.parametrize("T,V", [(5, 1003), (40, 8192), (3, 131072)])
def test_large_factors(T, V, dtype, top, step):
    """Weights that make the gradient's factor far more than 1, of either sign."""
    z, g = rows(T, V, dtype, top, step, 12, seed=V)
    y, old, adv, ref, w = losses.policy_inputs(z, g)
    losses.check_policy(z, y, old, adv, ref, 1000 * (w + 0.1))
    tau = max(step, 1.0)
    teacher, index, w = losses.distill_inputs(z, g, 16)
    losses.check_distill(z, teacher * tau, index, 1000 * (w - 0.5), tau)


# ---------------------------------------------------------------- a loss that is not a number

def test_a_loss_that_is_not_a_number_has_no_finite_gradient():
    """An advantage of NaN, and a ratio that overflowed beside an advantage of 0: min(r A, clip(r) A) is NaN, and so is what comes of it."""
    z, g = losses.logits(6, 1003, F32, seed=4)
    y, old, adv, ref, w = losses.policy_inputs(z, g)
    adv[1] = float("nan")
    old[3], adv[3] = -losses.INF, 0.0
    loss, grad = torch.empty(6, device="cuda"), torch.empty_like(z)
    lib.policy_loss(z, y, old, adv, loss, grad, weight=torch.ones_like(w))
    ok = torch.tensor([0, 2, 4, 5], device="cuda")
    assert torch.isnan(loss[[1, 3]]).all() and torch.isnan(grad[[1, 3]]).all()
    assert torch.isfinite(loss[ok]).all() and torch.isfinite(grad[ok]).all()
