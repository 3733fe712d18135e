"""distill_topk and policy_loss with their gradients against their 64-bit
forms: short and long rows, odd ones, every type, masked rows and places,
infinities, in-place gradients, pitches past 32 bits."""
import pytest
import torch

import adapter_oracle as ao
import dense_fp32_gemm_06_gb300 as lib

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
INF = float("inf")


@pytest.fixture(autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def logits(T, V, dtype, pitch=None, off=0, seed=0, std=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pitch = pitch or V
    buf = torch.full((off + T * pitch + 64,), float("nan"), device="cuda", dtype=dtype)
    z = buf.as_strided((T, V), (pitch, 1), off)
    z.copy_(torch.randn(T, V, device="cuda", generator=g) * std)
    return z, g


def like(z, off=None):
    """A gradient buffer of sevens with z's pitch, and the view in it."""
    off = z.storage_offset() if off is None else off
    buf = torch.full((off + z.shape[0] * max(z.stride(0), 1) + 64,), 7.0, device="cuda", dtype=z.dtype)
    return buf, buf.as_strided(z.shape, z.stride(), off)


def untouched(buf, view):
    m = torch.ones_like(buf, dtype=torch.bool)
    m.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(False)
    return bool((buf[m] == 7.0).all())


def distill_inputs(z, g, top, seed=0):
    T, V = z.shape
    index = torch.rand(T, V, device="cuda", generator=g).topk(min(top, V), 1).indices.int() if V <= 4096 else \
        (torch.randint(0, V, (T, 1), device="cuda", generator=g) + torch.arange(top, device="cuda") * 61).remainder(V).int()
    index = torch.cat([index, torch.full((T, top - index.shape[1]), -1, device="cuda", dtype=torch.int32)], 1)
    return torch.randn(T, top, device="cuda", generator=g) * 2, index, torch.rand(T, device="cuda", generator=g)


def check_distill(z, teacher, index, weight, tau, grad=None, buf=None):
    keep = z.clone()
    loss = torch.full((z.shape[0],), 7.0, device="cuda")
    if grad is None:
        buf, grad = like(z)
    lib.distill_topk(z, teacher, index, loss, grad, weight=weight, temperature=tau)
    want, bound, wg, gb = ao.distill(keep, teacher, index, weight, tau, z.dtype)
    ao.close(loss, want, bound, "loss")
    ao.close(grad, wg, gb, "grad")
    if buf is not None:
        assert untouched(buf, grad)
    only = torch.empty_like(loss)
    if grad.data_ptr() != z.data_ptr():
        lib.distill_topk(z, teacher, index, only, None, weight=weight, temperature=tau)
        assert torch.equal(only, loss)
    return loss, grad


def policy_inputs(z, g):
    """Old log-probabilities whose ratios stay 1e-3 away from where the clip begins."""
    T, V = z.shape
    y = torch.randint(0, V, (T,), device="cuda", generator=g).int()
    lp = torch.log_softmax(z.double(), 1).gather(1, y.long()[:, None])[:, 0]
    lp = torch.where(torch.isfinite(lp), lp, torch.full_like(lp, -5.0))
    step = torch.randn(T, device="cuda", generator=g) * 0.3
    for edge in (0.8, 1.28):
        near = (step.exp() - edge).abs() < 1e-2
        step = torch.where(near, step + 0.05, step)
    return y, (lp - step).float(), torch.randn(T, device="cuda", generator=g), (lp + 0.3 * torch.randn(T, device="cuda", generator=g)).float(), torch.rand(T, device="cuda", generator=g)


def check_policy(z, y, old, adv, ref, weight, kl=0.05, grad=None, buf=None):
    keep = z.clone()
    T = z.shape[0]
    loss, logp = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
    if grad is None:
        buf, grad = like(z)
    lib.policy_loss(z, y, old, adv, loss, grad, ref=ref, weight=weight, clip_low=0.2, clip_high=0.28, kl_coef=kl, logp=logp)
    want, bound, lp, lb, wg, gb = ao.policy(keep, y, old, adv, ref, weight, 0.2, 0.28, kl, z.dtype)
    ao.close(loss, want, bound, "loss")
    ao.close(logp, lp, lb, "logp")
    ao.close(grad, wg, gb, "grad")
    if buf is not None:
        assert untouched(buf, grad)
    if grad.data_ptr() != z.data_ptr():
        l2, g2 = torch.empty_like(loss), torch.empty_like(grad)
        lib.policy_loss(z, y, old, adv, l2, g2, ref=ref, weight=weight, clip_low=0.2, clip_high=0.28, kl_coef=kl)
        assert torch.equal(l2, loss) and torch.equal(g2, grad)
        lib.policy_loss(z, y, old, adv, l2, ref=ref, weight=weight, clip_low=0.2, clip_high=0.28, kl_coef=kl)
        assert torch.equal(l2, loss)


SIZES = [(1, 1), (3, 2), (2, 7), (5, 17), (4, 255), (3, 1000), (40, 4097), (7, 8192), (3, 32768), (2, 50021), (200, 16392), (1, 131072), (2, 262151), (330, 33000)]


@TYPES
@pytest.mark.parametrize("T,V", SIZES)
def test_distill_sizes(T, V, dtype):
    z, g = logits(T, V, dtype, seed=V)
    check_distill(z, *distill_inputs(z, g, 20), 2.0)


@TYPES
@pytest.mark.parametrize("T,V", SIZES)
def test_policy_sizes(T, V, dtype):
    z, g = logits(T, V, dtype, seed=V)
    check_policy(z, *policy_inputs(z, g))


@pytest.mark.parametrize("V", [600_001, 1_500_000])
def test_rows_longer_than_a_cluster_holds(V):
    z, g = logits(3, V, F32, seed=3)
    check_distill(z, *distill_inputs(z, g, 64), 1.0)
    check_policy(z, *policy_inputs(z, g))
    keep = z.clone()
    check_policy(z, *policy_inputs(z, g), grad=z)
    check_distill(keep, *distill_inputs(keep, g, 64), 1.0, grad=keep)


@TYPES
@pytest.mark.parametrize("top", [1, 2, 31, 64, 300, 1024])
@pytest.mark.parametrize("tau", [0.5, 1.0, 4.0])
def test_distill_tops_and_temperatures(top, tau, dtype):
    z, g = logits(9, 3001, dtype, seed=top)
    check_distill(z, *distill_inputs(z, g, top), tau)


@TYPES
@pytest.mark.parametrize("pitch,off", [(1001, 0), (1008, 1), (1003, 3), (1016, 5)])
def test_pitches(pitch, off, dtype):
    z, g = logits(21, 1000, dtype, pitch, off, seed=pitch)
    teacher, index, w = distill_inputs(z, g, 8)
    check_distill(z, teacher, index, w, 2.0)
    check_policy(z, *policy_inputs(z, g))
    buf, grad = like(z, off=off + 1)      # the gradient on other boundaries than the logits
    check_distill(z, teacher, index, w, 2.0, grad, buf)
    check_policy(z, *policy_inputs(z, g), grad=grad.clone(), buf=None)


@TYPES
@pytest.mark.parametrize("V", [37, 5000, 70001])
def test_in_place(V, dtype):
    z, g = logits(13, V, dtype, seed=1)
    teacher, index, w = distill_inputs(z, g, 16)
    check_distill(z, teacher, index, w, 2.0, grad=z)
    z, g = logits(13, V, dtype, seed=2)
    check_policy(z, *policy_inputs(z, g), grad=z)


@TYPES
def test_rows_that_count_for_nothing(dtype):
    z, g = logits(12, 3000, dtype, seed=5)
    teacher, index, w = distill_inputs(z, g, 8)
    w[2] = 0
    z[2] = float("nan")             # weight 0: not looked at
    index[3] = -1                   # no place
    index[4] = 3000                 # none inside
    teacher[5] = -INF               # none with a chance
    z[6] = -INF                     # nothing left of the row
    z[7, ::2] = -INF                # half of it left
    lowest = torch.finfo(dtype).min
    z[8] = lowest                   # a mask of the type's lowest value over all of the row
    z[9, 5:] = lowest               # and over most of it
    teacher[9, 1:] = torch.finfo(F32).min
    index[9] = torch.arange(8, dtype=torch.int32, device="cuda")   # places that are masked for the student have no chance
    index[9, 0] = 2
    index[10, 1::2] = index[10, 0]  # an index named again
    index[11, :] = index[11, 0]
    teacher[11, 3] = -INF
    index[7] = torch.arange(1, 17, 2, dtype=torch.int32, device="cuda")
    loss, grad = check_distill(z, teacher, index, w, 2.0)
    for t in (2, 3, 4, 5, 6):
        assert loss[t] == 0 and not grad[t].any()
    z, g = logits(12, 3000, dtype, seed=6)
    y, old, adv, ref, w = policy_inputs(z, g)
    w[2] = 0
    y[3], y[4] = -100, 3000
    z[3] = float("nan")
    z[6] = -INF
    z[7, ::2] = -INF
    y[7] = 1
    z[8] = lowest
    z[9, 5:] = lowest
    y[9] = 2
    old[7:10] = torch.log_softmax(z[7:10].double(), 1).gather(1, y[7:10].long()[:, None])[:, 0].float() - 0.1
    ref[7:10] = old[7:10]
    check_policy(z, y, old, adv, ref, w)
    check_policy(z, y, old, adv, None, None, kl=0.0)


def test_an_impossible_label_has_an_infinite_loss():
    """A place of the teacher's that the student's mask leaves no chance: KL is infinite, the gradient is not."""
    z, g = logits(4, 500, F32, seed=7)
    teacher, index, w = distill_inputs(z, g, 4)
    z[1].scatter_(0, index[1, :1].long(), -INF)
    loss, grad = check_distill(z, teacher, index, w, 1.0)
    assert loss[1] == INF and torch.isfinite(grad).all()
    y, old, adv, ref, w = policy_inputs(z, g)
    y[1] = index[1, 0]
    adv[1] = -1.0
    check_policy(z, y, old, adv, None, w, kl=0.0)     # ratio 0: the clipped side holds, no gradient


@TYPES
def test_nan_spreads_over_its_row_alone(dtype):
    z, g = logits(6, 4100, dtype, seed=8)
    teacher, index, w = distill_inputs(z, g, 8)
    want = [torch.empty(6, device="cuda"), torch.empty_like(z)]
    lib.distill_topk(z, teacher, index, want[0], want[1], weight=w)
    z[2, 77] = float("nan")
    z[4, 4099] = INF
    loss, grad = torch.empty(6, device="cuda"), torch.empty_like(z)
    lib.distill_topk(z, teacher, index, loss, grad, weight=w)
    ok = torch.tensor([0, 1, 3, 5], device="cuda")
    assert torch.equal(loss[ok], want[0][ok]) and torch.equal(grad[ok], want[1][ok])
    assert torch.isnan(loss[2]) and torch.isnan(grad[2]).all() and torch.isnan(loss[4])
    y, old, adv, ref, w = policy_inputs(torch.nan_to_num(z, posinf=0.0), g)
    lib.policy_loss(z, y, old, adv, loss, grad, ref=ref, weight=w, kl_coef=0.1)
    assert torch.isnan(loss[2]) and torch.isnan(grad[2]).all() and torch.isfinite(loss[ok]).all() and torch.isfinite(grad[ok]).all()


def test_large_logits():
    z, g = logits(8, 2000, F32, seed=9, std=1e4)
    check_distill(z, *distill_inputs(z, g, 8), 100.0)
    z.mul_(1e30)
    loss, grad = torch.empty(8, device="cuda"), torch.empty_like(z)
    teacher, index, w = distill_inputs(z, g, 8)
    lib.distill_topk(z, teacher, index, loss, grad, weight=w)
    assert torch.isfinite(grad).all()


@TYPES
def test_the_same_call_gives_the_same_bits(dtype):
    z, g = logits(77, 40001, dtype, seed=10)
    teacher, index, w = distill_inputs(z, g, 64)
    runs = []
    for _ in range(3):
        loss, grad = torch.empty(77, device="cuda"), torch.empty_like(z)
        lib.distill_topk(z, teacher, index, loss, grad, weight=w, temperature=2.0)
        runs.append((loss, grad))
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(runs[0], r))


def test_a_pitch_past_32_bits():
    z = torch.empty(0, device="cuda", dtype=BF16)
    buf = torch.empty(2 * ((1 << 31) - 8) + 4096, device="cuda", dtype=BF16)
    z = buf.as_strided((3, 1003), ((1 << 31) - 8, 1), 1)
    g = torch.Generator(device="cuda").manual_seed(1)
    z.copy_(torch.randn(3, 1003, device="cuda", generator=g))
    teacher, index, w = distill_inputs(z, g, 8)
    grad = torch.empty(3, 1003, device="cuda", dtype=BF16)
    loss = torch.empty(3, device="cuda")
    lib.distill_topk(z, teacher, index, loss, grad, weight=w)
    want, bound, wg, gb = ao.distill(z.clone(), teacher, index, w, 1.0, BF16)
    ao.close(loss, want, bound, "loss")
    ao.close(grad, wg, gb, "grad")


def test_streams_and_graphs():
    z, g = logits(50, 20000, BF16, seed=11)
    y, old, adv, ref, w = policy_inputs(z, g)
    want, wg = torch.empty(50, device="cuda"), torch.empty_like(z)
    lib.policy_loss(z, y, old, adv, want, wg, ref=ref, weight=w, kl_coef=0.1)
    loss, grad = torch.empty_like(want), torch.empty_like(z)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    lib.policy_loss(z, y, old, adv, loss, grad, ref=ref, weight=w, kl_coef=0.1, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(loss, want) and torch.equal(grad, wg)
    loss.zero_()
    grad.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.policy_loss(z, y, old, adv, loss, grad, ref=ref, weight=w, kl_coef=0.1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(loss, want) and torch.equal(grad, wg)


def test_gradients_against_differences_of_the_kernel():
    """A step along a direction changes the summed loss by the gradient times the step, to second order: h = 2^-9 on logits
    of size 2 leaves less than 1 % of the first order here."""
    z, g = logits(20, 300, F32, seed=12)
    teacher, index, w = distill_inputs(z, g, 8)
    y, old, adv, ref, _ = policy_inputs(z, g)
    step = torch.randn(z.shape, device="cuda", generator=g) * 2.0 ** -9

    def total(kind, zz, grad=None):
        loss = torch.empty(20, device="cuda")
        if kind == "distill":
            lib.distill_topk(zz, teacher, index, loss, grad, weight=w, temperature=2.0)
        else:
            lib.policy_loss(zz, y, old, adv, loss, grad, ref=ref, weight=w, clip_low=0.2, clip_high=0.28, kl_coef=0.05)
        return loss.double()

    for kind in ("distill", "policy"):
        grad = torch.empty_like(z)
        total(kind, z, grad)
        diff = (total(kind, z + step) - total(kind, z - step)) / 2
        want = (grad.double() * step.double()).sum(1)
        assert (diff - want).abs().max() <= 0.01 * want.abs().max() + 1e-5, kind


def test_binding_refusals_on_the_gpu():
    z, g = logits(4, 50, F32)
    teacher, index, w = distill_inputs(z, g, 4)
    loss = torch.empty(4, device="cuda")
    for over in (dict(index=index.long()), dict(index=index[:, :2]), dict(teacher=teacher.double()), dict(loss=loss[:3]), dict(grad=torch.empty(4, 51, device="cuda")),
                 dict(grad=z.half()), dict(weight=w[:2]), dict(logits=z.t()), dict(logits=z.double())):
        a = dict(logits=z, teacher=teacher, index=index, loss=loss, grad=None, weight=w)
        a.update(over)
        with pytest.raises(lib.SgemmError):
            lib.distill_topk(a["logits"], a["teacher"], a["index"], a["loss"], a["grad"], weight=a["weight"])
    y, old, adv, ref, w = policy_inputs(z, g)
    with pytest.raises(lib.SgemmError):
        lib.policy_loss(z, y, old, adv, loss, kl_coef=0.1)
    with pytest.raises(lib.SgemmError):
        lib.policy_loss(z, y, old, adv[:2], loss)
