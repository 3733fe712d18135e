"""That the inputs of test_mx_float32_gpu.py tell kernels with FP32 results
from such that leave out a bfloat16 part or never take out an accumulator: a
model of the tensor core's sums on the CPU, right and with each mistake."""
import numpy as np
import pytest
import torch


def cut(x):
    """To 24 bits, towards zero."""
    m, e = np.frexp(x)
    return np.ldexp(np.trunc(m * 2.0 ** 24), e - 24)


def planes(x, count):
    """The first `count` bfloat16 parts of FP32 values, each what the ones before left, rounded."""
    parts, left = [], torch.tensor(x, dtype=torch.float32)
    for _ in range(count):
        p = left.bfloat16().float()
        parts.append(p.double().numpy())
        left = left - p
    return parts


def model(parts, m, step, taken):
    """sum_i a_i m_i, a in parts: an accumulator cut off after each `step` products of a part, taken out after `taken` values into an FP32 sum."""
    total = np.float32(0)
    for i in range(0, len(m), taken):
        acc = 0.0
        for j in range(i, min(i + taken, len(m)), step):
            for p in parts:
                acc = cut(acc + float(p[j:j + step] @ m[j:j + step]))
        total = np.float32(total + np.float32(acc))
    return float(total)


def test_a_missing_part_shows_in_one_term():
    rng = np.random.default_rng(1)
    for _ in range(200):
        v = float(np.ldexp(int(rng.integers(2 ** 23, 2 ** 24)), int(rng.integers(-43, -3))))
        x, m = np.zeros(1000), np.ldexp(1.0, rng.integers(-10, 11, 1000))
        at = int(rng.integers(1000))
        x[at] = v
        want = v * m[at]
        assert model(planes(x, 3), m, 16, 128) == want
        two = model(planes(x, 2), m, 16, 128)
        assert two != want or sum(planes(v, 2)) == v


@pytest.mark.parametrize("depth,step,taken,first,small,lost", [(16384, 16, 128, 1, 1 / 16, 127 / 16), (16384 // 8, 16, 128, 1, 1 / 16, 127 / 16),
                                                               (32768, 64, 1024, 32, 1 / 64, 992 / 64), (32768 // 8, 64, 1024, 32, 1 / 64, 992 / 64)])
def test_an_accumulator_that_stays_shows_in_long_sums(depth, step, taken, first, small, lost):
    """The whole contraction and an eighth of it, of gradients and of products of 4-bit matrices."""
    x = np.full(depth, small)
    x[:first] = 0
    x[0] = 2.0 ** 24
    want, one = float(x.sum()), np.ones(depth)
    assert abs(model(planes(x, 3), one, step, taken) - want) <= lost + 1
    assert abs(model(planes(x, 3), one, step, depth) - want) > lost + 1
    assert abs(model(planes(x, 3), one, step, 8 * taken) - want) > lost + 1 or depth <= 8 * taken
