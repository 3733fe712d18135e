"""Cases for measuring the microscaled operators: what each is called with, its plain form in elementary torch
operations, its definition in 64 bits and its work.

A microscaled matrix holds blocks of 32 consecutive values of a row as small codes with one power of two: value =
code 2^e, e = scale byte - 127 (byte 255: the block is not finite).  e is the least that lets the block's largest
magnitude be held.  4 bits: e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), two codes a byte, the first in the low bits;
8 bits: whole numbers -127 .. 127.  Codes are rounded to nearest, ties to even, and fill whole blocks (zeros behind a
row's end); rows of scales start 16 bytes apart.

    store        Y = X^: a matrix is quantised, kept, and read back (a checkpoint of activations, weights laid out)
    linear       Y = X^ W^^T: X (T x K) is quantised to 4 bits within the call, W (N x K) is kept in 4 bits
    matmul       the same of an X that is there in 4 bits already
    grad_input   dX = dY W^, the gradient of linear by X, straight through the rounding
    grad_weight  dW = dY^T X^ from a checkpoint of X in 8 (or 4) bits

`own` False runs the plain forms, True the library's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the repository's odd problem (777 x 1500): an FP32 weight matrix stored k x n, laid out in 4 bits along k
        dict(name="store 4 bits 1500x777", op="store", dtype="f32", T=1500, K=777, bits=4, x_t=True),
        # activations of a short batch, kept in 8 bits for the backward pass
        dict(name="store 8 bits 257x4096", op="store", dtype="bf16", T=257, K=4096, bits=8, x_t=False),
        # the repository's largest matrix: activations of 8192 tokens
        dict(name="store 8 bits 8192x8192", op="store", dtype="bf16", T=8192, K=8192, bits=8, x_t=False),
        # one token of one request: the latency of a decoding step's projection
        dict(name="linear 1 token", op="linear", dtype="bf16", T=1, K=4096, N=4096),
        # the repository's odd problem (1000 x 1500 x 777) in FP32
        dict(name="linear 1000x1500x777", op="linear", dtype="f32", T=1000, K=777, N=1500),
        # the repository's largest problem as a batch of prompts
        dict(name="linear 8192^3", op="linear", dtype="bf16", T=8192, K=8192, N=8192),
        # a decoding step of 64 requests whose rows several projections read: quantised before
        dict(name="matmul 64 tokens", op="matmul", dtype="bf16", T=64, K=4096, N=4096),
        # the repository's worked size with FP32 results
        dict(name="matmul 2048^3", op="matmul", dtype="f32", T=2048, K=2048, N=2048),
        # a small ragged fine-tuning batch
        dict(name="grad_input 257x1500x1000", op="grad_input", dtype="bf16", T=257, K=1000, N=1500, bits=4),
        # an ordinary fine-tuning step of 8192 tokens
        dict(name="grad_input 8192x4096x4096", op="grad_input", dtype="bf16", T=8192, K=4096, N=4096, bits=4),
        # the repository's worked size in FP32
        dict(name="grad_weight 2048^3", op="grad_weight", dtype="f32", T=2048, K=2048, N=2048, bits=8),
        # an ordinary training step from a checkpoint of 8192 tokens
        dict(name="grad_weight 8192x4096x4096", op="grad_weight", dtype="bf16", T=8192, K=4096, N=4096, bits=8),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _size(rng, low, high):
    """A size of the range: half of the time a multiple of 64, else as it falls."""
    n = _log_int(rng, low, high)
    return max(64, n // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["store", "linear", "linear", "matmul", "grad_input", "grad_weight"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "store":
        return dict(c, T=_log_int(rng, 1, 8192), K=_size(rng, 256, 8192), bits=rng.choice([4, 8]), x_t=rng.random() < 0.25)
    if op in ("linear", "matmul"):
        return dict(c, T=_log_int(rng, 1, 8192), K=_size(rng, 256, 8192), N=_size(rng, 256, 8192))
    return dict(c, T=_log_int(rng, 16, 8192), K=_size(rng, 256, 4096), N=_size(rng, 256, 4096), bits=rng.choice([4, 8]))


def _blocks(k):
    return (k + 31) // 32


def _buffers(rows, k, bits):
    """Where the codes and scales of a rows x k matrix go: rows of whole blocks, rows of scales 16 bytes apart."""
    b = _blocks(k)
    codes = torch.empty(rows, b * 16, dtype=torch.uint8, device="cuda") if bits == 4 else torch.empty(rows, b * 32, dtype=torch.int8, device="cuda")
    return codes, torch.empty(rows, (b + 15) // 16 * 16, dtype=torch.uint8, device="cuda")[:, :b]


def _round_blocks(x, bits):
    """Codes as numbers (rows x blocks x 32) and exponents (rows x blocks) of finite values."""
    rows, k = x.shape
    x = torch.nn.functional.pad(x.float(), (0, _blocks(k) * 32 - k)).reshape(rows, -1, 32)
    m, p = torch.frexp(x.abs().amax(2))
    e = p - 3 + (m > 0.75).int() if bits == 4 else p - 7 + (m > 127 / 128).int()
    e = torch.where(m == 0, torch.full_like(e, -127), e).clamp(-127, 125 if bits == 4 else 121)
    y = x * ((127 - e) << 23).view(torch.float32)[:, :, None]
    if bits == 8:
        return y.round().clamp(-127, 127), e
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(((a / step).round() * step).clamp(max=6.0), y), e


def _powers(e):
    """2^e, e = -127 (a subnormal) included."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _quantised(x, bits):
    rows, k = x.shape
    codes, scales = _buffers(rows, k, bits)
    q, e = _round_blocks(x, bits)
    if bits == 8:
        codes.copy_(q.reshape(rows, -1))
    else:
        a = q.abs()
        c = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8) + (torch.signbit(q).to(torch.uint8) << 3)
        c = c.reshape(rows, -1, 2)
        codes.copy_(c[:, :, 0] + (c[:, :, 1] << 4))
    scales.copy_(e + 127)
    return codes, scales


def _values(codes, scales, dtype=torch.float32):
    """What codes and scales stand for, whole blocks."""
    rows, b = scales.shape
    if codes.dtype == torch.int8:
        q = codes.to(dtype)
    else:
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=dtype, device="cuda")
        q = grid[torch.stack([codes & 15, codes >> 4], 2).long()]
    return (q.reshape(rows, b, 32) * _powers(scales.int() - 127).to(dtype)[:, :, None]).reshape(rows, -1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)

    def activations(T, K, dtype):
        # one channel in 64 is eight times as wide as the others, as in the residual streams of language models
        wide = 1 + 7 * (torch.rand(K, device="cuda", generator=g) < 1 / 64).float()
        return (torch.randn(T, K, device="cuda", generator=g) * wide).to(dtype)

    op, dtype, T, K = case["op"], DTYPES[case["dtype"]], case["T"], case["K"]
    s = {"op": op}
    if op == "store":
        s["bits"] = case["bits"]
        s["X"] = normal(K, T, std=K ** -0.5, dtype=dtype).t() if case["x_t"] else activations(T, K, dtype)
        s["codes"], s["scales"] = _buffers(T, K, case["bits"])
        s["Y"] = torch.empty(T, K, device="cuda", dtype=dtype)
        return s
    N = case["N"]
    if op == "grad_weight":
        s["codes"], s["scales"] = _quantised(activations(T, K, dtype), case["bits"])
    else:
        s["codes"], s["scales"] = _quantised(normal(N, K, std=K ** -0.5, dtype=dtype), case.get("bits", 4))
    if op in ("linear", "matmul"):
        s["X"] = activations(T, K, dtype)
        if op == "matmul":
            s["X"] = _quantised(s["X"], 4)
        s["Y"] = torch.empty(T, N, device="cuda", dtype=dtype)
    else:
        s["dY"] = normal(T, N, std=N ** -0.5, dtype=dtype)
        s["out"] = torch.empty(*((T, K) if op == "grad_input" else (N, K)), device="cuda", dtype=dtype)
    return s


def _plain(s):
    op = s["op"]
    if op == "store":
        codes, e = _round_blocks(s["X"], s["bits"])
        return (codes * _powers(e)[:, :, None]).reshape(codes.shape[0], -1)[:, : s["X"].shape[1]].to(s["Y"].dtype)
    W = _values(s["codes"], s["scales"])
    if op == "linear":
        codes, e = _round_blocks(s["X"], 4)
        return ((codes * _powers(e)[:, :, None]).reshape(codes.shape[0], -1) @ W.t()).to(s["Y"].dtype)
    if op == "matmul":
        return (_values(*s["X"]) @ W.t()).to(s["Y"].dtype)
    k = s["out"].shape[1]
    if op == "grad_input":
        return (s["dY"].float() @ W[:, :k]).to(s["out"].dtype)
    return (s["dY"].float().t() @ W[:, :k]).to(s["out"].dtype)


def run(s):
    if not own:
        return _plain(s)
    import dense_fp32_gemm_06_gb300 as lib
    op = s["op"]
    if op == "store":
        lib.mx_quantize(s["X"], s["codes"], s["scales"])
        return lib.mx_dequantize(s["codes"], s["scales"], s["Y"])
    if op == "linear":
        return lib.mx4_linear(s["X"], s["codes"], s["scales"], s["Y"])
    if op == "matmul":
        return lib.mx4_matmul(*s["X"], s["codes"], s["scales"], s["Y"])
    if op == "grad_input":
        return lib.mx_grad_input(s["dY"], s["codes"], s["scales"], s["out"])
    return lib.mx_grad_weight(s["dY"], s["codes"], s["scales"], s["out"])


def _powers64(e):
    """2^e to the last bit (CUDA's exp2 need not be)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_rounded(x, bits):
    """A matrix rounded as its blocks are, in 64 bits and from the definition: the grid's nearest values, of two as near
    the one with the even code."""
    rows, k = x.shape
    x = torch.nn.functional.pad(x.double(), (0, -k % 32)).reshape(rows, -1, 32)
    top = x.abs().amax(2, keepdim=True)
    most, last = (6.0, 125) if bits == 4 else (127.0, 121)
    e = torch.full_like(top, -1000.0)
    # the least exponent with top <= most 2^e: first near, then put right by one (the logarithm may be off by a hair)
    near = torch.log2(torch.clamp(top, min=2.0 ** -140) / most).ceil()
    for step in (-1.0, 0.0, 1.0):
        fits = (top <= most * _powers64(near + step)) & (near + step >= -127)
        e = torch.where((e == -1000.0) & fits, near + step, e)
    scale = _powers64(e.clamp(-127, last))
    y = x / scale
    if bits == 8:
        return (y.round().clamp(-127, 127) * scale).reshape(rows, -1)[:, :k]
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    a = y.abs().clamp(max=6.0)
    above = torch.bucketize(a, grid).clamp(max=7)  # the first code whose value is at least a
    below = (above - 1).clamp(min=0)
    up, down = grid[above] - a, a - grid[below]
    code = torch.where((up < down) | ((up == down) & (above % 2 == 0)), above, below)
    return (torch.copysign(grid[code], y) * scale).reshape(rows, -1)[:, :k]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "store":
        return _exact_rounded(s["X"], case["bits"])
    W = _values(s["codes"], s["scales"], torch.float64)[:, : case["K"]]
    if case["op"] == "linear":
        return _exact_rounded(s["X"], 4) @ W.t()
    if case["op"] == "matmul":
        return _values(*s["X"], torch.float64)[:, : case["K"]] @ W.t()
    dY = s["dY"].double()
    return dY @ W if case["op"] == "grad_input" else dY.t() @ W


def work(case):
    e = {"f32": 4, "bf16": 2}[case["dtype"]]
    T, K = case["T"], case["K"]

    def held(rows, bits):
        return rows * (K * bits / 8 + _blocks(K))

    if case["op"] == "store":  # the codes and scales are written and read
        return {"bytes": 2 * e * T * K + 2 * held(T, case["bits"]), "flops": 5.0 * T * K}
    N = case["N"]
    flops = 2.0 * T * K * N
    if case["op"] == "linear":
        return {"bytes": e * T * K + held(N, 4) + e * T * N, "flops": flops}
    if case["op"] == "matmul":
        return {"bytes": held(T, 4) + held(N, 4) + e * T * N, "flops": flops}
    if case["op"] == "grad_input":
        return {"bytes": e * T * N + held(N, case["bits"]) + e * T * K, "flops": flops}
    return {"bytes": e * T * N + held(T, case["bits"]) + e * N * K, "flops": flops}
