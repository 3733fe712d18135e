"""Plain 64-bit forms of the adapter and loss operators, with the bounds that
the FP32 arithmetic of the kernels has to meet.  u = 2^-24 is FP32's unit
roundoff; a chain of h FP32 additions is within h u (1 + tiny) of its sum of
magnitudes."""
import numpy as np
import torch

U32 = 2.0 ** -24
OUT_U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def gamma(h):
    return 1.01 * h * U32


def product_bound(depth, dtype):
    """Relative to sum |a||b|: the library's own bound for FP32 products; for
    16-bit ones (exact products) the tensor core rounds its FP32 sum towards
    zero once per 16 of the depth, at most 2^-22 of it."""
    return 1e-5 if dtype == torch.float32 else (depth / 16 + 4) * 2.0 ** -22


def chain(depth):
    """Longest chain of FP32 additions of a skinny product: a thread takes
    every 32nd value at least, then trees over lanes and warps; or 16 at a
    time on the tensor core, whose roundings are up to four u."""
    return depth / 4 + 48


def lora_parts(X, W, A, B, ids, scale):
    """Everything in float64 on the CPU; row t's adapter as a loop over adapters."""
    X, W, A, B = (v.detach().cpu().double() for v in (X, W, A, B))
    ids = ids.cpu().long()
    s = scale.cpu().double() if scale is not None else torch.ones(A.shape[0], dtype=torch.float64)
    return X, W, A, B, ids, s


def lora_forward(X, W, A, B, ids, scale=None, dtype=torch.float32):
    """(Y, bound of |Y - kernel|, H, bound of H)."""
    X, W, A, B, ids, s = lora_parts(X, W, A, B, ids, scale)
    T, K = X.shape
    R = A.shape[1]
    Y, E = X @ W, X.abs() @ W.abs()
    bound = product_bound(K + R, dtype) * E
    H, HB = torch.zeros(T, R, dtype=torch.float64), torch.zeros(T, R, dtype=torch.float64)
    for a in range(A.shape[0]):
        rows = torch.nonzero(ids == a)[:, 0]
        if rows.numel() == 0:
            continue
        H[rows] = s[a] * (X[rows] @ A[a].t())
        HB[rows] = gamma(chain(K)) * abs(s[a]) * (X[rows].abs() @ A[a].abs().t())
        Y[rows] += H[rows] @ B[a]
        part = (gamma(R + 8) + (OUT_U[torch.bfloat16] if dtype != torch.float32 else 0) + product_bound(R, dtype)) * (H[rows].abs() @ B[a].abs())
        bound[rows] += part + HB[rows] @ B[a].abs() * 1.01
    return Y, bound + OUT_U[dtype] * (Y.abs() + bound) + 1e-30, H, HB + 1e-30


def lora_backward(dY, X, W, A, B, ids, H, scale=None, dtype=torch.float32):
    """{name: (gradient, bound)}."""
    dY = dY.detach().cpu().double()
    H = H.detach().cpu().double()
    ids_ = ids
    dX, bx, U, UB = lora_forward(dY, W.t(), B, A, ids, scale, dtype)   # the same two products, with the adapters' stacks in turn
    X, W, A, B, ids, s = lora_parts(X, W, A, B, ids_, scale)
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    ba, bb = torch.zeros_like(A), torch.zeros_like(B)
    for a in range(A.shape[0]):
        rows = torch.nonzero(ids == a)[:, 0]
        if rows.numel() == 0:
            continue
        rel = gamma(chain(rows.numel())) + (OUT_U[torch.bfloat16] if dtype != torch.float32 else 0)
        dA[a] = U[rows].t() @ X[rows]
        ba[a] = rel * (U[rows].abs().t() @ X[rows].abs()) + UB[rows].t() @ X[rows].abs() * 1.01
        dB[a] = H[rows].t() @ dY[rows]
        bb[a] = rel * (H[rows].abs().t() @ dY[rows].abs())
    o = OUT_U[dtype]
    return {"dX": (dX, bx), "dA": (dA, ba + o * (dA.abs() + ba) + 1e-30), "dB": (dB, bb + o * (dB.abs() + bb) + 1e-30)}


def _softmax(z, c):
    """(p, log p, bound of p's relative error, bound of log S's error) of softmax(z / tau), c = 1 / tau."""
    m = z.max(1, keepdim=True).values
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    x = (z - m) * c
    e = x.exp()
    S = e.sum(1, keepdim=True)
    p = e / S
    ax = torch.where(torch.isinf(x), torch.zeros_like(x), x.abs())
    # two roundings of the exponent, exp2 within 2^-21, sums of at most 96 in a chain
    d = 2.0 ** -22 * ax + 2.0 ** -21 + gamma(96)
    return p, x - S.log(), d, (p * d).sum(1, keepdim=True)


def distill(z, teacher, index, weight, tau, dtype):
    """(loss, bound, grad, bound)."""
    z, t = z.detach().cpu().double(), teacher.cpu().double()
    T, V = z.shape
    at = index.cpu().long()
    w = weight.cpu().double() if weight is not None else torch.ones(T, dtype=torch.float64)
    ok = (at >= 0) & (at < V) & ~torch.isneginf(t)
    live = ok.any(1) & (w != 0) & ~torch.isneginf(z).all(1)
    zz = torch.where(live[:, None], z, torch.zeros_like(z))
    tt = torch.where(ok, t, torch.full_like(t, -float("inf")))
    tt = torch.where(live[:, None], tt, torch.zeros_like(tt))
    at = torch.where(ok, at, torch.zeros_like(at))
    p, lp, d, dS = _softmax(zz, 1 / tau)
    q, lq, dt, dtS = _softmax(tt, 1 / tau)
    lpj = lp.gather(1, at)
    term = torch.where(q > 0, q * (lq - lpj), torch.zeros_like(q))
    loss = w * tau * tau * term.sum(1)
    size = torch.where(q > 0, q * (lq.abs() + lpj.abs() + 1) , torch.zeros_like(q)).sum(1)
    per = torch.where(q > 0, q * (dt + dtS) * ((lq - lpj).abs()), torch.zeros_like(q)).sum(1)
    lb = (w * tau * tau).abs() * (dS[:, 0] + dtS[:, 0] + (2.0 ** -21 + gamma(48)) * size + per)
    Q = torch.zeros_like(p).scatter_add_(1, at, torch.where(ok, q, torch.zeros_like(q)))
    QB = torch.zeros_like(p).scatter_add_(1, at, torch.where(ok, q * (dt + dtS + gamma(16)), torch.zeros_like(q)))
    g = (w * tau)[:, None] * (p - Q)
    gb = (w * tau).abs()[:, None] * (p * (d + dS + 2.0 ** -21) + QB)
    dead = ~live
    loss[dead], lb[dead], g[dead], gb[dead] = 0, 0, 0, 0
    return loss, lb + 1e-30, g, gb + OUT_U[dtype] * (g.abs() + gb) + tiny(dtype)


def tiny(dtype):
    """The least value the type (and exp2 without subnormals) tells from zero."""
    return {torch.float32: 2.0 ** -125, torch.bfloat16: 2.0 ** -125, torch.float16: 2.0 ** -24}[dtype]


def policy(z, labels, old, adv, ref, weight, lo, hi, kl, dtype):
    """(loss, bound, lp, bound, grad, bound)."""
    z = z.detach().cpu().double()
    T, V = z.shape
    y = labels.cpu().long()
    old, adv = old.cpu().double(), adv.cpu().double()
    w = weight.cpu().double() if weight is not None else torch.ones(T, dtype=torch.float64)
    ok = (y >= 0) & (y < V)
    some = ~torch.isneginf(z).all(1)
    seen = ok & some
    zz = torch.where(seen[:, None], z, torch.zeros_like(z))
    at = torch.where(ok, y, torch.zeros_like(y))[:, None]
    p, logp, d, dS = _softmax(zz, 1.0)
    lp = logp.gather(1, at)[:, 0]
    dlp = dS[:, 0] + 2.0 ** -22 * (torch.where(torch.isinf(lp), torch.zeros_like(lp), lp.abs()) + logp.logsumexp(1).abs() + 30)
    r = (lp - old).exp()
    dr = r * (dlp + 2.0 ** -21)
    a, b = r * adv, r.clamp(1 - lo, 1 + hi) * adv
    loss = -torch.minimum(a, b)
    lb = adv.abs() * (dr + 2.0 ** -22 * r)
    g = torch.where(a <= b, -a, torch.zeros_like(a))
    gb_ = lb.clone()
    if kl != 0:
        x = ref.cpu().double() - lp
        k = x.exp()
        loss = loss + kl * (k - x - 1)
        g = g + kl * (1 - k)
        e = kl * (k * (dlp + 2.0 ** -21) + dlp + 2.0 ** -22 * (k + x.abs() + 1))
        lb, gb_ = lb + e, gb_ + e
    loss, g, lb, gb_ = loss * w, g * w, lb * w.abs() + 2.0 ** -22 * (loss * w).abs(), gb_ * w.abs() + 2.0 ** -22 * (g * w).abs()
    Y = torch.zeros_like(p).scatter_(1, at, 1.0)
    G = g[:, None] * (Y - p)
    GB = gb_[:, None] * (Y + p) + g.abs()[:, None] * (p * (d + dS + 2.0 ** -21) + 2.0 ** -23 * Y)
    live = seen & (w != 0)
    for v in (loss, lb, G, GB):
        v[~live] = 0
    lp = torch.where(ok, torch.where(some, lp, torch.full_like(lp, -float("inf"))), torch.zeros_like(lp))
    return loss, lb + 1e-30, lp, dlp + 1e-30, G, GB + OUT_U[dtype] * (G.abs() + GB) + tiny(dtype)


def close(got, want, bound, what=""):
    """got within the bound of want everywhere (equal where want is infinite)."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fin), f"{what}: {int((torch.isfinite(got) != fin).sum())} values are not finite where they should be, or the other way round"
    assert torch.equal(got[~fin], want[~fin]), what
    if fin.any():
        ratio = ((got - want).abs() / bound)[fin]
        worst = float(ratio.max())
        assert worst <= 1.0, f"{what}: |got - want| / bound = {worst:.3g} at {np.unravel_index(int(torch.where(fin, (got - want).abs() / bound, torch.zeros_like(got)).argmax()), got.shape)}"
