"""Cases for measuring the adapter and loss operators: what each is called with, its plain form in elementary
torch operations, its definition in 64 bits and its work.

    lora_forward   Y = X W + s_a (X A_a^T) B_a, a = ids[t] the adapter of row t: many requests' low-rank adapters beside
                   one shared projection (X: T x K, W: K x N, A: L x R x K, B: L x R x N, H = s_a X A_a^T: T x R)
    lora_backward  its gradients: dX = dY W^T + U A_a with U = s_a dY B_a^T, dA_a = U^T X and dB_a = H^T dY over the
                   rows of adapter a
    distill_topk   per row w tau^2 KL(q || p), q the softmax of the teacher's top logits over tau and p that of all the
                   student's, and the gradient of the rows' sum by the student's logits
    policy_loss    per token the clipped policy loss -min(r A, clip(r) A), r = exp(lp - old), with a KL term
                   c (exp(ref - lp) - (ref - lp) - 1), and the gradient of the tokens' sum by the logits

`own` False runs the plain forms, True the library's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
CLIP_LOW, CLIP_HIGH, KL_COEF = 0.2, 0.28, 0.05


def listed():
    return [
        # one token of one request: the latency of a decoding step's projection
        dict(name="serve 1 token", op="lora_forward", dtype="bf16", T=1, K=4096, N=4096, L=16, R=16, reqs=1, w_t=True),
        # a decoding step of 64 requests, most with an adapter of their own
        dict(name="serve 64 tokens", op="lora_forward", dtype="bf16", T=64, K=4096, N=4096, L=64, R=16, reqs=64, w_t=True),
        # the repository's odd problem (1000 x 1500 x 777) as prompts of eight requests, in FP32
        dict(name="prompts 1000x1500x777", op="lora_forward", dtype="f32", T=1000, K=777, N=1500, L=8, R=8, reqs=8, w_t=False),
        # the repository's largest problem as a batch of prompts
        dict(name="prompts 8192^3", op="lora_forward", dtype="bf16", T=8192, K=8192, N=8192, L=16, R=32, reqs=24, w_t=True),
        # a small ragged fine-tuning batch of four adapters
        dict(name="grad 257x1500x1000", op="lora_backward", dtype="bf16", T=257, K=1000, N=1500, L=4, R=8, reqs=7, w_t=True),
        # the repository's worked size in FP32
        dict(name="grad 2048^3", op="lora_backward", dtype="f32", T=2048, K=2048, N=2048, L=4, R=16, reqs=8, w_t=False),
        # an ordinary fine-tuning step: two adapters, 8192 tokens
        dict(name="grad 8192x4096x4096", op="lora_backward", dtype="bf16", T=8192, K=4096, N=4096, L=2, R=64, reqs=16, w_t=True),
        # a short answer against a small vocabulary
        dict(name="distill 128x8192", op="distill_topk", dtype="f32", T=128, V=8192, top=32),
        # an ordinary distillation batch
        dict(name="distill 4096x32768", op="distill_topk", dtype="bf16", T=4096, V=32768, top=64),
        # one short answer
        dict(name="policy 32x32768", op="policy_loss", dtype="bf16", T=32, V=32768),
        # an odd vocabulary: rows that start at any 4-byte boundary
        dict(name="policy 1000x50021", op="policy_loss", dtype="f32", T=1000, V=50021),
        # many answers against a large vocabulary
        dict(name="policy 4096x131072", op="policy_loss", dtype="bf16", T=4096, V=131072),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _size(rng, low, high):
    """A size of the range: half of the time a multiple of 64, else as it falls."""
    n = _log_int(rng, low, high)
    return max(64, n // 64 * 64) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["lora_forward", "lora_forward", "lora_backward", "distill_topk", "policy_loss"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("lora"):
        T = _log_int(rng, 1, 8192) if op == "lora_forward" else _log_int(rng, 64, 8192)
        L = _log_int(rng, 1, 64)
        return dict(op=op, dtype=dtype, T=T, K=_size(rng, 256, 8192 if op == "lora_forward" else 4096), N=_size(rng, 256, 8192 if op == "lora_forward" else 4096),
                    L=L, R=rng.choice([4, 8, 16, 32, 64, _log_int(rng, 1, 64)]), reqs=T if rng.random() < 0.3 else min(T, _log_int(rng, 1, 64)), w_t=rng.random() < 0.5)
    V = _size(rng, 2048, 131072)
    T = min(_log_int(rng, 16, 8192), 4096 * 131072 // V, 8192)
    c = dict(op=op, dtype=dtype, T=T if dtype == "bf16" else max(1, T // 2), V=V)
    if op == "distill_topk":
        c["top"] = rng.choice([8, 20, 64, _log_int(rng, 1, 256)])
    return c


def _draws(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)

    def whole(low, high, *shape):
        return torch.randint(low, high, shape, device="cuda", generator=g, dtype=torch.int32)

    def share(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    return normal, whole, share


def prepare(case, seed):
    normal, whole, share = _draws(case, seed)
    dtype, s = DTYPES[case["dtype"]], dict(case)
    T = case["T"]
    if case["op"].startswith("lora"):
        K, N, L, R, reqs = (case[k] for k in ("K", "N", "L", "R", "reqs"))
        # the rows of a request lie together; where each starts is drawn, its adapter too, and one request in eight has none
        if reqs == T:
            req = torch.arange(T, device="cuda")
        else:
            cuts = torch.sort(torch.randperm(T - 1, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))[: reqs - 1] + 1).values if T > 1 else whole(0, 1, 0)
            req = torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)
        adapter = torch.where((share(reqs) < 0.125) & (torch.arange(reqs, device="cuda") > 0), torch.full((reqs,), -1, dtype=torch.int32, device="cuda"), whole(0, L, reqs))
        s["ids"] = adapter[req].contiguous()
        s["X"] = normal(T, K, dtype=dtype)
        s["W"] = normal(N, K, std=K ** -0.5, dtype=dtype).t() if case["w_t"] else normal(K, N, std=K ** -0.5, dtype=dtype)
        s["A"] = normal(L, R, K, std=K ** -0.5, dtype=dtype)
        s["B"] = normal(L, R, N, std=0.05, dtype=dtype)
        s["scale"] = 0.5 + 1.5 * share(L)
        if case["op"] == "lora_forward":
            s["Y"] = torch.empty(T, N, device="cuda", dtype=dtype)
        else:
            s["dY"] = normal(T, N, std=N ** -0.5, dtype=dtype)
            s["H"] = normal(T, R) * (s["ids"] >= 0)[:, None] * s["scale"][s["ids"].clamp(min=0).long()][:, None]
            s["dX"], s["dA"], s["dB"] = torch.empty_like(s["X"]), torch.empty_like(s["A"]), torch.empty_like(s["B"])
        return s
    V = case["V"]
    s["logits"] = normal(T, V, std=2.0, dtype=dtype)
    s["weight"] = (share(T) < 0.9).float() / T  # one row in ten is masked
    s["grad"], s["loss"] = torch.empty_like(s["logits"]), torch.empty(T, device="cuda")
    if case["op"] == "distill_topk":
        top = case["top"]
        # distinct places: a start and a step that has no divisor in common with V, and a teacher near the student there
        step = 7919 if V % 7919 else 7907
        s["index"] = ((whole(0, V, T, 1).long() + torch.arange(top, device="cuda") * step) % V).int()
        s["teacher"] = s["logits"].gather(1, s["index"].long()).float() + normal(T, top)
        s["temperature"] = 2.0
    else:
        s["labels"] = whole(0, V, T)
        lp = s["logits"].gather(1, s["labels"].long()[:, None])[:, 0].float() - _rows_lse(s["logits"])
        s["old"] = lp + normal(T, std=0.2)
        s["ref"] = lp + normal(T, std=0.3)
        s["advantage"] = normal(T)
        s["logp"] = torch.empty(T, device="cuda")
    return s


def _rows_lse(x):
    return torch.cat([torch.logsumexp(c.float(), 1) for c in x.split(1024)])


def _plain_lora(s):
    """(X, W, A, B as 32-bit matrices, the mask of each row's adapter times its scale)."""
    L, R = s["A"].shape[:2]
    of = (s["ids"][:, None] == torch.arange(L, device="cuda", dtype=torch.int32)).float()
    return s["X"].float(), s["W"].float(), s["A"].float().reshape(L * R, -1), s["B"].float().reshape(L * R, -1), of


def _plain_forward(s):
    X, W, A, B, of = _plain_lora(s)
    L, R = s["A"].shape[:2]
    H = (X @ A.t()).reshape(-1, L, R) * (of * s["scale"])[:, :, None]
    return (X @ W + H.reshape(-1, L * R) @ B).to(s["Y"].dtype)


def _plain_backward(s):
    X, W, A, B, of = _plain_lora(s)
    L, R = s["A"].shape[:2]
    dY = s["dY"].float()
    U = ((dY @ B.t()).reshape(-1, L, R) * (of * s["scale"])[:, :, None]).reshape(-1, L * R)
    H = (s["H"][:, None, :] * of[:, :, None]).reshape(-1, L * R)
    dX = dY @ W.t() + U @ A
    return {"dX": dX.to(s["X"].dtype), "dA": (U.t() @ X).to(s["A"].dtype).reshape(s["A"].shape), "dB": (H.t() @ dY).to(s["B"].dtype).reshape(s["B"].shape)}


def _plain_distill(s):
    tau, w = s["temperature"], s["weight"]
    z = s["logits"].float() / tau
    z = z - z.amax(1, keepdim=True)
    e = z.exp()
    total = e.sum(1, keepdim=True)
    at = s["index"].long()
    t = s["teacher"] / tau
    t = t - t.amax(1, keepdim=True)
    q = t.exp()
    n = q.sum(1, keepdim=True)
    q = q / n
    loss = w * tau * tau * (q * ((t - n.log()) - (z.gather(1, at) - total.log()))).sum(1)
    p = e / total
    p.scatter_add_(1, at, -q)
    return {"loss": loss, "grad": (p * (w * tau)[:, None]).to(s["grad"].dtype)}


def _plain_policy(s):
    w, adv = s["weight"], s["advantage"]
    z = s["logits"].float()
    z = z - z.amax(1, keepdim=True)
    e = z.exp()
    total = e.sum(1, keepdim=True)
    at = s["labels"].long()[:, None]
    lp = (z.gather(1, at) - total.log())[:, 0]
    r = (lp - s["old"]).exp()
    a, b = r * adv, r.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * adv
    k = (s["ref"] - lp).exp()
    loss = w * (-torch.minimum(a, b) + KL_COEF * (k - (s["ref"] - lp) - 1))
    by_lp = w * (torch.where(a <= b, -a, torch.zeros_like(a)) + KL_COEF * (1 - k))
    g = (e / total) * -by_lp[:, None]
    g.scatter_add_(1, at, by_lp[:, None])
    return {"loss": loss, "logp": lp, "grad": g.to(s["grad"].dtype)}


def run(s):
    op = s["op"]
    if not own:
        return {"lora_forward": _plain_forward, "lora_backward": _plain_backward, "distill_topk": _plain_distill, "policy_loss": _plain_policy}[op](s)
    import dense_fp32_gemm_06_gb300 as lib
    if op == "lora_forward":
        return lib.lora_forward(s["X"], s["W"], s["A"], s["B"], s["ids"], s["Y"], s["scale"])
    if op == "lora_backward":
        lib.lora_backward(s["dY"], s["X"], s["W"], s["A"], s["B"], s["ids"], s["H"], s["dX"], s["dA"], s["dB"], s["scale"])
        return {"dX": s["dX"], "dA": s["dA"], "dB": s["dB"]}
    if op == "distill_topk":
        lib.distill_topk(s["logits"], s["teacher"], s["index"], s["loss"], s["grad"], weight=s["weight"], temperature=s["temperature"])
        return {"loss": s["loss"], "grad": s["grad"]}
    lib.policy_loss(s["logits"], s["labels"], s["old"], s["advantage"], s["loss"], s["grad"], ref=s["ref"], weight=s["weight"],
                    clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl_coef=KL_COEF, logp=s["logp"])
    return {"loss": s["loss"], "logp": s["logp"], "grad": s["grad"]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("lora"):
        X, W = s["X"].double(), s["W"].double()
        back = case["op"] == "lora_backward"
        if not back:
            Y = X @ W
        else:
            dY, H = s["dY"].double(), s["H"].double()
            dX = dY @ W.t()
            dA, dB = torch.zeros_like(s["A"], dtype=torch.float64), torch.zeros_like(s["B"], dtype=torch.float64)
        for a in range(case["L"]):
            rows = torch.nonzero(s["ids"] == a)[:, 0]
            if rows.numel() == 0:
                continue
            A, B, c = s["A"][a].double(), s["B"][a].double(), float(s["scale"][a])
            if not back:
                Y[rows] += c * (X[rows] @ A.t()) @ B
            else:
                U = c * (dY[rows] @ B.t())
                dX[rows] += U @ A
                dA[a], dB[a] = U.t() @ X[rows], H[rows].t() @ dY[rows]
        return {"dX": dX, "dA": dA, "dB": dB} if back else Y
    losses, lps, grads = [], [], []
    for c in range(0, case["T"], 512):
        part = slice(c, c + 512)
        z, w = s["logits"][part].double(), s["weight"][part].double()
        rows = torch.arange(z.shape[0], device="cuda")
        if case["op"] == "distill_topk":
            tau = s["temperature"]
            logp = torch.log_softmax(z / tau, 1)
            logq = torch.log_softmax(s["teacher"][part].double() / tau, 1)
            at = s["index"][part].long()
            losses.append(w * tau ** 2 * (logq.exp() * (logq - logp[rows[:, None], at])).sum(1))
            g = logp.exp()
            g[rows[:, None], at] -= logq.exp()  # the places of a row are distinct
            grads.append((g * (tau * w)[:, None]))
        else:
            logp = torch.log_softmax(z, 1)
            at = s["labels"][part].long()
            lp, adv = logp[rows, at], s["advantage"][part].double()
            old, ref = s["old"][part].double(), s["ref"][part].double()
            r, k = (lp - old).exp(), (ref - lp).exp()
            a = r * adv
            b = torch.clamp(r, 1 - CLIP_LOW, 1 + CLIP_HIGH) * adv
            losses.append(w * (KL_COEF * (k - (ref - lp) - 1) - torch.minimum(a, b)))
            d = w * (KL_COEF * (1 - k) - a * (a <= b))
            g = logp.exp() * -d[:, None]
            g[rows, at] += d
            lps.append(lp)
            grads.append(g)
    out = {"loss": torch.cat(losses), "grad": torch.cat(grads)}
    if lps:
        out["logp"] = torch.cat(lps)
    return out


def work(case):
    e = {"f32": 4, "bf16": 2}[case["dtype"]]
    T = case["T"]
    if case["op"].startswith("lora"):
        K, N, R = case["K"], case["N"], case["R"]
        used = min(case["L"], case["reqs"])
        b = e * (T * K + K * N + T * N + used * R * (K + N)) + 4 * T + 4 * case["L"]
        f = 2.0 * T * K * N + 2.0 * T * R * (K + N)
        if case["op"] == "lora_backward":  # H too, and dX, dA and dB beside what the forward pass moves
            b += 4 * T * R + e * (T * K + case["L"] * R * (K + N))
            f += 2.0 * T * R * (K + N)
        return {"bytes": b, "flops": f}
    b = 2 * e * T * case["V"] + 8 * T
    if case["op"] == "distill_topk":
        return {"bytes": b + 8 * T * case["top"], "flops": 5.0 * T * case["V"]}
    return {"bytes": b + 20 * T, "flops": 5.0 * T * case["V"]}
