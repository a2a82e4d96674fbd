"""The output end of a model whose logits the losses take: from hidden states to log-probabilities.

Three operators.  The root-mean-square norm with the residual's addition: in the stream's own type,
with its gradient, or in 8 bits with a scale for each token (and the 8-bit form without a norm, for
other activations).  The product of 8-bit activations and 8-bit weights with a scale for each token
and each channel, which makes the logits.  The log-probabilities of given tokens with the entropy
and the top alternatives of each row, and the gradient of log-probability and entropy.  ``own``
selects the library's kernels; the plain forms are elementary torch operations in 32 bits, in 64
where a value is next to a rounding's border or a long sum is formed.  ``exact`` states each
operator again in 64 bits, its gradients by automatic differentiation.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-6
MOST_PRODUCTS = 4096 * 131072 * 4096   # of the largest listed product
MOST_LOGITS = 4096 * 131072 * 2        # bytes of logits in the largest listed rows


def listed():
    return [
        # the final norm of one step of decoding in four streams: only the launch costs
        dict(name="norm int8 4x4096", op="norm", mode="int8", type="bf16", T=4, d=4096, weight=True),
        # the final norm of a scored batch
        dict(name="norm int8 16384x5120", op="norm", mode="int8", type="bf16", T=16384, d=5120,
             weight=True),
        # other activations (behind a gate) on their way into an 8-bit product
        dict(name="quantize 2000x14336", op="norm", mode="quantize", type="bf16", T=2000, d=14336,
             weight=False),
        # one norm of a training step, forward and backward, in a stream of residuals
        dict(name="norm train 8192x4096", op="norm", mode="train", type="bf16", T=8192, d=4096,
             weight=True),
        # 32-bit training of a small model, rows of an odd length
        dict(name="norm train 777x2501 f32", op="norm", mode="train", type="f32", T=777, d=2501,
             weight=True),
        # the head for one new token in each of four streams: its weights are read once
        dict(name="linear 4x4096 to 131072", op="linear", type="bf16", T=4, K=4096, N=131072,
             bias=False),
        # a short sequence, odd sizes throughout, 32-bit logits
        dict(name="linear 333x1500 to 50001 f32", op="linear", type="f32", T=333, K=1500, N=50001,
             bias=True),
        # the head over a scored micro-batch
        dict(name="linear 4096x4096 to 131072", op="linear", type="bf16", T=4096, K=4096, N=131072,
             bias=False),
        # one new token in each of four streams, with its 20 best alternatives
        dict(name="scores 4x131072 k20 f32", op="scores", type="f32", T=4, V=131072, K=20, masked=0,
             labels=True, backward=False, scale=0.8),
        # a teacher's pass over a micro-batch: its 64 best tokens for distillation
        dict(name="scores 4096x131072 k64", op="scores", type="bf16", T=4096, V=131072, K=64,
             masked=512, labels=True, backward=False, scale=1.0),
        # a short prompt's rows, alternatives without labels, rows of an odd length
        dict(name="scores 500x50001 k5", op="scores", type="bf16", T=500, V=50001, K=5, masked=0,
             labels=False, backward=False, scale=1.0),
        # a policy's training step with an entropy bonus, 32-bit logits
        dict(name="scores train 3000x100003 f32", op="scores", type="f32", T=3000, V=100003, K=0,
             masked=0, labels=True, backward=True, scale=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm", "linear", "scores", "scores"))
    kind = rng.choice(("bf16", "f32"))
    if op == "norm":
        d = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            d = max(64, d - d % 64)
        mode = rng.choice(("int8", "quantize", "train"))
        T = _log(rng, 1, min(65536, 16384 * 5120 // d))
        return dict(op=op, mode=mode, type=kind, T=T, d=d,
                    weight=mode != "quantize" and rng.random() < 0.9)
    if op == "linear":
        K = _log(rng, 64, 14336)
        if rng.random() < 0.6:
            K = max(64, K - K % 64)
        N = _log(rng, 64, 131072)
        T = _log(rng, 1, max(1, min(8192, MOST_PRODUCTS // (K * N))))
        return dict(op=op, type=kind, T=T, K=K, N=N, bias=rng.random() < 0.3)
    V = _log(rng, 200, 160000)
    if rng.random() < 0.5:
        V = max(64, V - V % 64)
    backward = rng.random() < 0.4
    T = _log(rng, 1, min(8192, max(1, MOST_LOGITS // (V * BYTES[kind]) // (2 if backward else 1))))
    return dict(op=op, type=kind, T=T, V=V, K=0 if backward else _log(rng, 1, 128),
                masked=rng.choice((0, V // 50)), labels=backward or rng.random() < 0.7,
                backward=backward, scale=round(rng.uniform(0.5, 1.5), 3))


def _eight(x):
    """Rows in 8 bits, kept as a program keeps them for the product: each at a multiple of 16 bytes."""
    rows, K = x.shape
    scale = x.abs().amax(1) / 127.0
    q = torch.zeros(rows, -(-K // 16) * 16, dtype=torch.int8, device=x.device)
    q[:, :K] = torch.round(x / scale[:, None]).to(torch.int8)
    return q[:, :K], scale


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    T = case["T"]
    s = dict(case=case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        s["x"], s["xscale"] = _eight(normal(T, K) * (1.0 + 0.5 * normal(K).abs()))
        s["w"], s["wscale"] = _eight(normal(N, K) * (0.02 + 0.01 * normal(N).abs()[:, None]))
        s["bias"] = 0.1 * normal(N) if case["bias"] else None
        return s
    dtype = TYPES[case["type"]]
    if case["op"] == "norm":
        d = case["d"]
        # a residual stream has a few channels far larger than the others
        loud = torch.exp(0.5 * normal(d)) + 20.0 * (torch.rand(d, generator=g, device=dev) < 0.002)
        s["x"] = normal(T, d).to(dtype)
        s["residual"] = (normal(T, d) * loud).to(dtype)
        s["weight"] = (1.0 + 0.2 * normal(d)).to(dtype) if case["weight"] else None
        if case["mode"] == "train":
            s["dy"] = (normal(T, d) / T).to(dtype)
            s["dh"] = (normal(T, d) / T).to(dtype)
        return s
    # a model's logits: a broad floor, and a label that is often, not always, the likely one
    V = case["V"]
    z = normal(T, V).mul_(2.0)
    labels = torch.randint(0, V - case["masked"], (T,), generator=g, device=dev)
    z[torch.arange(T, device=dev), labels] += 4.0 + 4.0 * normal(T)
    if case["masked"]:
        z[:, V - case["masked"]:] = -math.inf       # columns that pad the vocabulary
    s["logits"] = z.to(dtype)
    s["labels"] = None
    if case["labels"]:
        s["labels"] = torch.where(torch.rand(T, generator=g, device=dev) < 0.1, -1, labels).int()
    if case["backward"]:
        s["grad"] = normal(T) / T
        s["grad_entropy"] = -0.01 * (0.5 + torch.rand(T, generator=g, device=dev)) / T
    return s


def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return PLAIN[case["op"]](case, state)


def _own(case, s):
    import sinkhorn_point_cloud_amd as sk
    if case["op"] == "linear":
        return sk.int8_linear(s["x"], s["xscale"], s["w"], s["wscale"], bias=s["bias"],
                              dtype=TYPES[case["type"]])
    if case["op"] == "norm":
        if case["mode"] == "quantize":
            q, scale = sk.quantize_int8(s["x"])
            return q * scale[:, None], scale
        if case["mode"] == "int8":
            q, scale, h = sk.rms_norm_int8(s["x"], s["weight"], s["residual"], eps=EPS)
            return q * scale[:, None], scale, h
        y, h = sk.rms_norm(s["x"], s["weight"], s["residual"], eps=EPS)
        dx, dw = sk.rms_norm_backward(s["dy"], h, s["weight"], dh=s["dh"], eps=EPS)
        return (y, h, dx) if dw is None else (y, h, dx, dw)
    out = sk.token_scores(s["logits"], s["labels"], top=case["K"], scale=case["scale"])
    out = tuple(o for o in out if o is not None)
    if not case["backward"]:
        return out
    return out + (sk.token_scores_backward(s["logits"], s["labels"], s["grad"], s["grad_entropy"],
                                           scale=case["scale"]),)


# ------------------------------------------------------------------ plain forms

def _plain_linear(case, s):
    out = (s["x"].float() @ s["w"].float().T) * s["xscale"][:, None] * s["wscale"]
    if s["bias"] is not None:
        out = out + s["bias"]
    return out.to(TYPES[case["type"]])


def _plain_eight(p, r):
    """Rows p (64 bits) times r [T, 1] in 8 bits: the values they stand for, and the scales."""
    most = p.abs().amax(1, keepdim=True)
    q = torch.round(127.0 * p / most)           # ties are common: half of the largest is one
    scale = (most * r / 127.0).float()
    return q.float() * scale, scale[:, 0]


def _plain_norm(case, s):
    x = s["x"]
    if case["mode"] == "quantize":
        return _plain_eight(x.double(), 1.0)
    d = case["d"]
    h = (x.float() + s["residual"].float()).to(x.dtype)      # the stream that goes on
    f = h.float()
    r = torch.rsqrt((f * f).sum(1, keepdim=True, dtype=torch.float64) / d + EPS)
    w = 1.0 if s["weight"] is None else s["weight"].float()
    if case["mode"] == "int8":
        p = h.double() if s["weight"] is None else h.double() * s["weight"].double()
        return _plain_eight(p, r) + (h,)
    r = r.float()
    n = f * r
    y = (n * w).to(x.dtype)
    dy = s["dy"].float()
    u = dy * w
    mean = (u * n).sum(1, keepdim=True, dtype=torch.float64) / d
    dx = (r * (u - n * mean.float()) + s["dh"].float()).to(x.dtype)
    if s["weight"] is None:
        return y, h, dx
    return y, h, dx, (dy * n).sum(0, dtype=torch.float64).float()


def _keys(z):
    """64-bit keys in the order of the values, among equal ones the lower index above the higher."""
    bits = (z.float() + 0.0).view(torch.int32)               # -0 counts as 0
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    return (order << 32) + torch.arange(z.shape[1] - 1, -1, -1, device=z.device)


def _plain_scores(case, s):
    z, scale, labels = s["logits"], case["scale"], s["labels"]
    x = z.float()
    top = x.amax(1, keepdim=True)
    gap = (top - x) * scale
    e = torch.exp(-gap)
    S = e.sum(1, dtype=torch.float64)
    gap = torch.where(e > 0, gap, 0.0)                       # no part of what has no probability
    D = (e * gap).sum(1, dtype=torch.float64) / S
    lse = top[:, 0].double() * scale + torch.log(S)
    used = torch.ones_like(S, dtype=torch.bool) if labels is None else labels >= 0
    out = []
    if labels is not None:
        at = labels.long().clamp(min=0)[:, None]
        logp = x.gather(1, at)[:, 0].double() * scale - lse
        out.append(torch.where(used, logp, 0.0).float())
    out += [torch.where(used, lse, 0.0).float(), torch.where(used, torch.log(S) + D, 0.0).float()]
    if case["K"]:
        best = z.shape[1] - 1 - (_keys(z).topk(min(case["K"], z.shape[1]), dim=1).values
                                 & 0xFFFFFFFF)
        best = torch.nn.functional.pad(best, (0, case["K"] - best.shape[1]))
        found = x.gather(1, best)
        listed_ = (used[:, None] & (found > -math.inf)
                   & (torch.arange(case["K"], device=z.device) < z.shape[1]))
        out += [torch.where(listed_, best, -1).int(),
                torch.where(listed_, found.double() * scale - lse[:, None], -math.inf).float()]
    if case["backward"]:
        a = torch.where(used, -(s["grad"].double() + s["grad_entropy"].double() * D) * scale / S, 0.0)
        b = torch.where(used, s["grad_entropy"].double() * scale / S, 0.0)
        grad = e * (a.float()[:, None] + b.float()[:, None] * gap)
        grad.scatter_add_(1, at, torch.where(used, s["grad"] * scale, 0.0)[:, None])
        out.append(grad.to(z.dtype))
    return tuple(out)


PLAIN = dict(norm=_plain_norm, linear=_plain_linear, scores=_plain_scores)


# ------------------------------------------------------------------ work and definitions

def work(case):
    T = case["T"]
    b = BYTES[case["type"]]
    if case["op"] == "linear":
        K, N = case["K"], case["N"]
        return {"bytes": T * K + N * K + T * N * b + 4.0 * (T + N) + (4.0 * N if case["bias"] else 0.0),
                "flops": 2.0 * T * N * K}
    if case["op"] == "norm":
        row = T * case["d"]
        if case["mode"] == "quantize":
            return {"bytes": row * (b + 1.0) + 4.0 * T, "flops": 3.0 * row}
        weight = case["d"] * b if case["weight"] else 0.0
        if case["mode"] == "int8":
            return {"bytes": row * (3.0 * b + 1.0) + 4.0 * T + weight, "flops": 6.0 * row}
        return {"bytes": row * 8.0 * b + 2.0 * weight + (4.0 * case["d"] if case["weight"] else 0.0),
                "flops": 16.0 * row}
    used = 0.9 if case["labels"] else 1.0
    rows = T * case["V"] * b
    return {"bytes": used * rows + (rows if case["backward"] else 0.0) + T * (16.0 + 8.0 * case["K"]),
            "flops": (14.0 if case["backward"] else 8.0) * used * T * case["V"]}


def exact(case, seed):
    s = prepare(case, seed)
    T = case["T"]
    if case["op"] == "linear":
        x = s["x"].double() * s["xscale"].double()[:, None]
        out = torch.matmul(x, s["w"].double().t()).mul_(s["wscale"].double())
        return out if s["bias"] is None else out.add_(s["bias"].double())
    if case["op"] == "norm":
        if case["mode"] == "quantize":
            y = s["x"].double()
            most = torch.linalg.vector_norm(y, math.inf, 1)
            return torch.round(y * 127 / most[:, None]) * (most / 127)[:, None], most / 127
        h = (s["x"].double() + s["residual"].double()).to(s["x"].dtype)
        stream = h.double().requires_grad_()
        weight = torch.ones(case["d"], dtype=torch.float64, device=h.device) \
            if s["weight"] is None else s["weight"].double()
        weight.requires_grad_()
        y = stream / (stream.square().mean(1, keepdim=True) + EPS).sqrt() * weight
        if case["mode"] == "int8":
            p = h.double() * weight.detach()                 # the norm's factor cancels within a row
            q = torch.round(127 * p / torch.linalg.vector_norm(p, math.inf, 1, keepdim=True))
            step = torch.linalg.vector_norm(y.detach(), math.inf, 1) / 127
            return q * step[:, None], step, h.double()
        total = (y * s["dy"].double()).sum() + (stream * s["dh"].double()).sum()
        dx, dw = torch.autograd.grad(total, (stream, weight))
        out = (y.detach(), h.double(), dx)
        return out if s["weight"] is None else out + (dw,)
    labels, K = s["labels"], case["K"]
    z = s["logits"].double().requires_grad_(case["backward"])
    used = torch.ones(T, dtype=torch.bool, device=z.device) if labels is None else labels >= 0
    logq = torch.log_softmax(z * case["scale"], 1)
    sound = torch.isfinite(logq.detach())
    q = logq.exp()
    entropy = -torch.where(sound, q * torch.where(sound, logq, 0.0), 0.0).sum(1)
    del sound, q
    lse = torch.logsumexp(z.detach() * case["scale"], 1)
    out = []
    if labels is not None:
        logp = logq.gather(1, labels.long().clamp(min=0)[:, None])[:, 0]
        logp = torch.where(used, logp, 0.0)
        out.append(logp.detach())
    out += [torch.where(used, lse, 0.0), torch.where(used, entropy.detach(), 0.0)]
    if K:
        index = torch.full((T, K), -1, dtype=torch.int32, device=z.device)
        value = torch.full((T, K), -math.inf, dtype=torch.float64, device=z.device)
        for a in range(0, T, 256):
            b = min(T, a + 256)
            order = torch.sort(s["logits"][a:b], dim=1, descending=True, stable=True).indices[:, :K]
            found = logq[a:b].gather(1, order)
            keep = used[a:b, None] & (found > -math.inf)
            index[a:b, :order.shape[1]] = torch.where(keep, order, -1).int()
            value[a:b, :order.shape[1]] = torch.where(keep, found, -math.inf)
        out += [index, value]
    if case["backward"]:
        total = (logp * s["grad"].double())[used].sum() + (entropy * s["grad_entropy"].double())[used].sum()
        out.append(torch.autograd.grad(total, z)[0])
    return tuple(out)
