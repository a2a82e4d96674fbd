"""Losses over rows of logits, as a training or scoring step calls them, with their plain forms.

Five operators: the log-probability of each token's label with its gradient, the clipped policy
loss with a KL term, the preference loss of paired sequences, distillation from a teacher's top
logits, and the balance loss of an expert router.  ``own`` selects the library's kernels; the
plain forms are elementary torch operations in 32 bits, in 64 where a long sum or a value next to
a clipping border is formed.  ``exact`` states each operator again in 64 bits, its gradients by
automatic differentiation of the loss.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
MOST = 8192 * 131072 * 2      # bytes of logits in the largest listed case


def listed():
    return [
        # scoring one drafted token in each of four streams: only the launches cost
        dict(name="logp score 4x32768", op="logp", type="bf16", T=4, V=32768, masked=0,
             backward=False, scale=0.7),
        # one micro-batch of cross-entropy training
        dict(name="logp train 4096x65536", op="logp", type="bf16", T=4096, V=65536, masked=512,
             backward=True, scale=1.0),
        # a few short rollouts with 32-bit logits, no reference model
        dict(name="policy 300x32000 f32", op="policy", type="f32", T=300, V=32000, S=3, pad=0,
             prompt=0.2, ref=False, mean=True, clip_lo=0.2, clip_hi=0.2, kl=0.0),
        # a micro-batch of long rollouts against a reference model; rows of padding at the end
        dict(name="policy 8192x131072", op="policy", type="bf16", T=8192, V=131072, S=12, pad=100,
             prompt=0.25, ref=True, mean=True, clip_lo=0.2, clip_hi=0.28, kl=0.05),
        # two pairs of short answers, rows of an odd length
        dict(name="preference 333x50001", op="preference", type="bf16", T=333, V=50001, P=2, pad=0,
             prompt=0.3, kind="sigmoid", beta=0.1, smoothing=0.1, mean=False),
        # a micro-batch of pairs that share long prompts
        dict(name="preference 8192x65536", op="preference", type="bf16", T=8192, V=65536, P=8,
             pad=64, prompt=0.5, kind="sigmoid", beta=0.1, smoothing=0.0, mean=False),
        # a teacher's 20 best tokens for a short sequence
        dict(name="distill 40x32000 k20 f32", op="distill", type="f32", T=40, V=32000, K=20,
             lse=False, tau=1.0, weights=False),
        # a micro-batch with a teacher's 64 best tokens, its own normaliser given, padding weighted 0
        dict(name="distill 4096x131072 k64", op="distill", type="bf16", T=4096, V=131072, K=64,
             lse=True, tau=1.0, weights=True),
        # 32-bit logits, rows of an odd length, a softened teacher
        dict(name="distill 1500x100003 f32", op="distill", type="f32", T=1500, V=100003, K=128,
             lse=False, tau=2.0, weights=False),
        # a small router on a short batch
        dict(name="balance 512x8 k2", op="balance", type="f32", T=512, E=8, K=2, G=1, pad=0,
             alpha=0.01, z=0.001),
        # one layer's router over a micro-batch
        dict(name="balance 16384x64 k6", op="balance", type="f32", T=16384, E=64, K=6, G=1, pad=0,
             alpha=0.01, z=0.0),
        # a wide router, the loss taken within each of the packed sequences, padding behind them
        dict(name="balance 65536x256 k8", op="balance", type="bf16", T=65536, E=256, K=8, G=24,
             pad=1000, alpha=0.001, z=0.0001),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("logp", "policy", "preference", "distill", "balance"))
    kind = rng.choice(("bf16", "f32"))
    if op == "balance":
        E = rng.choice((4, 8, 16, 32, 60, 64, 72, 128, 160, 256, 384, 512))
        T = _log(rng, 1, 65536 * 256 // E if E > 256 else 65536)
        G = rng.randint(1, max(1, min(32, T // 8)))
        return dict(op=op, type=kind, T=T, E=E, K=rng.randint(1, min(8, E)), G=G,
                    pad=rng.randint(0, T // 16), alpha=round(rng.uniform(0.001, 0.1), 4),
                    z=rng.choice((0.0, 0.0001, 0.001)))
    V = _log(rng, 200, 160000)
    if rng.random() < 0.5:
        V = max(64, V - V % 64)
    T = _log(rng, 1, min(8192, max(1, MOST // (V * BYTES[kind]))))
    case = dict(op=op, type=kind, T=T, V=V)
    if op == "logp":
        case.update(masked=rng.choice((0, V // 50)), backward=rng.random() < 0.7,
                    scale=round(rng.uniform(0.5, 1.5), 3))
    elif op == "policy":
        case.update(S=rng.randint(1, max(1, min(16, T // 4))), pad=rng.randint(0, T // 16),
                    prompt=round(rng.uniform(0.0, 0.5), 2), ref=rng.random() < 0.6,
                    mean=rng.random() < 0.7, clip_lo=0.2, clip_hi=rng.choice((0.2, 0.28)),
                    kl=round(rng.uniform(0.0, 0.1), 3))
    elif op == "preference":
        case.update(P=rng.randint(1, max(1, min(8, T // 8))), pad=rng.randint(0, T // 16),
                    prompt=round(rng.uniform(0.0, 0.6), 2), kind=rng.choice(("sigmoid", "square")),
                    beta=round(rng.uniform(0.05, 0.5), 2), smoothing=rng.choice((0.0, 0.1)),
                    mean=rng.random() < 0.3)
    else:
        case.update(K=min(V, _log(rng, 1, 256)), lse=rng.random() < 0.5,
                    tau=round(rng.uniform(0.7, 3.0), 2), weights=rng.random() < 0.5)
    return case


def _offsets(cut, g, groups, rows, dev):
    """Ragged packed lengths over the rows: offsets [groups + 1], int64."""
    share = torch.rand(groups, generator=g, device=dev, dtype=torch.float64) + 0.3
    off = (torch.cumsum(share, 0) / share.sum() * rows).round().to(torch.int64)
    return torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), off.clamp(max=cut)])


def _segments(off, T):
    """The sequence of each row; rows behind the last sequence get one number more."""
    return torch.bucketize(torch.arange(T, device=off.device), off[1:], right=True)


def _prompts(labels, off, part):
    """Labels of the first `part` of each sequence become -1 (not scored)."""
    T = labels.numel()
    seg = _segments(off, T)
    begin = torch.cat([off, off[-1:]])[seg]
    length = torch.cat([off[1:] - off[:-1], off.new_zeros(1)])[seg]
    return torch.where(torch.arange(T, device=off.device) - begin < (length * part).long(), -1,
                       labels)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dtype = TYPES[case["type"]]
    T = case["T"]
    s = dict(case=case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if case["op"] == "balance":
        E, K = case["E"], case["K"]
        z = normal(T, E) + 1.5 * normal(E)          # some experts are liked more than others
        s["logits"] = z.to(dtype)
        s["index"] = s["logits"].float().topk(K, dim=1).indices.int()
        s["offsets"] = _offsets(T - case["pad"], g, case["G"], T - case["pad"], dev)
        return s

    # a model's logits: a broad floor, and a label that is often, not always, the likely one
    V = case["V"]
    z = normal(T, V).mul_(2.0)
    labels = torch.randint(0, V - case.get("masked", 0), (T,), generator=g, device=dev)
    rows = torch.arange(T, device=dev)
    z[rows, labels] += 4.0 + 4.0 * normal(T)
    if case.get("masked"):
        z[:, V - case["masked"]:] = -math.inf       # columns that pad the vocabulary
    s["logits"] = z.to(dtype)
    del z
    scale = case.get("scale", 1.0)
    if case["op"] == "logp":
        labels = torch.where(torch.rand(T, generator=g, device=dev) < 0.1, -1, labels)
        s["grad"] = normal(T) / T
    elif case["op"] == "distill":
        K = case["K"]
        u = s["logits"].float() + 0.5 * normal(T, V)
        top = u.topk(K, dim=1)
        s["index"] = top.indices.int()
        s["teacher"] = top.values.contiguous()
        s["lse"] = torch.logsumexp(u.div_(case["tau"]), 1) if case["lse"] else None
        if case["weights"]:
            s["weights"] = (torch.rand(T, generator=g, device=dev) < 0.9).float() / T
        else:
            s["weights"] = None
        return s
    else:
        n = case["S"] if case["op"] == "policy" else 2 * case["P"]
        s["offsets"] = _offsets(T - case["pad"], g, n, T - case["pad"], dev)
        labels = _prompts(labels, s["offsets"], case["prompt"])
        at = labels.clamp(min=0)
        w = s["logits"].double()
        logp = w[rows, at] * scale - torch.logsumexp(w.mul_(scale), 1)
        del w
        if case["op"] == "policy":
            # the behaviour policy is a few updates old.  A ratio nearer than 1e-4 to a clipping
            # border is moved off it: what is clipped there would be left to the last bits
            drift = 0.12 * normal(T).double()
            for border in (math.log1p(-case["clip_lo"]), math.log1p(case["clip_hi"])):
                near = drift - border
                drift = torch.where(near.abs() < 1e-4, drift + 2e-4, drift)
            s["old"] = (logp - drift).float()
            s["adv"] = normal(T)
            s["ref"] = (logp + 0.2 * normal(T)).float() if case["ref"] else None
        else:
            s["ref"] = (logp + 0.2 * normal(T)).float()
    s["labels"] = labels.int()
    return s


def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return PLAIN[case["op"]](case, state)


def _own(case, s):
    import sinkhorn_point_cloud_amd as sk
    if case["op"] == "logp":
        logp, lse = sk.token_logprobs(s["logits"], s["labels"], scale=case["scale"])
        if not case["backward"]:
            return logp, lse
        return logp, lse, sk.token_logprobs_backward(s["logits"], s["labels"], s["grad"],
                                                     scale=case["scale"])
    if case["op"] == "policy":
        return sk.policy_loss(s["logits"], s["labels"], s["offsets"], s["old"], s["adv"],
                              ref=s["ref"], clip=(case["clip_lo"], case["clip_hi"]),
                              kl=case["kl"], mean=case["mean"])
    if case["op"] == "preference":
        return sk.preference_loss(s["logits"], s["labels"], s["offsets"], s["ref"],
                                  beta=case["beta"], smoothing=case["smoothing"],
                                  kind=case["kind"], mean=case["mean"])
    if case["op"] == "distill":
        return sk.distill_loss(s["logits"], s["index"], s["teacher"], teacher_lse=s["lse"],
                               temperature=case["tau"], weights=s["weights"])
    return sk.balance_loss(s["logits"], s["index"], offsets=s["offsets"], balance=case["alpha"],
                           z=case["z"])


# ------------------------------------------------------------------ plain forms

def _softmax_parts(logits, scale):
    """Row maximum m, e = exp(scale z - m) and its sum in 64 bits: softmax = e / S."""
    x = logits.float()
    if scale != 1.0:
        x = x * scale
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    return x, m, e, e.sum(1, keepdim=True, dtype=torch.float64)


def _label_logp(logits, labels, scale):
    """log softmax at the labels in 64 bits, 0 where there is none, and what a gradient needs."""
    x, m, e, S = _softmax_parts(logits, scale)
    at = labels.long().clamp(min=0)
    lse = m[:, 0].double() + torch.log(S[:, 0])
    logp = x.gather(1, at[:, None])[:, 0].double() - lse
    return torch.where(labels >= 0, logp, 0.0), lse, e, S, at


def _label_grad(logits, e, S, at, coef, scale):
    """coef (1[v = label] - softmax) scale, rounded once to the logits' type."""
    coef = (coef * scale).float()
    e *= (-coef.double() / S[:, 0]).float()[:, None]
    e.scatter_add_(1, at[:, None], coef[:, None])
    return e.to(logits.dtype)


def _plain_logp(case, s):
    scale = case["scale"]
    logp, lse, e, S, at = _label_logp(s["logits"], s["labels"], scale)
    lse = torch.where(s["labels"] >= 0, lse, 0.0)      # a row that is not scored has neither
    if not case["backward"]:
        return logp.float(), lse.float()
    coef = torch.where(s["labels"] >= 0, s["grad"], 0.0)
    return logp.float(), lse.float(), _label_grad(s["logits"], e, S, at, coef, scale)


def _member(seg, n):
    """1 where a row belongs to a sequence, [n, T]; the last of the n may be the rows behind."""
    return (seg[None, :] == torch.arange(n, device=seg.device)[:, None]).double()


def _sums(values, seg, n):
    """Sums over the rows of each sequence, and over those behind the last one, in 64 bits."""
    return (_member(seg, n + 1) * values.double()).sum(1)


def _plain_policy(case, s):
    T, n, off = case["T"], case["S"], s["offsets"]
    logp, _, e, S, at = _label_logp(s["logits"], s["labels"], 1.0)
    seg = _segments(off, T)
    used = (s["labels"] >= 0) & (seg < n)
    count = _sums(used, seg, n)
    w = torch.where(used, 1.0 / count[seg] if case["mean"] else 1.0, 0.0)
    A, lo, hi = s["adv"].double(), 1 - case["clip_lo"], 1 + case["clip_hi"]
    r = torch.exp(logp - s["old"].double())
    clipped = ((A > 0) & (r > hi)) | ((A < 0) & (r < lo))
    obj = torch.where(clipped, r.clamp(lo, hi), r) * A
    coef = torch.where(clipped, 0.0, -r * A)
    kl = torch.zeros_like(obj)
    if s["ref"] is not None:
        gap = s["ref"].double() - logp
        kl = torch.expm1(gap) - gap
        coef = coef - case["kl"] * torch.expm1(gap)
    kl = torch.where(used, kl * w, 0.0)
    loss = torch.where(used, -obj * w, 0.0) + case["kl"] * kl
    coef = torch.where(used, coef * w, 0.0)
    return (_sums(loss, seg, n)[:n].float(), _sums(kl, seg, n)[:n].float(),
            torch.where(seg < n, logp, 0.0).float(),
            _label_grad(s["logits"], e, S, at, coef, 1.0))


def _plain_preference(case, s):
    T, P, off = case["T"], case["P"], s["offsets"]
    logp, _, e, S, at = _label_logp(s["logits"], s["labels"], 1.0)
    seg = _segments(off, T)
    used = (s["labels"] >= 0) & (seg < 2 * P)
    ratio = _sums(torch.where(used, logp - s["ref"].double(), 0.0), seg, 2 * P)
    part = torch.ones_like(ratio)
    if case["mean"]:
        part = 1.0 / _sums(used, seg, 2 * P).clamp(min=1.0)
    ratio = ratio * part
    gap = ratio[:-1:2] - ratio[1::2]
    beta, eps = case["beta"], case["smoothing"]
    if case["kind"] == "sigmoid":
        h = beta * gap
        far = torch.log1p(torch.exp(-h.abs()))
        loss = (1 - eps) * (far + (-h).clamp(min=0)) + eps * (far + h.clamp(min=0))
        slope = beta * (eps - 1.0 / (1.0 + torch.exp(h)))
    else:
        loss = (gap - 0.5 / beta) ** 2
        slope = 2.0 * (gap - 0.5 / beta)
    both = torch.stack([slope, -slope], 1).reshape(-1) * part[:-1]
    coef = torch.where(used, torch.cat([both, both.new_zeros(1)])[seg], 0.0)
    return (loss.float(), (beta * ratio[:-1]).float(), torch.where(seg < 2 * P, logp, 0.0).float(),
            _label_grad(s["logits"], e, S, at, coef, 1.0))


def _plain_distill(case, s):
    tau = case["tau"]
    x, m, e, S = _softmax_parts(s["logits"], 1.0 / tau)
    at = s["index"].long()
    u = s["teacher"].double() / tau
    top = u.amax(1, keepdim=True)
    if s["lse"] is None:
        lse = top + torch.log(torch.exp(u - top).sum(1, keepdim=True))
    else:
        lse = s["lse"].double()[:, None]
    logq = x.gather(1, at).double() - m.double() - torch.log(S)
    p = torch.exp(u - lse)
    w = torch.ones_like(S) if s["weights"] is None else s["weights"].double()[:, None]
    loss = (p * (u - lse - logq)).sum(1) * w[:, 0] * tau * tau
    e *= (p.sum(1, keepdim=True) * w * tau / S).float()
    e.scatter_add_(1, at, (-p * w * tau).float())
    return loss.float(), e.to(s["logits"].dtype)


def _products(member, values):
    """member [n, T] @ values [T, E] in 64 bits, the long axis in blocks of 256 rows."""
    n, T = member.shape
    fill = -T % 256
    member = torch.nn.functional.pad(member, (0, fill)).view(n, -1, 256).transpose(0, 1)
    values = torch.nn.functional.pad(values, (0, 0, 0, fill)).view(-1, 256, values.shape[1])
    return torch.bmm(member.contiguous(), values).sum(0)


def _plain_balance(case, s):
    T, E, K, n = case["T"], case["E"], case["K"], case["G"]
    seg = _segments(s["offsets"], T)
    x, m, e, S = _softmax_parts(s["logits"], 1.0)
    lse = m[:, 0].double() + torch.log(S[:, 0])
    p = (e / S).double()
    hot = torch.zeros(T, E, dtype=torch.float64, device=x.device).scatter_(1, s["index"].long(), 1)
    member = _member(seg, n + 1)
    both = _products(member, torch.cat([hot, p], 1))
    counts, share = both[:, :E], both[:, E:]
    each = member.sum(1).clamp(min=1.0)
    f = counts * (E / K) / each[:, None]
    balance = (f * share).sum(1) / each
    zloss = _sums(lse * lse, seg, n) / each
    row = f[seg]
    grad = p * (case["alpha"] * (row - (row * p).sum(1, keepdim=True))
                + 2.0 * case["z"] * lse[:, None]) / each[seg][:, None]
    grad = torch.where((seg < n)[:, None], grad, 0.0).to(s["logits"].dtype)
    return balance[:n].float(), zloss[:n].float(), counts[:n].int(), grad


PLAIN = dict(logp=_plain_logp, policy=_plain_policy, preference=_plain_preference,
             distill=_plain_distill, balance=_plain_balance)


# ------------------------------------------------------------------ work and definitions

def work(case):
    T, b = case["T"], BYTES[case["type"]]
    if case["op"] == "balance":
        row = T * case["E"] * b
        return {"bytes": 2.0 * row + 4.0 * T * case["K"] + 4.0 * case["G"] * case["E"],
                "flops": 12.0 * T * case["E"]}
    row, V = T * b, case["V"]
    if case["op"] == "logp":
        read = 0.9 * row * V + 8.0 * T
        return {"bytes": read + (row * V + 4.0 * T if case["backward"] else 0.0) + 4.0 * T,
                "flops": (8.0 if case["backward"] else 5.0) * 0.9 * T * V}
    if case["op"] == "distill":
        used = 0.9 if case["weights"] else 1.0
        return {"bytes": (used + 1.0) * row * V + 8.0 * T * case["K"] + 4.0 * T,
                "flops": 8.0 * used * T * V}
    used = (1.0 - case["prompt"]) * (1.0 - case["pad"] / T)
    return {"bytes": (used + 1.0) * row * V + 20.0 * T, "flops": 8.0 * used * T * V}


def exact(case, seed):
    s = prepare(case, seed)
    T = case["T"]
    z = s["logits"].double().requires_grad_()
    if case["op"] == "logp":
        logq = torch.log_softmax(z * case["scale"], 1)
        lse = torch.logsumexp(z.detach() * case["scale"], 1)
        labels = s["labels"].long()
        keep = labels >= 0
        lse = torch.where(keep, lse, 0.0)
        logp = torch.where(keep, logq[torch.arange(T, device=z.device), labels.clamp(min=0)], 0.0)
        if not case["backward"]:
            return logp.detach(), lse
        total = (logp * s["grad"].double())[keep].sum()
        return logp.detach(), lse, torch.autograd.grad(total, z)[0]
    if case["op"] == "distill":
        tau = case["tau"]
        u = s["teacher"].double() / tau
        logt = torch.log_softmax(u, 1) if s["lse"] is None else u - s["lse"].double()[:, None]
        logq = torch.log_softmax(z / tau, 1).gather(1, s["index"].long())
        loss = tau ** 2 * (logt.exp() * (logt - logq)).sum(1)
        if s["weights"] is not None:
            loss = loss * s["weights"].double()
        return loss.detach(), torch.autograd.grad(loss.sum(), z)[0]
    off = s["offsets"].tolist()
    if case["op"] == "balance":
        E, K = case["E"], case["K"]
        total, out = z.sum() * 0.0, ([], [], [])
        for a, b in zip(off[:-1], off[1:]):
            n = max(1, b - a)
            hot = torch.bincount(s["index"][a:b].reshape(-1).long(), minlength=E)
            part = torch.softmax(z[a:b], 1).sum(0) / n
            balance = E * (hot.double() / (K * n) * part).sum()
            zloss = (torch.logsumexp(z[a:b], 1) ** 2).sum() / n
            total = total + case["alpha"] * balance + case["z"] * zloss
            for o, v in zip(out, (balance, zloss, hot)):
                o.append(v.detach())
        return (torch.stack(out[0]), torch.stack(out[1]), torch.stack(out[2]).int(),
                torch.autograd.grad(total, z)[0])
    rows = torch.arange(T, device=z.device)
    labels = s["labels"].long()
    logp = torch.log_softmax(z, 1)[rows, labels.clamp(min=0)]
    logp = torch.where((labels >= 0) & (rows < off[-1]), logp, 0.0)
    if case["op"] == "policy":
        losses, kls = [], []
        for a, b in zip(off[:-1], off[1:]):
            keep = labels[a:b] >= 0
            lp, old, adv = logp[a:b][keep], s["old"][a:b][keep].double(), s["adv"][a:b][keep].double()
            r = (lp - old).exp()
            v = -torch.minimum(r * adv, r.clamp(1 - case["clip_lo"], 1 + case["clip_hi"]) * adv)
            kl = torch.zeros_like(v)
            if s["ref"] is not None:
                d = s["ref"][a:b][keep].double() - lp
                kl = d.exp() - d - 1
            n = max(1, int(keep.sum())) if case["mean"] else 1
            losses.append((v + case["kl"] * kl).sum() / n)
            kls.append(kl.sum().detach() / n)
        losses = torch.stack(losses)
        return (losses.detach(), torch.stack(kls), logp.detach(),
                torch.autograd.grad(losses.sum(), z)[0])
    ratios = []
    for a, b in zip(off[:-1], off[1:]):
        keep = labels[a:b] >= 0
        v = (logp[a:b][keep] - s["ref"][a:b][keep].double()).sum()
        ratios.append(v / max(1, int(keep.sum())) if case["mean"] else v)
    ratios = torch.stack(ratios)
    gap = ratios[0::2] - ratios[1::2]
    if case["kind"] == "sigmoid":
        loss = (-(1 - case["smoothing"]) * torch.nn.functional.logsigmoid(case["beta"] * gap)
                - case["smoothing"] * torch.nn.functional.logsigmoid(-case["beta"] * gap))
    else:
        loss = (gap - 1 / (2 * case["beta"])) ** 2
    return (loss.detach(), case["beta"] * ratios.detach(), logp.detach(),
            torch.autograd.grad(loss.sum(), z)[0])
