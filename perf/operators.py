"""The loss operators over rows of logits, for measurement: their cases, their plain form in
elementary torch operations, and their definition in 64 bits.

Operators: log-probabilities of given tokens (with the entropy) and their gradient, the clipped
policy loss with a KL term and its gradient, the preference loss on paired sequences and its
gradient. Inputs are rows of logits as a language model's head gives them, the tokens drawn from
them, and (where a rollout was sampled from a truncated set) the keep-mask of that set.
"""

import math
import random

import torch

own = False

# Vocabularies and batches are those of this repository's workloads (4 x 32000 up to
# 1024 x 262144), and odd ones between.
_MAX_ELEMENTS = 1024 * 262144


def listed():
    return [
        # one decode step of a small batch: the log-probability of each drawn token is stored
        dict(name="logprobs 4x32000 f32", op="logprobs", B=4, V=32000, dtype="f32", mask=0, inv_t=1.0, entropy=False, ignored=0.0),
        # a decode step under truncated sampling: log-probabilities renormalised over the kept set
        dict(name="logprobs 64x128256 bf16 kept", op="logprobs", B=64, V=128256, dtype="bf16", mask=256, inv_t=1.25, entropy=True, ignored=0.0),
        # rescoring whole rollouts (reference or old policy): log-probabilities and entropies
        dict(name="logprobs 1024x262144 bf16", op="logprobs", B=1024, V=262144, dtype="bf16", mask=0, inv_t=1.0, entropy=True, ignored=0.05),
        # the gradient of a user's own loss of log-probabilities and entropies, odd vocabulary
        dict(name="grad 255x50021 f32", op="grad", B=255, V=50021, dtype="f32", mask=0, inv_t=1.0, entropy=True, ignored=0.1),
        # the same for one long supervised sequence: log-probabilities alone
        dict(name="grad 512x151936 bf16", op="grad", B=512, V=151936, dtype="bf16", mask=0, inv_t=1.0, entropy=False, ignored=0.2),
        # a policy step on a micro batch of one short answer
        dict(name="policy 16x32000 bf16", op="policy", B=16, V=32000, dtype="bf16", mask=0, inv_t=1.0, kl=0.05, ent=0.0, ignored=0.0),
        # a policy step on rows sampled with top-k, scored over the same kept set
        dict(name="policy 128x151936 f32 kept", op="policy", B=128, V=151936, dtype="f32", mask=64, inv_t=1.0, kl=0.02, ent=0.0, ignored=0.1),
        # a policy step with KL and entropy terms at a temperature
        dict(name="policy 257x201088 bf16", op="policy", B=257, V=201088, dtype="bf16", mask=0, inv_t=1.375, kl=0.05, ent=0.01, ignored=0.05),
        # the largest policy step: a batch of long answers
        dict(name="policy 1024x262144 bf16", op="policy", B=1024, V=262144, dtype="bf16", mask=0, inv_t=1.0, kl=0.04, ent=0.0, ignored=0.1),
        # one pair of short answers
        dict(name="preference 1 pair x32000 f32", op="preference", pairs=1, lo=9, hi=17, lens=5, V=32000, dtype="f32", beta=0.1, smooth=0.0, margin=0.0, norm=False, ignored=0.0),
        # pairs of ragged lengths, prompt rows ignored
        dict(name="preference 6 pairs x128256 bf16", op="preference", pairs=6, lo=20, hi=90, lens=7, V=128256, dtype="bf16", beta=0.1, smooth=0.1, margin=0.0, norm=False, ignored=0.25),
        # the largest: long answers, length-normalised with a margin
        dict(name="preference 4 pairs x201088 bf16", op="preference", pairs=4, lo=96, hi=200, lens=3, V=201088, dtype="bf16", beta=2.0, smooth=0.0, margin=0.5, norm=True, ignored=0.1),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "grad", "policy", "policy", "preference", "preference"])
    V = _log_uniform(rng, 1000, 262144)
    c = dict(op=op, V=V, dtype=rng.choice(["f32", "bf16", "bf16"]), ignored=rng.choice([0.0, 0.05, 0.3]))
    # an fp32 element is twice the bytes of a bf16 one
    room = _MAX_ELEMENTS // (2 if c["dtype"] == "f32" else 1)
    if op == "preference":
        rows = min(2048, room // (2 * V))
        c["pairs"] = _log_uniform(rng, 1, max(1, min(64, rows // 8)))
        per = max(2, rows // (2 * c["pairs"]))
        c["hi"] = _log_uniform(rng, 2, max(2, min(per, 512)))
        c["lo"] = rng.randint(1, c["hi"])
        c["lens"] = rng.randint(0, 10**6)
        c.update(beta=rng.choice([0.05, 0.1, 0.5, 2.0]), smooth=rng.choice([0.0, 0.1]), margin=rng.choice([0.0, 0.5]), norm=rng.random() < 0.3)
        return c
    c["B"] = _log_uniform(rng, 1, max(1, min(4096, room // V)))
    c["mask"] = rng.choice([0, 0, rng.randint(2, 1000)])
    c["inv_t"] = rng.choice([1.0, 1.0, rng.randint(45, 102) / 64])
    if op == "policy":
        c.update(kl=rng.choice([0.0, 0.04]), ent=rng.choice([0.0, 0.0, 0.01]))
    else:
        c["entropy"] = rng.random() < 0.5
    return c


def _starts(case):
    r = random.Random(case["lens"])
    s = [0]
    for _ in range(2 * case["pairs"]):
        s.append(s[-1] + r.randint(case["lo"], case["hi"]))
    return s


def _rows(case):
    return _starts(case)[-1] if case["op"] == "preference" else case["B"]


def prepare(case, seed):
    """Logits of a peaked language-model head, tokens drawn from their softmax (within the kept
    set where there is one), and what an earlier policy and a reference gave for those tokens."""
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    B, V = _rows(case), case["V"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    x = torch.empty(B, V, dtype=dt, device=dev)
    tokens = torch.empty(B, dtype=torch.int32, device=dev)
    logp = torch.empty(B, device=dev)
    keep = case.get("mask", 0)
    mask = torch.empty(B, V, dtype=torch.bool, device=dev) if keep else None
    step = max(1, (1 << 26) // V)
    for a in range(0, B, step):
        b = min(B, a + step)
        f = normal(b - a, V).mul_(2.0)
        # a few likely tokens, as a trained head has them
        where = (uniform(b - a, 12) * V).long().clamp_(max=V - 1)
        f.scatter_add_(1, where, 6.0 + 2.0 * normal(b - a, 12))
        f = f.to(dt)
        x[a:b] = f
        y = f.float() * case.get("inv_t", 1.0)
        if keep:
            k = min(V, keep)
            mask[a:b] = y >= y.topk(k, dim=1).values[:, -1:]
            y.masked_fill_(~mask[a:b], -math.inf)
        # the largest of logit + Gumbel noise is a draw from the softmax
        noise = uniform(b - a, V).clamp_(min=1e-30).log_().neg_().clamp_(min=1e-30).log_().neg_()
        t = (y + noise).argmax(dim=1)
        tokens[a:b] = t.int()
        top = y.amax(dim=1, keepdim=True)
        logp[a:b] = (y.gather(1, t[:, None]) - top - (y - top).exp().sum(dim=1, keepdim=True).log())[:, 0]
    if keep:
        # a few rows kept nothing (a voided row), a few tokens have left the kept set since
        first = torch.arange(B, device=dev) == 0
        mask[(uniform(B) < 0.01) & ~first] = False
        lost = (uniform(B) < 0.01) & ~first
        mask[lost, tokens[lost].long()] = False
    tokens[1:][uniform(B - 1) < case["ignored"]] = -1
    s = dict(case=case, x=x, tokens=tokens, mask=mask)
    if case["op"] == "grad":
        s["g_logp"] = normal(B) / B
        s["g_ent"] = normal(B) / B if case["entropy"] else None
    elif case["op"] == "policy":
        s["old"] = logp + 0.1 * normal(B)
        s["ref"] = logp + 0.3 * normal(B) if case["kl"] else None
        s["adv"] = normal(B)
        s["w"] = (0.5 + uniform(B)) / B
    elif case["op"] == "preference":
        starts = _starts(case)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
        n = s["starts"].diff().float()
        # the reference's sequence log-probabilities: the policy has moved toward the preferred ones
        at = s["starts"].long()
        run_sum = torch.cat([torch.zeros(1, device=dev, dtype=torch.float64), torch.where(tokens >= 0, logp, 0 * logp).double().cumsum(0)])
        seq = (run_sum[at[1:]] - run_sum[at[:-1]]).float()
        s["ref"] = (seq / n if case["norm"] else seq) + 0.4 * normal(2 * case["pairs"])
        s["ref"][0::2] -= 1.0
        s["ref"][1::2] += 1.0
        s["w"] = (0.5 + uniform(case["pairs"])) / case["pairs"]
    return s


CLIP_LOW, CLIP_HIGH = 0.2, 0.28


def _softmax(x, tokens, mask, inv_t, entropy):
    """exp(y) in 32 bits and its sums in 64, y = (x - max) * inv_t over the kept set; the tokens'
    log-probabilities in 64 bits (0 in ignored rows, -inf where the token has no probability)."""
    f = x.float()
    if mask is not None:
        f = f.masked_fill(~mask, -math.inf)
    top = f.amax(dim=1, keepdim=True)
    y = f - top.masked_fill(top == -math.inf, 0.0)
    ignored = tokens < 0
    t = tokens.long().clamp(min=0)[:, None]
    y_t = y.gather(1, t)[:, 0].double() * inv_t
    if inv_t != 1.0:
        y = y * inv_t
    e = y.exp()
    S = e.sum(dim=1, dtype=torch.float64)
    logp = torch.where(S > 0, y_t - S.log(), -math.inf).masked_fill(ignored, 0.0)
    H = None
    if entropy:
        y = y.clamp(min=-1e4)
        H = S.log() - (e * y).sum(dim=1, dtype=torch.float64) / S
        H = torch.where((S > 0) & ~ignored, H, 0.0)
    return e, S, y, logp, H, ignored, t


def _logits_grad(e, S, y, H, ignored, t, logp, g, h, inv_t, dtype):
    """sum of g * d logp + h * d H with respect to the logits, rounded once."""
    live = ~ignored & (S > 0)
    a = torch.where(live & (logp > -math.inf), g.double(), 0.0) * inv_t
    per = torch.where(live, 1.0 / S, 0.0)
    if h is None:
        out = e * (-a * per).float()[:, None]
    else:
        b = torch.where(live, h.double(), 0.0) * inv_t
        # -p (a + b (log p + H)), log p = y - log S
        shift = torch.where(live, H - S.log(), 0.0)
        inner = y * b.float()[:, None] + (a + b * shift).float()[:, None]
        out = e * inner * (-per).float()[:, None]
    out.scatter_add_(1, t, a.float()[:, None])
    # 1 - p loses digits near 1: the token's own entry again in 64 bits
    p = torch.where(live, logp.exp(), 0.0)
    at = a * -torch.expm1(torch.where(live, logp, 0.0))
    if h is not None:
        at = at - torch.where(p > 0, b * p * (logp + H), 0.0)
    at = torch.where(live & (logp > -math.inf), at, out.gather(1, t)[:, 0].double())
    out.scatter_(1, t, at.float()[:, None])
    return out.to(dtype)


def _policy_plain(s):
    c, x = s["case"], s["x"]
    e, S, y, logp, H, ignored, t = _softmax(x, s["tokens"], s["mask"], c["inv_t"], c["ent"] != 0)
    joins = ~ignored & (logp > -math.inf)
    lp = torch.where(joins, logp, 0.0)
    adv, w = s["adv"].double(), s["w"].double()
    rho = (lp - s["old"].double()).exp()
    near = rho.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH)
    row = torch.maximum(-adv * rho, -adv * near)
    flows = ~(((adv > 0) & (rho > 1.0 + CLIP_HIGH)) | ((adv < 0) & (rho < 1.0 - CLIP_LOW)))
    g = torch.where(flows, -adv * rho, 0.0)
    kl = torch.zeros_like(rho)
    if s["ref"] is not None:
        q = s["ref"].double() - lp
        kl = torch.expm1(q) - q
        row = row + c["kl"] * kl
        g = g - c["kl"] * torch.expm1(q)
    if H is not None:
        row = row - c["ent"] * H
    row, kl, g = (torch.where(joins, v, 0.0) for v in (row, kl, g))
    h = torch.where(joins, -c["ent"] * w, 0.0) if H is not None else None
    grad = _logits_grad(e, S, y, H, ignored, t, logp, w * g, h, c["inv_t"], x.dtype)
    return [(w * row).sum().float(), grad, row.float(), logp.float(), kl.float()] + ([H.float()] if H is not None else [])


def _preference_plain(s):
    c, x = s["case"], s["x"]
    e, S, y, logp, _, ignored, t = _softmax(x, s["tokens"], None, 1.0, False)
    joins = ~ignored & (logp > -math.inf)
    at = s["starts"].long()
    zero = torch.zeros(1, device=x.device, dtype=torch.float64)
    sums = torch.cat([zero, torch.where(joins, logp, 0.0).cumsum(0)])
    seq = sums[at[1:]] - sums[at[:-1]]
    of = torch.bucketize(torch.arange(len(logp), device=x.device), at[1:], right=True)
    scale = torch.ones_like(seq)
    if c["norm"]:
        n = torch.cat([zero, joins.double().cumsum(0)])
        scale = 1.0 / (n[at[1:]] - n[at[:-1]]).clamp(min=1.0)
    seq = seq * scale
    rel = seq - s["ref"].double()
    ratio = rel[0::2] - rel[1::2]
    z = c["beta"] * ratio - c["margin"]
    soft = lambda v: v.clamp(min=0) + torch.log1p((-v.abs()).exp())  # noqa: E731
    pair = (1.0 - c["smooth"]) * soft(-z) + c["smooth"] * soft(z)
    w = s["w"].double()
    dz = w * c["beta"] * (c["smooth"] * z.sigmoid() - (1.0 - c["smooth"]) * (-z).sigmoid())
    by_seq = torch.stack([dz, -dz], dim=1).flatten() * scale
    grad = _logits_grad(e, S, y, None, ignored, t, logp, by_seq[of], None, 1.0, x.dtype)
    return [(w * pair).sum().float(), grad, pair.float(), ratio.float(), seq.float(), logp.float()]


def _run_own(s):
    import top_selection_row_gb300 as q

    c = s["case"]
    if c["op"] == "logprobs":
        logp, H = q.qrita_token_logprobs(s["x"], s["tokens"], mask=s["mask"], inv_temperature=c["inv_t"], entropy=c["entropy"])
        return [logp] if H is None else [logp, H]
    if c["op"] == "grad":
        return [q.qrita_token_logprobs_grad(s["x"], s["tokens"], s["g_logp"], s["g_ent"], mask=s["mask"], inv_temperature=c["inv_t"])]
    if c["op"] == "policy":
        r = q.qrita_policy_loss(s["x"], s["tokens"], s["old"], s["adv"], ref_logp=s["ref"], weights=s["w"], mask=s["mask"], inv_temperature=c["inv_t"],
                                clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl_coef=c["kl"], entropy_coef=c["ent"])
        return [r.loss, r.grad, r.row_loss, r.logp, r.kl] + ([r.entropy] if c["ent"] else [])
    r = q.qrita_preference_loss(s["x"], s["tokens"], s["starts"], ref_logp=s["ref"], weights=s["w"], beta=c["beta"], label_smoothing=c["smooth"],
                                margin=c["margin"], length_norm=c["norm"])
    return [r.loss, r.grad, r.pair_loss, r.log_ratio, r.seq_logp, r.logp]


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] == "policy":
        return _policy_plain(state)
    if c["op"] == "preference":
        return _preference_plain(state)
    e, S, y, logp, H, ignored, t = _softmax(state["x"], state["tokens"], state["mask"], c["inv_t"], c["entropy"])
    if c["op"] == "logprobs":
        return [logp.float()] if H is None else [logp.float(), H.float()]
    return [_logits_grad(e, S, y, H, ignored, t, logp, state["g_logp"], state["g_ent"], c["inv_t"], state["x"].dtype)]


def work(case):
    """Logits read once (under a mask: the mask, and the kept logits), gradient written once,
    and the per-row values; a multiply-add, an exponential, a sum and a maximum an element for
    the softmax, as much again for the gradient."""
    B, V = _rows(case), case["V"]
    s = 4 if case["dtype"] == "f32" else 2
    live = int(round(B * (1.0 - case["ignored"])))
    keep = case.get("mask", 0)
    touched = live * min(V, keep) if keep else live * V
    read = touched * s + (live * V if keep else 0)
    if case["op"] == "logprobs":
        return {"bytes": read + B * (12 if case["entropy"] else 8), "flops": touched * (7 if case["entropy"] else 5)}
    return {"bytes": read + B * V * s + B * 28, "flops": touched * 10}


def exact(case, seed):
    """The definitions in 64 bits, a block of rows at a time."""
    s = prepare(case, seed)
    x, tokens, mask = s["x"], s["tokens"].long(), s["mask"]
    B, V = x.shape
    D = torch.float64
    it = case.get("inv_t", 1.0)
    step = max(1, (1 << 25) // V)
    blocks = [(a, min(B, a + step)) for a in range(0, B, step)]
    every = torch.arange(B, device=x.device)
    live = tokens >= 0

    def log_softmax(a, b):
        u = x[a:b].to(D) * it
        if mask is not None:
            u = torch.where(mask[a:b], u, torch.full((), -math.inf, dtype=D, device=x.device))
        return u - torch.logsumexp(u, dim=1, keepdim=True)  # NaN in a row that keeps nothing

    logp = torch.zeros(B, dtype=D, device=x.device)
    H = torch.zeros(B, dtype=D, device=x.device)
    for a, b in blocks:
        l = log_softmax(a, b)
        rows = torch.arange(b - a, device=x.device)
        v = l[rows, tokens[a:b].clamp(min=0)]
        logp[a:b] = torch.nan_to_num(v, nan=-math.inf, neginf=-math.inf)
        H[a:b] = torch.special.entr(torch.nan_to_num(l, nan=-math.inf, neginf=-math.inf).exp()).sum(dim=1)
    logp[~live] = 0
    H[~live] = 0
    joins = live & torch.isfinite(logp)

    def gradient(g, h):
        out = torch.empty(B, V, dtype=D, device=x.device)
        for a, b in blocks:
            l = torch.nan_to_num(log_softmax(a, b), nan=-math.inf, neginf=-math.inf)
            p = l.exp()
            part = -g[a:b, None] * p
            if h is not None:
                part += h[a:b, None] * (torch.special.entr(p) - p * H[a:b, None])
            r = every[: b - a]
            part[r, tokens[a:b].clamp(min=0)] += g[a:b]
            part[~live[a:b]] = 0
            out[a:b] = part * it
        return out

    zero = torch.zeros((), dtype=D, device=x.device)
    if case["op"] == "logprobs":
        return [logp, H] if case["entropy"] else [logp]
    if case["op"] == "grad":
        g = torch.where(joins, s["g_logp"].to(D), zero)
        return [gradient(g, s["g_ent"].to(D) if case["entropy"] else None)]
    w = s["w"].to(D)
    if case["op"] == "policy":
        A = s["adv"].to(D)
        lp = torch.where(joins, logp, s["old"].to(D))
        rho = torch.exp(lp - s["old"].to(D))
        first, second = A * rho, A * torch.clamp(rho, 1 - CLIP_LOW, 1 + CLIP_HIGH)
        row = -torch.minimum(first, second)
        g = torch.where(first <= second, -first, zero)
        kl = torch.zeros_like(row)
        if s["ref"] is not None:
            q = torch.where(joins, s["ref"].to(D) - logp, zero)
            kl = torch.special.expm1(q) - q
            row = row + case["kl"] * kl
            g = g - case["kl"] * torch.special.expm1(q)
        row = row - case["ent"] * H
        row, kl, g = (torch.where(joins, v, zero) for v in (row, kl, g))
        grad = gradient(w * g, torch.where(joins, -case["ent"] * w, zero) if case["ent"] else None)
        return [torch.dot(w, row), grad, row, logp, kl] + ([H] if case["ent"] else [])
    at = _starts(case)
    seq, scale = [], []
    for a, b in zip(at, at[1:]):
        ok = joins[a:b]
        n = max(1, int(ok.sum())) if case["norm"] else 1
        seq.append(logp[a:b][ok].sum() / n)
        scale.append(1.0 / n)
    seq = torch.stack(seq)
    rel = seq - s["ref"].to(D)
    ratio = rel[::2] - rel[1::2]
    z = case["beta"] * ratio - case["margin"]
    ls = case["smooth"]
    pair = -(1 - ls) * torch.nn.functional.logsigmoid(z) - ls * torch.nn.functional.logsigmoid(-z)
    slope = w * case["beta"] * (torch.sigmoid(z) - (1 - ls))
    g = torch.zeros(B, dtype=D, device=x.device)
    for i, (a, b) in enumerate(zip(at, at[1:])):
        g[a:b] = slope[i // 2] * scale[i] * (1 if i % 2 == 0 else -1)
    return [torch.dot(w, pair), gradient(torch.where(joins, g, zero), None), pair, ratio, seq, logp]
