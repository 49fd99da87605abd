"""Scores of given tokens with their alternatives, and the eviction of a key-value cache, for measurement: cases, plain
form in elementary torch operations, and definition in 64 bits.

Operators: log-probabilities of given tokens with the drawn one's rank, the entropy and the top alternatives, and their
gradient; attention weights accumulated for each slot of a cache; the slots that a budget keeps, packed; and one token
put into a full cache over the slot that is last by weight.
"""

import math

import torch

own = False

# Vocabularies and batches are those of this repository's workloads (4 x 32000 up to 1024 x 262144), and odd ones
# between; caches have the usual head sizes, one to sixty-four sequences and up to 64 Ki slots.
_MAX_LOGITS = 1024 * 262144  # of 16 bits
_MAX_CACHE = 1 << 30  # bytes of keys

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one decode step of a small batch that reports the drawn token and five alternatives
        dict(name="scores 4x32000 f32 top 5", op="scores", B=4, V=32000, dtype="f32", M=1, top=5, mask=0, inv_t=1.0, entropy=False),
        # a decode step under truncated sampling: the drawn token, fifteen fixed ones and twenty alternatives of the kept set
        dict(name="scores 64x128256 bf16 kept, top 20", op="scores", B=64, V=128256, dtype="bf16", M=16, top=20, mask=256, inv_t=1.25, entropy=True),
        # a whole prompt's log-probabilities, ranks and twenty alternatives a token: the largest
        dict(name="scores 1024x262144 bf16 top 20", op="scores", B=1024, V=262144, dtype="bf16", M=1, top=20, mask=0, inv_t=1.0, entropy=True),
        # distillation on a teacher's 64 alternatives a token, odd vocabulary, with an entropy term
        dict(name="grad 255x50021 f32, 64 ids", op="grad", B=255, V=50021, dtype="f32", K=64, mask=0, inv_t=0.5, entropy=True),
        # the same on 20 alternatives for a long sequence
        dict(name="grad 512x151936 bf16, 20 ids", op="grad", B=512, V=151936, dtype="bf16", K=20, mask=0, inv_t=1.0, entropy=False),
        # a decode step's weights, a few sequences in a small cache
        dict(name="weights 4 x 1024, one query", op="weights", B=4, H=8, G=4, T=1, S=1024, D=128, dtype="bf16", slots=True),
        # a decode step's weights in a long cache
        dict(name="weights 16 x 32768, one query", op="weights", B=16, H=8, G=4, T=1, S=32768, D=128, dtype="bf16", slots=False),
        # the last 32 queries of long prompts, whose weights decide what the prompt's cache keeps
        dict(name="weights 8 x 16384, 32 queries", op="weights", B=8, H=8, G=4, T=32, S=16384, D=128, dtype="bf16", slots=False),
        # a prompt's cache cut to a small budget
        dict(name="evict 2 x 1500 to 256", op="evict", B=2, H=8, S=1500, budget=256, D=64, dtype="bf16", sink=4, recent=32, slots=False),
        # long prompts cut to an eighth
        dict(name="evict 16 x 32768 to 4096", op="evict", B=16, H=8, S=32768, budget=4096, D=128, dtype="bf16", sink=4, recent=64, slots=False),
        # a decode step of a full batch over full caches
        dict(name="insert 64 x 4096", op="insert", B=64, H=8, S=4096, D=128, dtype="bf16", sink=4, recent=128),
        # a decode step of one sequence
        dict(name="insert 1 x 1000", op="insert", B=1, H=8, S=1000, D=128, dtype="bf16", sink=4, recent=32),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scores", "scores", "grad", "weights", "weights", "evict", "insert"])
    dtype = rng.choice(["f32", "bf16", "bf16"])
    c = dict(op=op, dtype=dtype)
    size = 4 if dtype == "f32" else 2
    if op in ("scores", "grad"):
        c["V"] = _log_uniform(rng, 1000, 262144)
        c["B"] = _log_uniform(rng, 1, min(4096, _MAX_LOGITS * 2 // size // c["V"]))
        c["mask"] = rng.choice([0, 0, rng.randint(2, 1000)])
        c["inv_t"] = rng.choice([1.0, 1.0, rng.randint(45, 102) / 64])
        c["entropy"] = rng.random() < 0.5
        if op == "grad":
            c["K"] = _log_uniform(rng, 1, 128)
        else:
            c["M"] = rng.choice([1, 1, _log_uniform(rng, 2, 64)])
            c["top"] = rng.choice([0, 5, 20, _log_uniform(rng, 1, 128)])
        return c
    c["H"] = rng.choice([1, 2, 4, 8])
    c["D"] = rng.choice([64, 128, 128, 96, 256])
    c["S"] = _log_uniform(rng, 64, 65536)
    most = max(1, _MAX_CACHE // (size * c["H"] * c["D"] * c["S"]))
    if op == "weights":
        c["G"] = rng.choice([1, 4, 8])
        c["T"] = rng.choice([1, 1, _log_uniform(rng, 2, 32)])
        # 32 bits have no tensor-core product to use: shorter windows
        c["T"] = min(c["T"], 4) if dtype == "f32" else c["T"]
        most = max(1, min(most, (8 * 8 * 128 * 16384 * 128) // (c["H"] * c["G"] * c["T"] * c["S"] * c["D"])))
        c["slots"] = rng.random() < 0.5
    else:
        c["sink"] = rng.choice([0, 4])
        c["recent"] = rng.randint(0, min(128, c["S"] // 4))
        if op == "evict":
            c["budget"] = max(c["sink"] + c["recent"], _log_uniform(rng, 16, c["S"]))
            c["slots"] = rng.random() < 0.5
    c["B"] = _log_uniform(rng, 1, min(64, most))
    return c


def _prepare_rows(case, g, dev):
    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    B, V = case["B"], case["V"]
    x = torch.empty(B, V, dtype=_TYPES[case["dtype"]], device=dev)
    M = case["M"] if case["op"] == "scores" else case["K"]
    ids = torch.empty(B, M, dtype=torch.int32, device=dev)
    keep = case["mask"]
    mask = torch.empty(B, V, dtype=torch.bool, device=dev) if keep else None
    step = max(1, (1 << 26) // V)
    for a in range(0, B, step):
        b = min(B, a + step)
        f = normal(b - a, V).mul_(2.0)
        # a few likely tokens, as a trained head has them
        f.scatter_add_(1, (uniform(b - a, 12) * V).long().clamp_(max=V - 1), 6.0 + 2.0 * normal(b - a, 12))
        x[a:b] = f
        y = x[a:b].float() * case["inv_t"]
        if keep:
            mask[a:b] = y >= y.topk(min(V, keep), dim=1).values[:, -1:]
            y.masked_fill_(~mask[a:b], -math.inf)
        if case["op"] == "grad":
            # a teacher's likely tokens: the student's own, shaken
            ids[a:b] = y.add_(normal(b - a, V)).topk(min(M, V), dim=1).indices.int()
        else:
            # the largest of logit + Gumbel noise is a draw from the softmax; the other given tokens are any
            noise = uniform(b - a, V).clamp_(min=1e-30).log_().neg_().clamp_(min=1e-30).log_().neg_()
            ids[a:b] = (uniform(b - a, M) * V).int().clamp_(max=V - 1)
            ids[a:b, 0] = y.add_(noise).argmax(dim=1).int()
    first = torch.arange(B, device=dev) == 0
    if keep:
        # a few rows kept nothing (a voided row)
        mask[(uniform(B) < 0.01) & ~first] = False
    ids[(uniform(B, M) < 0.05) & ~first[:, None]] = -1  # padding
    s = dict(case=case, x=x, ids=ids, mask=mask)
    if case["op"] == "grad":
        s["g_logp"] = -uniform(B, M) / (B * M)
        s["g_ent"] = 0.1 * normal(B) / B if case["entropy"] else None
    return s


def _prepare_cache(case, g, dev):
    B, H, S, D = case["B"], case["H"], case["S"], case["D"]
    dt = _TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = dict(case=case)
    # keys of slots that many queries look at are long
    s["k"] = torch.empty(B, H, S, D, dtype=dt, device=dev)
    for b in range(B):
        s["k"][b] = normal(H, S, D) * (0.8 + 0.3 * normal(H, S, 1).abs())
    short = torch.randint(max(1, S // 2), S + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    s["lengths"] = torch.where(torch.rand(B, generator=g, device=dev) < 0.25, short, S).int()
    # weight gathered so far: spread over orders of magnitude, and none for slots that no query has looked at
    w = (2.0 * normal(B, H, S)).exp_()
    w[torch.rand(B, H, S, generator=g, device=dev) < 0.05] = 0.0
    s["w"] = w
    s["seen"] = s["positions"] = None
    if case["op"] == "insert" or case["slots"]:
        # a cache that has evicted before: later tokens, in slots of any order
        s["seen"] = s["lengths"] + torch.randint(0, S + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        at = torch.rand(B, H, S, generator=g, device=dev)
        at.masked_fill_(torch.arange(S, device=dev) >= s["lengths"][:, None, None], 2.0)
        order = at.argsort(dim=2).argsort(dim=2).int()
        s["positions"] = (order + (s["seen"] - s["lengths"])[:, None, None] * (order >= 4)).contiguous()
    if case["op"] == "weights":
        s["q"] = (1.5 * normal(B, case["T"], H * case["G"], D)).to(dt)
    else:
        s["v"] = torch.empty(B, H, S, D, dtype=dt, device=dev)
        for b in range(B):
            s["v"][b] = normal(H, S, D)
    if case["op"] == "insert":
        s["new_k"], s["new_v"] = normal(B, H, D).to(dt), normal(B, H, D).to(dt)
    return s


def prepare(case, seed):
    """Logits of a peaked language-model head with the tokens given for them, or a cache with the weight that its slots
    have gathered."""
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    return _prepare_rows(case, g, dev) if case["op"] in ("scores", "grad") else _prepare_cache(case, g, dev)


DECAY = 0.98


def _softmax(s):
    """y - max in 32 bits and its exponentials, their sums in 64; log-probabilities of the ids in 64 bits (0 where there is
    none, -inf where the token has no probability)."""
    c, x = s["case"], s["x"]
    f = x.float()
    if s["mask"] is not None:
        f = f.masked_fill(~s["mask"], -math.inf)
    top = f.amax(dim=1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    y = f - top
    none = s["ids"] < 0
    t = s["ids"].long().clamp(min=0)
    y_t = y.gather(1, t).double() * c["inv_t"]
    if c["inv_t"] != 1.0:
        y = y * c["inv_t"]
    e = y.exp()
    S = e.sum(dim=1, dtype=torch.float64)[:, None]
    logp = torch.where(S > 0, y_t - S.log(), -math.inf).masked_fill(none, 0.0)
    H = None
    if c["entropy"]:
        y = y.clamp(min=-1e4)
        H = S[:, 0].log() - (e * y).sum(dim=1, dtype=torch.float64) / S[:, 0]
        H = torch.where(S[:, 0] > 0, H, 0.0)
    return f, top, y, e, S, t, none, logp, H


def _scores_plain(s):
    c = s["case"]
    f, top, _, _, S, t, none, logp, H = _softmax(s)
    x_t = f.gather(1, t[:, :1])
    at = torch.arange(c["V"], device=f.device, dtype=torch.int32)
    rank = ((f > x_t) | ((f == x_t) & (at < s["ids"][:, :1]))).sum(dim=1, dtype=torch.int32)
    out = [logp.float(), torch.where(none[:, 0] | (logp[:, 0] == -math.inf), -1, rank)]
    if H is not None:
        out.append(H.float())
    if c["top"]:
        # one whole number for each logit, larger for larger ones and for lower ids among equal ones
        bits = (f + 0.0).view(torch.int32)
        key = (torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() << 32) | (0x7FFFFFFF - at)
        ids = key.topk(min(c["top"], c["V"]), dim=1).indices
        x = f.gather(1, ids)
        some = x > -math.inf
        lp = (x - top).double() * c["inv_t"] - S.log()
        out += [torch.where(some, ids, -1).int(), torch.where(some, lp, -math.inf).float()]
    return out


def _grad_plain(s):
    c = s["case"]
    _, _, y, e, S, t, none, logp, H = _softmax(s)
    it = c["inv_t"]
    a = torch.where(~none & (logp > -math.inf), s["g_logp"].double(), 0.0) * it
    per = torch.where(S > 0, 1.0 / S, 0.0)
    inner = a.sum(dim=1, keepdim=True)
    if H is None:
        out = e * (-inner * per).float()
    else:
        b = torch.where(S > 0, s["g_ent"].double()[:, None], 0.0) * it
        shift = torch.where(S > 0, H[:, None] - S.log(), 0.0)
        out = e * (y * b.float() + (inner + b * shift).float()) * (-per).float()
    out.scatter_add_(1, t, a.float())
    return [out.to(s["x"].dtype)]


def _weights_plain(s):
    c = s["case"]
    B, H, S, D, G, T = (c[n] for n in ("B", "H", "S", "D", "G", "T"))
    q = s["q"].float().view(B, T, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, D)
    x = torch.matmul(q, s["k"].float().transpose(2, 3)).view(B, H, T, G, S) * (1.0 / math.sqrt(D))
    slot = torch.arange(S, device=x.device, dtype=torch.int32)
    at = slot.expand(B, H, S) if s["positions"] is None else s["positions"]
    live = slot < s["lengths"][:, None, None]
    seen = s["lengths"] if s["seen"] is None else s["seen"]
    last = seen[:, None] - T + torch.arange(T, device=x.device, dtype=torch.int32)
    sees = (at[:, :, None] <= last[:, None, :, None]) & live[:, :, None]
    x.masked_fill_(~sees[:, :, :, None], -math.inf)
    top = x.amax(dim=4, keepdim=True)
    x.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = x.sum(dim=4, keepdim=True)
    x.div_(total.masked_fill(total == 0, 1.0))
    s["w"].copy_(torch.where(live, s["w"] * DECAY + x.sum(dim=(2, 3)), s["w"]))
    return [s["w"]]


def _order(s, lengths):
    """One whole number a slot, larger for slots that are kept longer: protected ones first, then by weight, then by slot."""
    c, w = s["case"], s["w"]
    S = c["S"]
    slot = torch.arange(S, device=w.device, dtype=torch.int32)
    at = slot.expand_as(w) if s["positions"] is None else s["positions"]
    seen = (lengths if s["seen"] is None else s["seen"])[:, None, None]
    guarded = (at < c["sink"]) | (at >= seen - c["recent"])
    bits = (w + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * 65536 + (65535 - slot)
    key = key + guarded.long() * (1 << 52)
    live = slot < lengths[:, None, None]
    return key, live, at


def _evict_plain(s):
    c = s["case"]
    n = min(c["budget"], c["S"])
    key, live, at = _order(s, s["lengths"])
    key = key.masked_fill(~live, -(1 << 60))
    # the kept slots, in slot order; behind them, where a sequence is shorter than the budget, nothing
    slots = key.topk(n, dim=2).indices.sort(dim=2).values
    some = torch.arange(n, device=key.device) < s["lengths"].clamp(max=n)[:, None, None]
    some = some.expand_as(slots)

    def rows(x):
        got = x.gather(2, slots[..., None].expand(*slots.shape, c["D"]))
        return torch.nn.functional.pad(got.masked_fill_(~some[..., None], 0), (0, 0, 0, c["budget"] - n))

    def values(x, fill):
        return torch.nn.functional.pad(x.gather(2, slots).masked_fill_(~some, fill), (0, c["budget"] - n), value=fill)

    return [rows(s["k"]), rows(s["v"]), values(s["w"], 0.0), values(at, -1), s["lengths"].clamp(max=n)]


def _insert_plain(s):
    c = s["case"]
    lengths, D = s["lengths"], c["D"]
    key, live, _ = _order(s, lengths)
    last = key.masked_fill(~live, 1 << 60).argmin(dim=2)
    slot = torch.where((lengths < c["S"])[:, None], lengths.long()[:, None], last)
    where = slot[..., None]
    s["k"].scatter_(2, where[..., None].expand(*where.shape, D), s["new_k"][:, :, None])
    s["v"].scatter_(2, where[..., None].expand(*where.shape, D), s["new_v"][:, :, None])
    s["w"].scatter_(2, where, 0.0)
    s["positions"].scatter_(2, where, s["seen"][:, None, None].expand_as(where))
    lengths.add_(1).clamp_(max=c["S"])
    s["seen"].add_(1)
    return [slot.int(), s["k"], s["v"], s["w"], s["positions"], lengths, s["seen"]]


def _run_own(s):
    import top_selection_row_gb300 as q

    c = s["case"]
    if c["op"] == "scores":
        r = q.qrita_token_scores(s["x"], s["ids"], top=c["top"], mask=s["mask"], inv_temperature=c["inv_t"], entropy=c["entropy"], rank=True)
        return [r.logp, r.rank] + ([r.entropy] if c["entropy"] else []) + ([r.top_ids, r.top_logp] if c["top"] else [])
    if c["op"] == "grad":
        return [q.qrita_token_scores_grad(s["x"], s["ids"], s["g_logp"], s["g_ent"], mask=s["mask"], inv_temperature=c["inv_t"])]
    if c["op"] == "weights":
        return [q.qrita_cache_weights(s["q"], s["k"], s["w"], s["lengths"], positions=s["positions"], seen=s["seen"], decay=DECAY)]
    if c["op"] == "evict":
        r = q.qrita_cache_evict(s["k"], s["v"], s["w"], s["lengths"], c["budget"], sink=c["sink"], recent=c["recent"], positions=s["positions"], seen=s["seen"])
        return [r.keys, r.values, r.weights, r.positions, r.lengths]
    slots = q.qrita_cache_insert(s["k"], s["v"], s["w"], s["positions"], s["lengths"], s["seen"], s["new_k"], s["new_v"], c["S"], sink=c["sink"], recent=c["recent"])
    return [slots, s["k"], s["v"], s["w"], s["positions"], s["lengths"], s["seen"]]


def run(state):
    if own:
        return _run_own(state)
    return {"scores": _scores_plain, "grad": _grad_plain, "weights": _weights_plain, "evict": _evict_plain, "insert": _insert_plain}[state["case"]["op"]](state)


def work(case):
    """Inputs read once (under a mask: the mask, and the kept logits), outputs written once. A multiply-add, an exponential,
    a sum and maxima for a logit's scores; a multiply-add a dimension for a query's weight on a key."""
    s = 4 if case["dtype"] == "f32" else 2
    B = case["B"]
    if case["op"] in ("scores", "grad"):
        V = case["V"]
        touched = B * (min(V, case["mask"]) if case["mask"] else V)
        read = touched * s + (B * V if case["mask"] else 0)
        if case["op"] == "scores":
            return {"bytes": read + B * (8 * case["M"] + 8 * case["top"] + (8 if case["entropy"] else 4)), "flops": touched * (9 if case["entropy"] else 7)}
        return {"bytes": read + B * V * s + B * (8 * case["K"] + 4), "flops": touched * 10}
    H, S, D = case["H"], case["S"], case["D"]
    if case["op"] == "weights":
        R = case["G"] * case["T"]
        return {"bytes": B * H * (S * D * s + R * D * s + S * (12 if case["slots"] else 8)), "flops": B * H * R * S * (2 * D + 4)}
    if case["op"] == "evict":
        n = min(S, case["budget"])
        return {"bytes": B * H * (S * (8 if case["slots"] else 4) + n * (4 * D * s + 8)), "flops": B * H * S * 4}
    return {"bytes": B * H * (S * 8 + 4 * D * s + 12), "flops": B * H * S * 4}


def exact(case, seed):
    """The definitions in 64 bits, a block of rows or a sequence at a time. Packed and replaced slots are moved, not
    computed: they have none."""
    if case["op"] in ("evict", "insert"):
        return None
    s = prepare(case, seed)
    D64 = torch.float64
    if case["op"] == "weights":
        B, H, S, G, T = (case[n] for n in ("B", "H", "S", "G", "T"))
        out = torch.empty(B, H, S, dtype=D64, device=s["k"].device)
        for b in range(B):
            n = int(s["lengths"][b])
            seen = n if s["seen"] is None else int(s["seen"][b])
            for h in range(H):
                out[b, h] = s["w"][b, h]
                p = torch.arange(n, device=out.device) if s["positions"] is None else s["positions"][b, h, :n]
                total = DECAY * s["w"][b, h, :n].to(D64)
                k = s["k"][b, h, :n].to(D64)
                for t in range(T):
                    x = s["q"][b, t, h * G : (h + 1) * G].to(D64) @ k.T / math.sqrt(case["D"])
                    x[:, p > seen - T + t] = -math.inf
                    total += torch.nan_to_num(torch.softmax(x, dim=1), nan=0.0).sum(dim=0)
                out[b, h, :n] = total
        return [out]
    x, ids, mask = s["x"], s["ids"].long(), s["mask"]
    B, V = x.shape
    it = case["inv_t"]
    step = max(1, (1 << 24) // V)
    low = torch.full((), -math.inf, dtype=D64, device=x.device)
    parts = []
    for a in range(0, B, step):
        b = min(B, a + step)
        u = x[a:b].to(D64)
        if mask is not None:
            u = torch.where(mask[a:b], u, low)
        l = torch.nan_to_num(torch.log_softmax(u * it, dim=1), nan=-math.inf, neginf=-math.inf)
        H = torch.special.entr(l.exp()).sum(dim=1)
        t = ids[a:b]
        at = l.gather(1, t.clamp(min=0))
        if case["op"] == "scores":
            got = [torch.where(t < 0, torch.zeros_like(at), at)]
            ranks = u.argsort(dim=1, descending=True, stable=True)
            rank = (ranks == t[:, :1]).int().argmax(dim=1)
            got.append(torch.where((t[:, 0] < 0) | ~torch.isfinite(at[:, 0]), -torch.ones_like(rank), rank).int())
            if case["entropy"]:
                got.append(H)
            if case["top"]:
                first = ranks[:, : case["top"]]
                lp = l.gather(1, first)
                got += [torch.where(torch.isfinite(lp), first, -torch.ones_like(first)).int(), lp]
        else:
            g = torch.where((t >= 0) & torch.isfinite(at), s["g_logp"][a:b].to(D64), torch.zeros_like(at))
            p = l.exp()
            part = -g.sum(dim=1, keepdim=True) * p
            if case["entropy"]:
                part += s["g_ent"][a:b, None].to(D64) * (torch.special.entr(p) - p * H[:, None])
            got = [part.scatter_add_(1, t.clamp(min=0), g) * it]
        parts.append(got)
    return [torch.cat(v) for v in zip(*parts)]
