"""GPU parity of the losses over rows of logits and their gradients, through
the C ABI, against the fp64 oracle (oracle/qrita_losses.py).

Tolerances, from the arithmetic include/qrita.h states. An exponential is off
by at most 2^-22 (the hardware instruction) plus |y| ln2 2^-23 (two roundings
of its argument y, weighed by p: the mean of |y| is at most log2 V < 24), a
sum of n fp32 terms by about 4 sqrt(n) 2^-24 (n below 1024 a thread), so
log S, and with it logp and H before their rounding, is off by at most
2.4e-7 + 2.0e-6 + 7.7e-6 < 1e-5 (ABS). H adds the same again for T. A
probability is off by that much relatively, plus |y| ln2 2^-23 of its own
(|y| < 150 before it underflows): REL = 2.5e-5. A gradient entry is
inv_t (a [j = t] - p (a + h (log p + H))), so it may be off by REL of the
magnitudes of those terms, where a (through rho = exp(logp - old) and
e^q) is off by ABS of rho |A| + kl e^q; bf16 gradients add their one
rounding, 2^-8.
"""

import numpy as np
import pytest

from oracle import bf16_bits_to_f64, dentropy, dlogp, policy_row, preference, row_softmax
from parity_helpers import to_device
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

ABS, REL = 1e-5, 2.5e-5
BF16_ROUND = 2.0 ** -8
F32_ROUND = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import top_selection_row_gb300 as q

    q.lib()
    return torch.device("cuda", 0)


def make_rows(seed, B, V, dtype, keep=0):
    """Logits of a peaked head, tokens (a few ignored), a keep-mask of about
    `keep` ids a row (row 1 keeps nothing, row 2's token is not kept)."""
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((B, V)) * 2).astype(np.float32)
    n = min(V, 5)
    for r in range(B):
        x[r, rng.integers(0, V, n)] += rng.uniform(2, 9, n).astype(np.float32)
    tokens = np.array([int(np.argmax(x[r] + rng.gumbel(size=V))) for r in range(B)], np.int32)
    mask = None
    if keep:
        mask = np.zeros((B, V), np.uint8)
        for r in range(B):
            mask[r, np.argsort(-x[r])[: max(1, min(V, keep))]] = rng.integers(1, 256)
            mask[r, tokens[r]] = 1
        if B > 2:
            mask[1] = 0
            mask[2, tokens[2]] = 0
    if B > 4:
        tokens[3] = -1
        tokens[4] = V  # past the vocabulary: ignored too
    if dtype == "bf16":
        x = f32_to_bf16_bits(x)
    return rng, x, tokens, mask


def widened(x, dtype):
    return bf16_bits_to_f64(x) if dtype == "bf16" else np.asarray(x, np.float64)


def put(dev, a, dt=None):
    import torch

    if a is None:
        return None
    return torch.from_numpy(np.ascontiguousarray(a if dt is None else np.asarray(a, dt))).to(dev)


def padded(t, ld, fill):
    """The rows of t in a buffer of leading dimension ld filled with `fill`."""
    import torch

    buf = torch.full((t.shape[0], ld), fill, dtype=t.dtype, device=t.device)
    buf[:, : t.shape[1]] = t
    return buf


def softmaxes(x, dtype, mask, tokens, inv_t=1.0):
    xs = widened(x, dtype)
    return [row_softmax(xs[r], None if mask is None else mask[r], int(tokens[r]), inv_t) for r in range(len(tokens))]


def near(got, want, tol, what):
    got, want, tol = (np.asarray(v, np.float64) for v in (got, want, tol))
    assert got.shape == want.shape, what
    special = ~np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    assert np.array_equal(got[special & ~np.isnan(want)], want[special & ~np.isnan(want)]), what
    ok = ~special
    bad = ok & ~(np.abs(got - np.where(ok, want, 0)) <= np.broadcast_to(tol, want.shape))
    assert not bad.any(), (what, np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


def near_rows(got, want, what, extra=0.0):
    want = np.asarray(want, np.float64)
    near(got, want, ABS + extra + 2 * F32_ROUND * np.abs(np.where(np.isfinite(want), want, 0)), what)


def near_grad(got, dtype, soft, tokens, a, h, a_tol, inv_t):
    """got [B, V] against inv_t (a dlogp + h dH), a known to a_tol."""
    g = got.float().cpu().numpy().astype(np.float64) if dtype == "bf16" else got.cpu().numpy().astype(np.float64)
    for r, s in enumerate(soft):
        want = a[r] * dlogp(s, int(tokens[r]), inv_t) if a[r] != 0 and s.joins else np.zeros_like(s.p)
        if h[r] != 0:
            want = want + h[r] * dentropy(s, inv_t)
        if not s.ignored and np.isnan(s.logp):
            kept = np.isnan(s.p)
            assert np.isnan(g[r][kept]).all() and not g[r][~kept].any(), r
            continue
        with np.errstate(divide="ignore"):
            lp = np.where(s.p > 0, np.log(np.where(s.p > 0, s.p, 1)), 0)
        terms = s.p * (abs(a[r]) + abs(h[r]) * (np.abs(lp) + s.entropy + 1))
        one = np.zeros_like(s.p)
        if s.joins:
            one[int(tokens[r])] = 1.0
        tol = inv_t * (REL * terms + a_tol[r] * (one + s.p)) + REL * np.abs(want) + 1e-37
        if dtype == "bf16":
            tol = tol + BF16_ROUND * np.abs(want) * 1.01
        near(g[r], want, tol, f"gradient of row {r}")
        if s.ignored or (not s.joins and h[r] == 0):
            assert not g[r].any(), r


# V: one token, odd, below and above a vector, a tile and a CTA's share; the workloads' vocabularies
SIZES = [(1, 1), (3, 2), (5, 7), (6, 8), (5, 31), (7, 257), (6, 1000), (5, 4099), (3, 32000), (6, 50021), (2, 128256)]
FORMS = [("f32", 0), ("bf16", 0), ("f32", 12), ("bf16", 40)]


@pytest.mark.parametrize("dtype,keep", FORMS)
@pytest.mark.parametrize("B,V", SIZES)
def test_logprobs_and_their_gradient(dev, B, V, dtype, keep):
    import torch

    import top_selection_row_gb300 as q

    inv_t = 1.0 if V % 2 else 0.75
    rng, x, tokens, mask = make_rows(V + B, B, V, dtype, keep)
    soft = softmaxes(x, dtype, mask, tokens, inv_t)
    xd, td, md = to_device(x, dtype, dev), put(dev, tokens), put(dev, mask)
    logp, none = q.qrita_token_logprobs(xd, td, mask=md, inv_temperature=inv_t)
    logp2, ent = q.qrita_token_logprobs(xd, td, mask=md, inv_temperature=inv_t, entropy=True)
    assert none is None
    near_rows(logp.cpu().numpy(), [s.logp for s in soft], "logp")
    near_rows(logp2.cpu().numpy(), [s.logp for s in soft], "logp beside H")
    near_rows(ent.cpu().numpy(), [s.entropy for s in soft], "entropy", extra=ABS)
    a = rng.standard_normal(B).astype(np.float32)
    h = rng.standard_normal(B).astype(np.float32)
    zero = np.zeros(B)
    for ga, gh in ((a, None), (None, h), (a, h)):
        got = q.qrita_token_logprobs_grad(xd, td, put(dev, ga), put(dev, gh), mask=md, inv_temperature=inv_t)
        assert got.dtype == xd.dtype
        near_grad(got, dtype, soft, tokens, zero if ga is None else ga, zero if gh is None else gh, zero, inv_t)
    torch.cuda.synchronize()


def policy_case(dev, rng, x, dtype, tokens, mask, inv_t=1.0, kl=0.1, ent=0.0, old=True, ref=True, weights=True, gl=None,
                hi=0.3, **kw):
    import top_selection_row_gb300 as q

    B = len(tokens)
    soft = softmaxes(x, dtype, mask, tokens, inv_t)
    base = np.array([s.logp if s.joins and np.isfinite(s.logp) else -1.0 for s in soft])
    old_v = (base + 0.3 * rng.standard_normal(B)).astype(np.float32) if old else None
    if old:  # draws keep away from the clip's corners, where the slope is not defined
        for corner in (0.8, 1 + hi):
            old_v[np.abs(np.exp(base - old_v) - corner) < 1e-3] += np.float32(0.01)
    ref_v = (base + 0.5 * rng.standard_normal(B)).astype(np.float32) if ref else None
    adv = rng.standard_normal(B).astype(np.float32)
    w = rng.uniform(0.1, 1, B).astype(np.float32) if weights else None
    got = q.qrita_policy_loss(kw.pop("xd", None) if "xd" in kw else to_device(x, dtype, dev), put(dev, tokens),
                              put(dev, old_v), put(dev, adv), ref_logp=put(dev, ref_v), weights=put(dev, w),
                              mask=put(dev, mask), inv_temperature=inv_t, clip_low=0.2, clip_high=hi, kl_coef=kl,
                              entropy_coef=ent, grad_loss=None if gl is None else put(dev, [gl], np.float32), **kw)
    a, h, a_tol, loss, rows, kls, row_tol, kl_tol = (np.zeros(B) for _ in range(8))
    for r, s in enumerate(soft):
        rows[r], kls[r], da, dh = policy_row(s, None if old_v is None else float(old_v[r]), None if ref_v is None else float(ref_v[r]),
                                             float(adv[r]), 0.2, hi, kl, ent)
        wr = (1.0 / B if w is None else float(w[r])) * (1.0 if gl is None else gl)
        rho = 1.0 if old_v is None else np.exp(s.logp - old_v[r]) if s.joins else 0.0
        eq = np.exp(ref_v[r] - s.logp) if ref_v is not None and s.joins else 0.0
        # d row / d logp is at most |A| rho + kl (1 + e^q); an error of ABS in logp moves a by as much
        slope = abs(float(adv[r])) * rho + kl * (1 + eq)
        a[r], h[r], a_tol[r] = wr * da, wr * dh, abs(wr) * ABS * slope
        kl_tol[r] = ABS * (1 + eq)
        row_tol[r] = ABS * slope + 2 * ABS * abs(ent)
        loss[r] = (1.0 / B if w is None else float(w[r])) * rows[r]
        if old_v is not None and s.joins and np.isfinite(rho):
            assert min(abs(rho - 0.8), abs(rho - 1 - hi)) > 1e-4
    near_rows(got.logp.cpu().numpy(), [s.logp for s in soft], "logp")
    near(got.row_loss.cpu().numpy(), rows, row_tol + 2 * F32_ROUND * np.abs(np.where(np.isfinite(rows), rows, 0)), "row loss")
    near(got.kl.cpu().numpy(), kls, kl_tol + 2 * F32_ROUND * np.abs(np.where(np.isfinite(kls), kls, 0)), "kl")
    if got.entropy is not None:
        near_rows(got.entropy.cpu().numpy(), [s.entropy for s in soft], "entropy", extra=ABS)
    wabs = np.full(B, 1.0 / B) if w is None else w
    near(float(got.loss), loss.sum(), (wabs * (row_tol + 4 * F32_ROUND * np.abs(rows))).sum() + F32_ROUND * abs(loss.sum()), "loss")
    if got.grad is not None:
        near_grad(got.grad, dtype, soft, tokens, a, h, a_tol, inv_t)
    return got


@pytest.mark.parametrize("dtype,keep", FORMS)
@pytest.mark.parametrize("B,V", SIZES)
def test_policy_loss(dev, B, V, dtype, keep):
    rng, x, tokens, mask = make_rows(100 + V + B, B, V, dtype, keep)
    policy_case(dev, rng, x, dtype, tokens, mask, inv_t=1.0 if V % 2 else 1.25, ent=0.0 if B % 2 else 0.02)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,V,density", [(2, 262144, 0.5), (3, 100003, 1.0), (700, 2500, 0.9), (1, 32767, 0.99)])
def test_wide_kept_sets(dev, dtype, B, V, density):
    """Masks that keep far more ids than a sampler's, up to all of them."""
    rng = np.random.default_rng(B + V)
    x = (rng.standard_normal((B, V)) * 2).astype(np.float32)
    tokens = rng.integers(0, V, B).astype(np.int32)
    mask = (rng.random((B, V)) < density).astype(np.uint8)
    mask[np.arange(B), tokens] = 1
    if dtype == "bf16":
        x = f32_to_bf16_bits(x)
    policy_case(dev, rng, x, dtype, tokens, mask, ent=0.02)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,V,counts", [
    (400, 20000, (0, 1, 2047, 2048, 2049, 20000)),       # one CTA a row, a short one's list
    (400, 40007, (1, 4095, 4096, 4097, 9000)),           # one CTA a row, a longer one's list; odd rows
    (320, 131072, (4096, 4097, 131072)),                 # the whole of a CTA's map
    (320, 131073, (8000, 8300, 131073)),                 # just beyond it: two CTAs a row
    (1, 16 * 131072 + 4099, (300,)), (1, 16 * 131072 + 4099, (900000,)),  # shares beyond the map
])
def test_kept_counts_around_the_limits(dev, dtype, B, V, counts):
    """Rows that keep as many ids as a list or a map holds, and one more; the
    rows between them are ignored. In place gives the same bits."""
    import torch

    rng = np.random.default_rng(V + len(counts))
    n = len(counts)
    at = np.linspace(0, B - 1, n).astype(np.int64)
    x = np.zeros((B, V), np.float32)
    mask = np.zeros((B, V), np.uint8)
    tokens = np.full(B, -1, np.int32)
    for r, c in zip(at, counts):
        x[r] = rng.standard_normal(V) * 2
        ids = rng.permutation(V)[:c]
        mask[r, ids] = rng.integers(1, 256, c)
        tokens[r] = ids[-1] if c else 5
    if dtype == "bf16":
        x = f32_to_bf16_bits(x)
    got = policy_case(dev, rng, x, dtype, tokens, mask, ent=0.02)
    rng = np.random.default_rng(9)
    args = dict(old=False, ref=False, kl=0.0, ent=0.02)
    apart = policy_case(dev, rng, x, dtype, tokens, mask, **args)
    rng, xd = np.random.default_rng(9), to_device(x, dtype, dev)
    onto = policy_case(dev, rng, x, dtype, tokens, mask, xd=xd, out_grad=xd, **args)
    assert onto.grad.data_ptr() == xd.data_ptr()
    assert torch.equal(onto.grad, apart.grad) and torch.equal(onto.row_loss, apart.row_loss)
    assert torch.equal(got.logp, apart.logp)


@pytest.mark.parametrize("kw", [dict(old=False), dict(ref=False), dict(weights=False), dict(kl=0.0), dict(gl=-3.0),
                                dict(ent=-0.05, entropy=True), dict(entropy=True), dict(grad=False), dict(hi=np.inf)],
                         ids=str)
def test_policy_options(dev, kw):
    rng, x, tokens, _ = make_rows(7, 6, 3001, "bf16")
    if kw.get("hi") == np.inf:
        import top_selection_row_gb300 as q

        # no upper clip: with A > 0 and rho above 1 the row is -A rho
        xd, td = to_device(x, "bf16", dev), put(dev, tokens)
        logp, _ = q.qrita_token_logprobs(xd, td)
        got = q.qrita_policy_loss(xd, td, logp - 2.0, put(dev, np.full(6, 2.0), np.float32), clip_high=np.inf)
        want = np.where((tokens >= 0) & (tokens < 3001), -2.0 * np.exp(2.0), 0.0)
        near(got.row_loss.cpu().numpy(), want, 1e-5 * np.abs(want), "row loss")
        return
    policy_case(dev, rng, x, "bf16", tokens, None, **kw)


def pref_case(dev, seed, lens, V, dtype, ref=True, weights=True, beta=0.5, ls=0.0, margin=0.0, norm=False, gl=None,
              before=0, behind=0, inv_t=1.0, ignore=0.2, edit=None, **kw):
    import top_selection_row_gb300 as q

    B = before + sum(lens) + behind
    rng, x, tokens, _ = make_rows(seed, B, V, dtype)
    if B:
        tokens[rng.random(B) < ignore] = -1
    if edit is not None:
        edit(x, tokens)
    starts = np.concatenate([[before], before + np.cumsum(lens)]).astype(np.int32)
    P = len(lens) // 2
    soft = softmaxes(x, dtype, None, tokens, inv_t) if B else []
    refv = rng.standard_normal(2 * P).astype(np.float32) if ref else None
    w = rng.uniform(0.2, 1, P).astype(np.float32) if weights else None
    xd = to_device(x, dtype, dev) if B else put(dev, np.zeros((0, V), np.float32))
    got = q.qrita_preference_loss(xd, put(dev, tokens), put(dev, starts), ref_logp=put(dev, refv), weights=put(dev, w),
                                  inv_temperature=inv_t, beta=beta, label_smoothing=ls, margin=margin, length_norm=norm,
                                  grad_loss=None if gl is None else put(dev, [gl], np.float32), **kw)
    loss, pair, ratio, seq, coef = preference(soft, starts, refv, w, beta, ls, margin, norm)
    # every row of a sequence may be off by ABS, its mean by as much
    n = np.array([1 if norm else max(1, k) for k in lens], np.float64)
    tol_seq = ABS * n + F32_ROUND * np.abs(seq)
    tol_ratio = ABS * (n[0::2] + n[1::2]) + F32_ROUND * np.abs(ratio) if P else np.zeros(0)
    near(got.seq_logp.cpu().numpy(), seq, tol_seq, "sequence logp")
    near(got.log_ratio.cpu().numpy(), ratio, tol_ratio, "log ratio")
    tol_pair = beta * tol_ratio + F32_ROUND * np.abs(pair)
    near(got.pair_loss.cpu().numpy(), pair, tol_pair, "pair loss")
    wv = (np.full(P, 1.0 / P) if P else np.zeros(0)) if w is None else w
    near(float(got.loss), loss, (wv * (tol_pair + F32_ROUND * np.abs(pair))).sum() + F32_ROUND * abs(loss), "loss")
    inside = np.zeros(B, bool)
    inside[starts[0]:starts[-1]] = True
    near_rows(got.logp.cpu().numpy(), [s.logp if i else 0.0 for s, i in zip(soft, inside)], "logp")
    if got.grad is not None and B:
        coef = coef * (1.0 if gl is None else gl)
        # the slope of a sigmoid is at most 1/4
        seq_of = np.searchsorted(starts, np.arange(B), side="right") - 1
        a_tol = np.zeros(B)
        for r in range(B):
            if inside[r] and P:
                i = seq_of[r] // 2
                scale = 1.0 if not norm else 1.0 / max(1, sum(soft[j].joins for j in range(starts[seq_of[r]], starts[seq_of[r] + 1])))
                a_tol[r] = abs(1.0 if gl is None else gl) * wv[i] * beta * beta * tol_ratio[i] / 4 * scale
        near_grad(got.grad, dtype, soft, tokens, coef, np.zeros(B), a_tol, inv_t)
        assert not got.grad[: starts[0]].any() and not got.grad[starts[-1]:].any()
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,V", [([1, 1], 1), ([1, 1], 33), ([2, 3], 1000), ([0, 4, 3, 0], 257), ([0, 0], 50),
                                    ([3, 1, 130, 7, 1, 140], 519), ([4, 2, 5, 3], 32000), ([2, 2], 50021)])
def test_preference_loss(dev, lens, V, dtype):
    pref_case(dev, V + sum(lens), lens, V, dtype)


@pytest.mark.parametrize("kw", [dict(ref=False), dict(weights=False), dict(ls=0.2), dict(ls=1.0), dict(margin=0.7), dict(norm=True),
                                dict(norm=True, ref=False, beta=2.0, margin=0.5), dict(gl=0.25), dict(inv_t=1.5),
                                dict(before=3, behind=4), dict(grad=False), dict(ignore=1.0), dict(beta=50.0)], ids=str)
def test_preference_options(dev, kw):
    pref_case(dev, 21, [4, 6, 2, 9], 777, "bf16", **kw)


@pytest.mark.parametrize("dtype,lens,V,kw", [
    ("bf16", [700, 800], 2003, {}),                    # a pair of more rows than wait for its end
    ("f32", [2, 3, 480, 300, 1, 1], 8000, dict(before=2, behind=1)),
    ("bf16", [40, 60, 55, 33, 47, 52, 61, 39], 5000, dict(norm=True)),
])
def test_preference_over_many_rows(dev, dtype, lens, V, kw):
    pref_case(dev, sum(lens), lens, V, dtype, **kw)


# rows past what a cluster holds on chip (16 x 56 KB)
@pytest.mark.parametrize("dtype,V", [("bf16", 600001), ("f32", 300007)])
def test_rows_longer_than_a_cluster_holds(dev, dtype, V):
    import torch

    import top_selection_row_gb300 as q

    rng, x, tokens, _ = make_rows(V, 5, V, dtype)
    policy_case(dev, rng, x, dtype, tokens, None, ent=0.02)
    a = rng.standard_normal(5).astype(np.float32)
    xd = to_device(x, dtype, dev)
    soft = softmaxes(x, dtype, None, tokens)
    got = q.qrita_token_logprobs_grad(xd, put(dev, tokens), put(dev, a), out_grad=xd.clone())
    near_grad(got, dtype, soft, tokens, a, np.zeros(5), np.zeros(5), 1.0)
    over = q.qrita_token_logprobs_grad(xd, put(dev, tokens), put(dev, a), out_grad=xd)
    assert torch.equal(over, got)
    pref_case(dev, V + 1, [2, 2], V, dtype)


@pytest.mark.parametrize("masked", [False, True])
def test_offsets_past_32_bits(dev, masked):
    """More than 2^31 logits in a batch: first, middle and last rows."""
    import torch

    import top_selection_row_gb300 as q

    B, V = 70000, 32000
    g = torch.Generator(device=dev).manual_seed(4)
    x = torch.empty(B, V, dtype=torch.bfloat16, device=dev)
    for a in range(0, B, 10000):
        x[a:a + 10000] = torch.randn(10000, V, generator=g, device=dev)
    t = torch.randint(0, V, (B,), generator=g, device=dev, dtype=torch.int32)
    adv = torch.randn(B, generator=g, device=dev)
    mask = None
    if masked:
        mask = torch.zeros(B, V, dtype=torch.bool, device=dev)
        mask[:, ::1000] = True
        mask[torch.arange(B, device=dev), t.long()] = True
    w = torch.ones(B, device=dev)
    got = q.qrita_policy_loss(x, t, None, adv, weights=w, mask=mask)
    rows = [0, 1, B // 2, 67108, 67109, B - 1]  # 67108 * 32000 < 2^31 < 67109 * 32000
    xs = x[rows].float().cpu().numpy()
    ts, avs = t[rows].cpu().numpy(), adv[rows].cpu().numpy()
    ms = None if mask is None else mask[rows].cpu().numpy()
    soft = softmaxes(xs, "f32", ms, ts)
    near_rows(got.logp[rows].cpu().numpy(), [s.logp for s in soft], "logp")
    near_grad(got.grad[rows], "bf16", soft, ts, -avs, np.zeros(len(rows)), np.abs(avs) * ABS, 1.0)


def test_preference_with_bad_starts_touches_nothing_else(dev):
    """Starts out of order or out of range leave everything outside the
    arguments as it was, and a later call is right."""
    import torch

    import top_selection_row_gb300 as q

    rng, x, tokens, _ = make_rows(5, 9, 301, "f32")
    xd, td = to_device(x, "f32", dev), put(dev, tokens)
    flat = torch.full((11, 301), 7.0, device=dev)
    for bad in ([-5, 3, 2, 7, 99], [9, 0, 9, 0, 9], [2**31 - 1, -(2**31), 4, 4, 4]):
        q.qrita_preference_loss(xd, td, put(dev, np.array(bad, np.int32)), out_grad=flat[1:10])
        assert (flat[0] == 7).all() and (flat[10] == 7).all()
    pref_case(dev, 5, [2, 3, 1, 3], 301, "f32")


def test_preference_calls_at_the_same_time(dev):
    """Two calls on two streams, each with pairs that could fill the device:
    rows that wait for their pair may find its rest not running."""
    import torch

    import top_selection_row_gb300 as q

    rng = np.random.default_rng(2)
    B, V = 900, 32000
    xs = [torch.from_numpy((rng.standard_normal((B, V)) * 2).astype(np.float32)).to(dev).bfloat16() for _ in range(2)]
    t = put(dev, rng.integers(0, V, B).astype(np.int32))
    starts = put(dev, np.array([0, 200, 420, 700, 900], np.int32))
    want = [q.qrita_preference_loss(x, t, starts) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        got = [q.qrita_preference_loss(x, t, starts, stream=s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for u, v in zip(a, b):
                assert torch.equal(u, v)


def test_preference_without_pairs_or_rows(dev):
    got = pref_case(dev, 3, [], 40, "f32", before=2, behind=3)
    assert float(got.loss) == 0.0 and not got.grad.any()
    got = pref_case(dev, 3, [0, 0, 0, 0], 40, "f32")
    assert got.grad.shape == (0, 40)


def test_policy_without_rows(dev):
    import top_selection_row_gb300 as q

    x = put(dev, np.zeros((0, 40), np.float32))
    e, t = put(dev, np.zeros(0, np.float32)), put(dev, np.zeros(0, np.int32))
    got = q.qrita_policy_loss(x, t, e, e)
    assert float(got.loss) == 0.0 and got.grad.shape == (0, 40)
    assert q.qrita_token_logprobs(x, t)[0].shape == (0,) and q.qrita_token_logprobs_grad(x, t, e).shape == (0, 40)


def special_rows(V, dtype):
    """Rows a mask, an overflow or a broken step leaves behind."""
    rng = np.random.default_rng(17)
    x = (rng.standard_normal((9, V)) * 3).astype(np.float32)
    low = np.float32(np.finfo(np.float32).min)
    x[0, :] = -np.inf                    # nothing
    x[1, 1:] = -np.inf                   # one token alone
    x[2, ::2] = -np.inf
    x[3, V // 2] = np.nan
    x[4, 3] = np.inf
    x[5, :] = low                        # all of the type's lowest value: uniform
    x[6, 5:] = low                       # masked that way beside ordinary logits
    x[7, :] = 1e4                        # large and equal
    x[8, 7] = 3e38                       # one token takes all
    tokens = np.array([2, 0, 1, 4, 5, 6, 2, 0, 7], np.int32)
    return (x if dtype == "f32" else f32_to_bf16_bits(x)), tokens


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [9, 1003, 40000])
@pytest.mark.parametrize("masked", [False, True])
def test_special_rows(dev, dtype, V, masked):
    import top_selection_row_gb300 as q

    x, tokens = special_rows(V, dtype)
    if dtype == "bf16":  # fp32's lowest value rounds to -inf in bf16: take bf16's own
        bits = x.copy()
        wide = widened(bits, "bf16")
        low = np.uint16(0xFF7F)
        for r, a in ((5, 0), (6, 5)):
            bits[r, a:] = low
        x = bits
        assert np.isfinite(widened(x, "bf16")[5]).all() and wide.shape == x.shape
    mask = None
    if masked:
        rng = np.random.default_rng(5)
        mask = (rng.random((9, V)) < 0.7).astype(np.uint8)
        mask[np.arange(9), tokens] = 1
        mask[3, V // 2] = 0              # the NaN is not kept
    soft = softmaxes(x, dtype, mask, tokens)
    xd, td, md = to_device(x, dtype, dev), put(dev, tokens), put(dev, mask)
    logp, ent = q.qrita_token_logprobs(xd, td, mask=md, entropy=True)
    near_rows(logp.cpu().numpy(), [s.logp for s in soft], "logp")
    near_rows(ent.cpu().numpy(), [s.entropy for s in soft], "entropy", extra=ABS)
    rng = np.random.default_rng(8)
    a, h = rng.standard_normal(9).astype(np.float32), rng.standard_normal(9).astype(np.float32)
    got = q.qrita_token_logprobs_grad(xd, td, put(dev, a), put(dev, h), mask=md)
    near_grad(got, dtype, soft, tokens, a, h, np.zeros(9), 1.0)
    policy_case(dev, rng, x, dtype, tokens, mask, ent=0.01)


@pytest.mark.parametrize("dtype,keep", FORMS)
@pytest.mark.parametrize("V,ld,ldg,shift", [(1000, 1024, 1000, 0), (1001, 1008, 1011, 0), (515, 515, 600, 1), (32000, 32064, 32000, 3)])
def test_padded_rows_and_misaligned_pointers(dev, dtype, keep, V, ld, ldg, shift):
    """Leading dimensions above V, and buffers that start `shift` elements
    into their storage: same results, and nothing outside the rows is touched."""
    import torch

    import top_selection_row_gb300 as q

    B = 6
    rng, x, tokens, mask = make_rows(V, B, V, dtype, keep)
    tight = to_device(x, dtype, dev)
    flat = torch.full((shift + B * ld,), float("nan"), dtype=tight.dtype, device=dev)
    xd = flat[shift:].view(B, ld)[:, :V]
    xd.copy_(tight)
    gflat = torch.full((shift + B * ldg + 8,), 7.0, dtype=tight.dtype, device=dev)
    gd = gflat[shift:shift + B * ldg].view(B, ldg)[:, :V]
    got = policy_case(dev, rng, x, dtype, tokens, mask, xd=xd, out_grad=gd, ent=0.01)
    assert got.grad.data_ptr() == gd.data_ptr()
    left = gflat.clone()
    left[shift:shift + B * ldg].view(B, ldg)[:, :V] = 7.0
    assert (left == 7.0).all()  # padding columns, and what lies before and behind
    # (not bit for bit what tight rows give: the order of the fp32 sums follows
    # the rows' alignment, and both are held to the oracle)
    g = rng.standard_normal(B).astype(np.float32)
    q.qrita_token_logprobs_grad(xd, put(dev, tokens), put(dev, g), mask=put(dev, mask), out_grad=gd)
    near_grad(gd, dtype, softmaxes(x, dtype, mask, tokens), tokens, g, np.zeros(B), np.zeros(B), 1.0)


@pytest.mark.parametrize("dtype,keep", FORMS)
@pytest.mark.parametrize("V", [9, 1003, 40000, 262144])
def test_gradient_over_the_logits_themselves(dev, dtype, keep, V):
    import torch

    import top_selection_row_gb300 as q

    rng, x, tokens, mask = make_rows(V + 1, 5, V, dtype, keep)
    td, md = put(dev, tokens), put(dev, mask)
    adv = put(dev, rng.standard_normal(5).astype(np.float32))
    a = to_device(x, dtype, dev)
    want = q.qrita_policy_loss(a, td, None, adv, mask=md, entropy_coef=0.1)
    b = a.clone()
    got = q.qrita_policy_loss(b, td, None, adv, mask=md, entropy_coef=0.1, out_grad=b)
    assert torch.equal(want.grad, b) and torch.equal(want.loss, got.loss)
    b = a.clone()
    q.qrita_token_logprobs_grad(b, td, adv, mask=md, out_grad=b)
    assert torch.equal(q.qrita_token_logprobs_grad(a, td, adv, mask=md), b)
    if not keep:
        starts = put(dev, np.array([0, 2, 5], np.int32))
        want = q.qrita_preference_loss(a, td, starts)
        b = a.clone()
        got = q.qrita_preference_loss(b, td, starts, out_grad=b)
        assert torch.equal(want.grad, b) and torch.equal(want.loss, got.loss)


def test_outputs_are_reused(dev):
    """out=: the tensors of an earlier call are filled again, others refused."""
    import torch

    import top_selection_row_gb300 as q

    rng, x, tokens, _ = make_rows(23, 6, 1201, "bf16")
    xd, td = to_device(x, "bf16", dev), put(dev, tokens)
    adv = put(dev, rng.standard_normal(6).astype(np.float32))
    starts = put(dev, np.array([0, 2, 6], np.int32))
    calls = [lambda **k: q.qrita_token_logprobs(xd, td, entropy=True, **k),
             lambda **k: q.qrita_policy_loss(xd, td, None, adv, entropy_coef=0.1, **k),
             lambda **k: q.qrita_preference_loss(xd, td, starts, **k)]
    for f in calls:
        want = f()
        held = type(want)(*[torch.full_like(t, 7) for t in want]) if hasattr(want, "_fields") else tuple(torch.full_like(t, 7) for t in want)
        got = f(out=held)
        for a, b, c in zip(got, want, held):
            assert a.data_ptr() == c.data_ptr() and torch.equal(a, b)
        for i in range(len(held)):
            for wrong in (held[i].double(), held[i].reshape(-1)[:0], None):
                if wrong is None and hasattr(want, "grad") and i == 1:
                    continue  # (no tensor for the gradient: one is made)
                bad = tuple(wrong if j == i else t for j, t in enumerate(held))
                with pytest.raises(ValueError):
                    f(out=bad)


def test_gradient_beside_the_logits(dev):
    """Logits and gradient as two halves of the same wider rows."""
    import torch

    import top_selection_row_gb300 as q

    V = 1003
    rng, x, tokens, _ = make_rows(19, 5, V, "bf16")
    buf = torch.zeros(5, 2 * V + 3, dtype=torch.bfloat16, device=dev)
    buf[:, :V] = to_device(x, "bf16", dev)
    got = policy_case(dev, rng, x, "bf16", tokens, None, xd=buf[:, :V], out_grad=buf[:, V + 1:2 * V + 1])
    assert torch.equal(buf[:, :V], to_device(x, "bf16", dev)) and not buf[:, V].any() and not buf[:, 2 * V + 1:].any()
    assert got.grad.data_ptr() == buf[:, V + 1:].data_ptr()
    with pytest.raises(q.QritaError):
        q.qrita_token_logprobs_grad(buf[:, :V], put(dev, tokens), got.logp, out_grad=buf[:, V - 1:2 * V - 1])


def test_binding_refusals(dev):
    import torch

    import top_selection_row_gb300 as q

    x = torch.zeros(3, 10, device=dev)
    t = torch.zeros(3, dtype=torch.int32, device=dev)
    f = torch.zeros(3, device=dev)
    ok = q.qrita_token_logprobs(x, t)[0]
    assert torch.allclose(ok, torch.full((3,), -np.log(10.0), dtype=torch.float32, device=dev))
    for bad in (x.half(), x.double()):
        with pytest.raises(TypeError):
            q.qrita_token_logprobs(bad, t)
    for args in ((x.t(), t), (x[:, ::2], t), (x, t.long()), (x, t[:2]), (x, t.cpu()), (x[0], t), (x.expand(3, 10)[:, :0], t),
                 (x[:1].expand(3, 10), t), (x, None)):
        with pytest.raises(ValueError):
            q.qrita_token_logprobs(*args)
    for m in (torch.ones(3, 10, device=dev), torch.ones(3, 9, dtype=torch.bool, device=dev), torch.ones(3, 10, dtype=torch.bool),
              torch.ones(10, 3, dtype=torch.bool, device=dev).t()):
        with pytest.raises(ValueError):
            q.qrita_token_logprobs(x, t, mask=m)
    with pytest.raises(ValueError):
        q.qrita_token_logprobs_grad(x, t)
    with pytest.raises(ValueError):
        q.qrita_token_logprobs_grad(x, t, f, out_grad=torch.zeros(3, 10, dtype=torch.bfloat16, device=dev))
    with pytest.raises(ValueError):
        q.qrita_policy_loss(x, t, f, None)
    with pytest.raises(ValueError):
        q.qrita_policy_loss(x, t, f, f.double())
    for starts in (torch.zeros(4, dtype=torch.int32, device=dev), torch.zeros(3, device=dev)):
        with pytest.raises(ValueError):
            q.qrita_preference_loss(x, t, starts)
    s = torch.zeros(3, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError):
        q.qrita_preference_loss(x, t, s, workspace=torch.zeros(8, dtype=torch.uint8, device=dev))
    for kw in (dict(inv_temperature=0.0), dict(clip_low=2.0), dict(kl_coef=-1.0)):
        with pytest.raises(q.QritaError) as err:
            q.qrita_policy_loss(x, t, f, f, **kw)
        assert err.value.code == q.EINVAL
    flat = torch.zeros(40, device=dev)  # a gradient that overlaps the logits elsewhere than at their start
    with pytest.raises(q.QritaError) as err:
        q.qrita_policy_loss(flat[:30].view(3, 10), t, f, f, out_grad=flat[10:].view(3, 10))
    assert err.value.code == q.EINVAL


def test_sampled_rollout_to_policy_step(dev):
    """The run these entry points belong to: select, draw, score the draw over
    the kept set, take a policy step, and score again."""
    import torch

    import top_selection_row_gb300 as q

    rng = np.random.default_rng(31)
    B, V = 12, 32000
    x = torch.from_numpy((rng.standard_normal((B, V)) * 2).astype(np.float32)).to(dev)
    k = torch.full((B,), 50, dtype=torch.int32, device=dev)
    p = torch.full((B,), 0.95, dtype=torch.float32, device=dev)
    mask = q.qrita_select(x, k, p)
    u = torch.from_numpy(rng.random(B).astype(np.float32)).to(dev)
    ids, probs, count, token = q.qrita_candidates(x, mask, 64, u=u)
    logp, ent = q.qrita_token_logprobs(x, token, mask=mask, entropy=True)
    at = (ids == token[:, None]).int().argmax(dim=1)
    drawn = probs[torch.arange(B, device=dev), at]
    # probs are within 4e-6 of fp64, exp(logp) within ABS
    assert torch.allclose(logp.exp(), drawn, rtol=2e-5, atol=0)
    H = torch.stack([-(r[:c] * r[:c].log()).sum() for r, c in zip(probs, count.tolist())])
    assert torch.allclose(ent, H, rtol=1e-4, atol=1e-4)
    adv = torch.ones(B, device=dev)
    step = q.qrita_policy_loss(x, token, logp, adv, ref_logp=logp, mask=mask, kl_coef=0.1)
    assert torch.allclose(step.loss, torch.tensor(-1.0, device=dev), atol=1e-5) and torch.equal(step.grad != 0, mask & (step.grad != 0))
    # a small step against the gradient raises the drawn tokens' probability
    up, _ = q.qrita_token_logprobs(x - 0.1 * step.grad, token, mask=mask)
    want = (step.grad.double() ** 2).sum(dim=1) * B * 0.1  # first order: |grad logp|^2 / B
    assert (up > logp).all() and torch.allclose((up - logp).double(), want, rtol=0.1)
    # a voided row (nothing kept, draw -1) is ignored
    mask2 = mask.clone()
    mask2[3] = False
    token2 = q.qrita_candidates(x, mask2, 64, u=u)[3]
    assert int(token2[3]) == -1
    again = q.qrita_policy_loss(x, token2, logp, adv, mask=mask2)
    assert float(again.row_loss[3]) == 0 and not again.grad[3].any() and float(again.logp[3]) == 0


def test_preference_equals_its_parts(dev):
    """The preference loss from qrita_token_logprobs' sums, and its gradient
    from qrita_token_logprobs_grad."""
    import torch

    import top_selection_row_gb300 as q

    rng, x, tokens, _ = make_rows(77, 20, 5003, "bf16")
    xd, td = to_device(x, "bf16", dev), put(dev, tokens)
    starts = put(dev, np.array([0, 7, 11, 11, 20], np.int32))
    got = q.qrita_preference_loss(xd, td, starts, beta=0.3)
    logp, _ = q.qrita_token_logprobs(xd, td)
    assert torch.allclose(got.logp, logp, atol=2 * ABS)
    seq = [logp[a:b].double().sum() for a, b in ((0, 7), (7, 11), (11, 11), (11, 20))]
    z = 0.3 * torch.stack([seq[0] - seq[1], seq[2] - seq[3]])
    assert torch.allclose(got.loss.double(), torch.nn.functional.softplus(-z).mean(), rtol=1e-5, atol=20 * ABS)
    d = -0.3 * torch.sigmoid(-z) / 2
    g = torch.cat([d[0].repeat(7), -d[0].repeat(4), -d[1].repeat(9)]).float()
    part = q.qrita_token_logprobs_grad(xd, td, g)
    assert torch.allclose(part.float(), got.grad.float(), rtol=2 * BF16_ROUND, atol=1e-7)


def test_side_stream_repeat_and_captured_graph(dev):
    """Same bits on another stream, call after call, and replayed from a
    captured graph on new inputs; two graphs with a workspace each."""
    import torch

    import top_selection_row_gb300 as q

    rng, x, tokens, _ = make_rows(13, 9, 20011, "bf16")
    _, x2, tokens2, _ = make_rows(14, 9, 20011, "bf16")
    xd, td = to_device(x, "bf16", dev), put(dev, tokens)
    adv = put(dev, rng.standard_normal(9).astype(np.float32))
    starts = put(dev, np.array([0, 4, 9], np.int32))

    def both(x, t, stream=None):
        a = q.qrita_policy_loss(x, t, None, adv, entropy_coef=0.1, stream=stream)
        b = q.qrita_preference_loss(x, t, starts, stream=stream)
        return [a.loss, a.grad, a.row_loss, a.logp, b.loss, b.grad, b.pair_loss, b.logp]

    def same(a, b):
        return all(torch.equal(torch.nan_to_num(u), torch.nan_to_num(v)) for u, v in zip(a, b))

    want, want2 = both(xd, td), both(to_device(x2, "bf16", dev), put(dev, tokens2))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        got = both(xd, td, side)
        side.synchronize()
        assert same(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both(xd, td)
    graph.replay()
    torch.cuda.synchronize()
    assert same(held, want)
    xd.copy_(to_device(x2, "bf16", dev))
    td.copy_(put(dev, tokens2))
    graph.replay()
    torch.cuda.synchronize()
    assert same(held, want2)


def test_temporaries_of_a_call_on_another_stream(dev):
    """Inputs that are dropped as soon as the call returns, on a stream that is
    behind: their memory is not handed out again before the kernels have run."""
    import torch

    import top_selection_row_gb300 as q

    rng, x, tokens, _ = make_rows(3, 8, 32000, "bf16")
    xd, td = to_device(x, "bf16", dev), put(dev, tokens)
    adv = put(dev, rng.standard_normal(8).astype(np.float32))
    starts = put(dev, np.array([0, 4, 8], np.int32))
    want = [q.qrita_token_logprobs(xd, td)[0], q.qrita_token_logprobs_grad(xd, td, adv),
            q.qrita_policy_loss(xd, td, None, adv).grad, q.qrita_preference_loss(xd, td, starts).grad]
    side, work = torch.cuda.Stream(), torch.randn(4096, 4096, device=dev)
    calls = [lambda v, t, a: q.qrita_token_logprobs(v, t, stream=side)[0],
             lambda v, t, a: q.qrita_token_logprobs_grad(v, t, a, stream=side),
             lambda v, t, a: q.qrita_policy_loss(v, t, None, a, stream=side).grad,
             lambda v, t, a: q.qrita_preference_loss(v, t, starts.clone(), stream=side).grad]
    torch.cuda.synchronize()
    for f, w in zip(calls, want):
        v, t, a = xd.clone(), td.clone(), adv.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):
                work @ work  # the side stream is busy for a few milliseconds
        got = f(v, t, a)
        del v, t, a
        for _ in range(8):  # would land in their memory, were it free
            torch.full_like(xd, 9), torch.full_like(td, 9), torch.full_like(adv, 9)
        torch.cuda.synchronize()
        assert torch.equal(got, w)


def test_beside_matrix_products_of_another_stream(dev):
    """Rows held in tensor memory while another stream's products take theirs."""
    import torch

    import top_selection_row_gb300 as q

    rng, x, tokens, _ = make_rows(5, 64, 200000, "bf16")
    xd, td = to_device(x, "bf16", dev), put(dev, tokens)
    adv = put(dev, rng.standard_normal(64).astype(np.float32))
    want = q.qrita_policy_loss(xd, td, None, adv)
    a = torch.randn(4096, 4096, device=dev, dtype=torch.bfloat16)
    product = a @ a
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(20):
        with torch.cuda.stream(side):
            b = a @ a
        got.append(q.qrita_policy_loss(xd, td, None, adv))
    torch.cuda.synchronize()
    assert torch.equal(b, product)
    for g in got:
        assert torch.equal(g.loss, want.loss) and torch.equal(g.grad, want.grad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_against_differences(dev, dtype):
    """The gradient of the loss against differences of the loss itself along
    random directions. logits move by eps in fp32 rows (bf16 rows by steps
    their type holds); the loss is off by at most about 1e-5 / (2 eps)."""
    import torch

    import top_selection_row_gb300 as q

    rng = np.random.default_rng(41)
    B, V = 4, 300
    # multiples of 1/8 below 8: bf16 holds them and their moves by 1/16 exactly
    x = torch.from_numpy((np.round(rng.standard_normal((B, V)) * 8) / 8).clip(-7, 7).astype(np.float32)).to(dev)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x = x.to(dt)
    t = put(dev, rng.integers(0, V, B).astype(np.int32))
    starts = put(dev, np.array([0, 2, 4], np.int32))
    old = put(dev, (rng.standard_normal(B) * 0.01 - 5).astype(np.float32))
    adv = put(dev, rng.standard_normal(B).astype(np.float32))
    eps = 1.0 / 32
    for f in (lambda v: q.qrita_policy_loss(v, t, old, adv, ref_logp=old, clip_low=1.0, clip_high=np.inf, kl_coef=0.3, entropy_coef=0.2),
              lambda v: q.qrita_preference_loss(v, t, starts, beta=0.7)):
        g = f(x).grad.double()
        for trial in range(4):
            d = torch.from_numpy(rng.choice([-1.0, 0.0, 1.0], (B, V))).to(dev)
            up, dn = ((x.double() + s * eps * d).to(dt) for s in (1, -1))
            assert torch.equal(up.double() - x.double(), eps * d)
            num = (f(up).loss.double() - f(dn).loss.double()) / (2 * eps)
            want = (g * d).sum()
            # third-order term: eps^2 / 6 of a third derivative of order |loss|; bf16 gradients round
            tol = 2e-3 * (1 + abs(float(want))) + (BF16_ROUND * float((g * d).abs().sum()) if dtype == "bf16" else 0)
            assert abs(float(num - want)) < tol
