"""How far logp and H are from their definitions, at the accuracy include/qrita.h
states, which is finer than fp32 holds of a logp near -20.

A ratio and a KL term see logp before its rounding to fp32. With a reference
that lies q = 2^-6 above the exact logp, kl = e^q - 1 - q gives q, and so logp,
back to 2^-23 of kl, which is q 2^-24 = 1e-9: that is how logp is read here.

Bounds, from the arithmetic: a weight is off by at most 2^-22 (the instruction)
and 2^-24 times its exponent's logarithm (one rounding of the exponent); a
thread's compensated sum of groups, a group's tree of at most 5 additions and
the merges by at most 6 * 2^-24: log S, and so logp, is off by no more than
  BOUND(E) = 2^-22 + 2^-24 (6 + E),  E the mean of |log p_j / p_max| under p.
These errors are spread over many weights with either sign and their mean is
taken back: the root mean square over rows, and the mean, stay below RMS = 1e-7.
H = log S + E exactly, E a quotient of two such sums: twice the bound, and
RMS (1 + E).
"""

import numpy as np
import pytest

from test_gpu_losses import dev  # noqa: F401

pytestmark = pytest.mark.gpu

RMS = 1e-7
HALF = 2.0 ** -24


def bound(E):
    return 2.0 ** -22 + HALF * (6 + E)


def exact(x, tokens, inv_t, mask=None):
    """(logp, H, E) of every row in fp64."""
    import torch

    logp, H, E = [], [], []
    for a in range(0, x.shape[0], 32):
        u = x[a:a + 32].double() * inv_t
        if mask is not None:
            u = u.masked_fill(~mask[a:a + 32], -np.inf)
        y = u - u.amax(dim=1, keepdim=True)
        e = y.exp()
        S = e.sum(dim=1)
        mean = -(e * y.clamp(min=-1e6)).sum(dim=1) / S
        logp.append(y.gather(1, tokens[a:a + 32, None].long())[:, 0] - S.log())
        H.append(S.log() + mean)
        E.append(mean)
    return [torch.cat(v).cpu().numpy() for v in (logp, H, E)]


def check(x, tokens, inv_t=1.0, mask=None, mean=RMS):
    import torch

    import top_selection_row_gb300 as q

    want, H, E = exact(x, tokens, inv_t, mask)
    ref = torch.from_numpy((want + 2.0 ** -6).astype(np.float32)).to(x.device)
    zero = torch.zeros_like(ref)
    for form in (dict(grad=False), dict(), dict(grad=False, entropy=True)):  # each of the kernels' sums
        got = q.qrita_policy_loss(x, tokens, ref, zero, ref_logp=ref, mask=mask, inv_temperature=inv_t, **form)
        kl = got.kl.cpu().numpy().astype(np.float64)
        d = np.full_like(kl, 2.0 ** -6)
        for _ in range(6):  # e^d - 1 - d = kl, by Newton
            d -= (np.expm1(d) - d - kl) / np.expm1(d)
        err = ref.cpu().numpy().astype(np.float64) - d - want
        assert (np.abs(err) <= bound(E) + 2e-9).all(), (form, np.abs(err).max(), bound(E).max())
        assert np.sqrt((err ** 2).mean()) <= RMS and abs(err.mean()) <= mean, (form, np.sqrt((err ** 2).mean()), err.mean())
        # the fp32 value given out is that, rounded
        out = got.logp.cpu().numpy().astype(np.float64)
        assert (np.abs(out - want) <= bound(E) + HALF * np.abs(want) * 1.01).all()


def logits(dev, seed, B, V, dtype, scale=2.0):
    import torch

    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn(B, V, generator=g, device=dev) * scale
    where = torch.randint(0, V, (B, 8), generator=g, device=dev)
    x.scatter_add_(1, where, 5 + 2 * torch.randn(B, 8, generator=g, device=dev))
    x = x.to(torch.float32 if dtype == "f32" else torch.bfloat16)
    return g, x


DTYPES = pytest.mark.parametrize("dtype", ["f32", "bf16"])


@DTYPES
@pytest.mark.parametrize("inv_t", [1.0, 0.71875, 0.75, 1.25, 1.4375])
@pytest.mark.parametrize("B,V", [(256, 3001), (128, 50021), (40, 128256)])
def test_rare_tokens_at_any_temperature(dev, dtype, inv_t, B, V):
    """The least likely token of each row: what the temperature's own rounding
    would move the most."""
    _, x = logits(dev, V, B, V, dtype)
    check(x, x.float().argmin(dim=1).int(), inv_t)


@DTYPES
@pytest.mark.parametrize("span", [0.25, 1.0, 4.0, 20.0])
@pytest.mark.parametrize("B,V", [(160, 50021), (320, 128256)])
def test_rows_that_rise_slowly(dev, dtype, span, B, V):
    """Ascending logits over a range of `span`: a thread meets a new maximum at
    nearly each of its groups."""
    import torch

    x = (torch.arange(V, device=dev, dtype=torch.float64) * (span / V)).expand(B, V)
    x = (x + torch.linspace(0, 0.3, B, device=dev, dtype=torch.float64)[:, None]).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    check(x.contiguous(), torch.arange(B, device=dev, dtype=torch.int32) * (V // B))


def check_entropies(x, inv_t=1.0, mask=None):
    """H against its definition: beside the roundings of the values given out (half
    a step of either sign: three times their mean's standard error), no bias is left
    above 5e-8 in log S and 2.7e-8 of E (what the exponential's mean error differs
    by within an octave of the maximum)."""
    import torch

    import top_selection_row_gb300 as q

    B = x.shape[0]
    t = x.float().masked_fill(~mask, -np.inf).argmax(dim=1) if mask is not None else x.float().argmax(dim=1)
    _, H, E = exact(x, t, inv_t, mask)
    outs = [q.qrita_token_logprobs(x, t.int(), mask=mask, inv_temperature=inv_t, entropy=True)[1],
            q.qrita_policy_loss(x, t.int(), None, torch.zeros(B, device=x.device), mask=mask, inv_temperature=inv_t, entropy=True).entropy]
    for got in outs:
        err = got.cpu().numpy().astype(np.float64) - H
        assert (np.abs(err) <= 2 * bound(E) + HALF * H * 1.01).all(), np.abs(err).max()
        noise = 3 * HALF * np.sqrt((H ** 2).mean() / 3 / B)
        assert abs(err.mean()) <= 5e-8 + 2.7e-8 * E.mean() + noise, (err.mean(), E.mean())


@DTYPES
@pytest.mark.parametrize("B,V,scale,inv_t", [(512, 3001, 0.5, 1.0), (256, 50021, 2.0, 1.0), (256, 50021, 2.0, 1.4375), (64, 262144, 2.0, 1.0),
                                             (700, 32000, 4.0, 0.71875), (300, 32000, 0.0, 1.0)])
def test_entropies(dev, dtype, B, V, scale, inv_t):
    _, x = logits(dev, V + B, B, V, dtype, scale)
    check_entropies(x, inv_t)


@DTYPES
@pytest.mark.parametrize("far", [-60.0, -7.0, 3.0, 23.0, 61.0, 79.0, 84.0])
def test_ratios_and_kl_terms_far_from_one(dev, dtype, far):
    """e^d of a d that fp32 holds to |d| 2^-24 only: the ratio, the KL term, their
    sum and the gradient's entry of the token (p_t is near 0) see d as a pair. Off by
    logp's own bound, an exponential's rounding of 2^-22 and a product's and the
    output's 2^-23, relative to the terms."""
    import torch

    import top_selection_row_gb300 as q

    B, V = 200, 5003
    g, x = logits(dev, 71, B, V, "f32")
    t = torch.randint(0, V, (B,), generator=g, device=dev, dtype=torch.int32)
    x[torch.arange(B, device=dev), t.long()] = torch.linspace(-25, -22, B, device=dev)
    x = x.to(torch.float32 if dtype == "f32" else torch.bfloat16)
    want, _, E = exact(x, t, 1.0)
    near = torch.from_numpy((want - far).astype(np.float32)).to(dev)
    there = torch.from_numpy((want + far).astype(np.float32)).to(dev)
    d, k = want - near.cpu().numpy().astype(np.float64), there.cpu().numpy().astype(np.float64) - want
    one = torch.full((B,), -1.0, device=dev)
    coef = float(np.float32(1e-3))
    tol = bound(E) + 2.0 ** -21
    got = q.qrita_policy_loss(x, t, near, one, ref_logp=there, clip_low=1.0, weights=-one, kl_coef=coef, out_grad=torch.empty_like(x))
    rho, kl = np.exp(d), np.expm1(k) - k
    assert (np.abs(got.kl.cpu().numpy() - kl) <= tol * (np.exp(k) + np.abs(k) + 1)).all()
    row = rho + coef * kl
    assert (np.abs(got.row_loss.cpu().numpy() - row) <= tol * (rho + coef * (np.exp(k) + np.abs(k) + 1))).all()
    at = got.grad[torch.arange(B, device=dev), t.long()].double().cpu().numpy()
    slope = (rho - coef * np.expm1(k)) * -np.expm1(want)
    assert (np.abs(at - slope) <= tol * (rho + coef * (np.exp(k) + 1)) + (2.0 ** -8 * np.abs(slope) if dtype == "bf16" else 0)).all()


@pytest.mark.parametrize("z", [-80.0, -9.0, 0.5, 9.0, 30.0, 80.0])
def test_slopes_of_distant_pairs(dev, z):
    """Pairs far apart: the sigmoid's slope, of a z that fp32 holds to |z| 2^-24
    only, in the gradient's entry of a token whose probability is near 0."""
    import torch

    import top_selection_row_gb300 as q

    P, V = 64, 3001
    g, x = logits(dev, 5, 2 * P, V, "f32")
    t = torch.randint(0, V, (2 * P,), generator=g, device=dev, dtype=torch.int32)
    x[torch.arange(2 * P, device=dev), t.long()] = -22.0
    want, _, E = exact(x, t, 1.0)
    ref = np.zeros(2 * P)
    ref[0::2] = want[0::2] - want[1::2] - np.linspace(z, z * 1.01, P)
    ref = torch.from_numpy(ref.astype(np.float32)).to(dev)
    got = q.qrita_preference_loss(x, t, torch.arange(2 * P + 1, device=dev, dtype=torch.int32), ref_logp=ref, beta=1.0,
                                  weights=torch.ones(P, device=dev))
    r = ref.cpu().numpy().astype(np.float64)
    zz = (want[0::2] - r[0::2]) - (want[1::2] - r[1::2])
    slope = -1 / (1 + np.exp(zz)) * -np.expm1(want[0::2])
    at = got.grad[torch.arange(0, 2 * P, 2, device=dev), t[0::2].long()].double().cpu().numpy()
    assert (np.abs(at / slope - 1) <= 2 * bound(E).max() + 2.0 ** -21).all(), np.abs(at / slope - 1).max()


def test_a_beta_beyond_fp32(dev):
    """Slopes of pairs under a beta of 1e39: 0 where z saturates, beta's own value
    times a small weight where it does not."""
    import torch

    import top_selection_row_gb300 as q

    x = torch.zeros(4, 100, device=dev)
    x[2, 5] = 3.0
    t = torch.full((4,), 5, dtype=torch.int32, device=dev)
    w = torch.tensor([1e-4, 1.0], device=dev)
    got = q.qrita_preference_loss(x, t, torch.arange(5, device=dev, dtype=torch.int32), weights=w, beta=1e39)
    assert abs(float(got.grad[0, 5]) / (-0.5 * 1e35 * 0.99) - 1) < 1e-5  # (z = 0)
    assert abs(float(got.pair_loss[0]) - np.log(2)) < 1e-6 and float(got.pair_loss[1]) == 0
    assert not got.grad[2:].any()


@DTYPES
@pytest.mark.parametrize("warm", [True, False])
@pytest.mark.parametrize("B,V", [(700, 128256), (64, 262144), (1000, 3001), (16, 32000)])
def test_ordinary_tokens(dev, dtype, B, V, warm):
    """The mean over rows adds up in a sequence's sum. The instruction's own is 0
    to 5e-8 from octave to octave, and 2.5e-8 of it are taken back; a group of 32
    logits takes the low part of c = log2(e) inv_t by its largest, which leaves c's
    error in fp32 times their mean distance below it under p: at most 1.83 (that of
    31 logits 3 below one)."""
    import torch

    g, x = logits(dev, V + 1, B, V, dtype)
    noise = torch.rand(B, V, generator=g, device=dev).clamp_(min=1e-30).log_().neg_().log_().neg_()
    inv_t = 1.25 if not warm else 1.0 if V % 2 else 0.75
    c = np.log2(np.e) * inv_t
    off = abs(float(np.float32(c)) / c - 1)  # (3e-9 at 1.25)
    check(x, (x.float() + noise).argmax(dim=1).int(), inv_t, mean=2.5e-8 + 1.83 * off + 3 * 5e-8 / np.sqrt(B))


@DTYPES
@pytest.mark.parametrize("lead", [10.0, 14.0])
@pytest.mark.parametrize("B,V", [(700, 128256), (100, 50021)])
def test_a_token_that_outweighs_its_row(dev, dtype, lead, B, V):
    """Most of a row's weight in one token (p from 0.15 to 0.9): every other group
    of its thread's share is added to a sum near that token's weight."""
    import torch

    g, x = logits(dev, V + 2, B, V, "f32", 0.5)
    t = torch.randint(0, V, (B,), generator=g, device=dev, dtype=torch.int32)
    x = torch.randn(B, V, generator=g, device=dev) * 0.5
    x[torch.arange(B, device=dev), t.long()] = lead
    check(x.to(torch.float32 if dtype == "f32" else torch.bfloat16), t)


@DTYPES
def test_rows_of_few_values(dev, dtype):
    """Uniform rows, and one token above rows of one other value: every weight has
    the same error, so only the bound holds of these."""
    import torch

    import top_selection_row_gb300 as q

    B, V = 64, 50021
    x = torch.full((B, V), 3.0, device=dev)
    t = torch.arange(B, device=dev, dtype=torch.int32) * 700
    x[torch.arange(B, device=dev), t.long()] += torch.arange(B, device=dev) * 0.25
    x = x.to(torch.float32 if dtype == "f32" else torch.bfloat16)
    want, _, E = exact(x, t, 1.0)
    for ent in (False, True):
        got = q.qrita_token_logprobs(x, t, entropy=ent)[0].cpu().numpy().astype(np.float64)
        assert (np.abs(got - want) <= bound(E) + HALF * np.abs(want) * 1.01).all()


@DTYPES
@pytest.mark.parametrize("B,V,density", [(128, 50021, 0.001), (128, 50021, 0.5), (500, 30000, 0.03), (24, 262144, 0.3)])
def test_kept_sets(dev, dtype, B, V, density):
    import torch

    g, x = logits(dev, V + 3, B, V, dtype)
    mask = torch.rand(B, V, generator=g, device=dev) < density
    t = torch.where(mask, torch.rand(B, V, generator=g, device=dev), -1.0).argmax(dim=1)
    for inv_t in (1.0, 1.4375):
        check(x, t.int(), inv_t, mask)
    check_entropies(x, 1.0, mask)


@pytest.mark.parametrize("ref", [False, True])
@pytest.mark.parametrize("ent", [0.0, 0.01])
def test_row_losses_are_rounded_once(dev, ref, ent):
    """Rows of one token (logp is exactly 0): a row's loss is within half a step of
    the formula's, an exponential's error (a step of e^d - 1) and the KL term's
    three roundings apart."""
    import torch

    import top_selection_row_gb300 as q

    B = 5000
    g = torch.Generator(device=dev).manual_seed(9)
    adv = torch.randn(B, generator=g, device=dev)
    old = torch.randn(B, generator=g, device=dev) * 0.3
    there = torch.randn(B, generator=g, device=dev) * 0.5 if ref else None
    got = q.qrita_policy_loss(torch.zeros(B, 1, device=dev), torch.zeros(B, dtype=torch.int32, device=dev), old, adv, ref_logp=there,
                              clip_low=0.2, clip_high=0.28, kl_coef=0.05, entropy_coef=ent, grad=False)
    a, d = adv.double().cpu().numpy(), -old.double().cpu().numpy()
    rho = np.exp(d)
    surrogate = np.maximum(-a * rho, -a * np.clip(rho, 1 - 0.2, 1 + 0.28))
    kl = 0.0
    if ref:
        k = there.double().cpu().numpy()
        kl = 0.05 * (np.expm1(k) - k)
    row = surrogate + kl
    err = np.abs(got.row_loss.double().cpu().numpy() - row)
    edge = np.minimum(np.abs(rho - 0.8), np.abs(rho - 1.28)) < 1e-6
    tol = HALF * np.abs(row) * 1.01 + 2.0 ** -23 * np.abs(a) * np.abs(np.expm1(d)) + 3 * 2.0 ** -23 * np.abs(kl)
    # (below rho = 1/2 the exponential itself is taken, off by two steps)
    tol = tol + np.where(rho < 0.51, 2.0 ** -22 * np.abs(a) * rho, 0.0)
    assert (err <= tol)[~edge].all(), ((err - tol)[~edge].max(), np.argmax(np.where(edge, 0, err - tol)))
    assert abs(float(got.loss) - row.mean()) <= HALF * (abs(row.mean()) + np.abs(row).mean())


@DTYPES
@pytest.mark.parametrize("scale", [0.25, 0.5, 1.0])
@pytest.mark.parametrize("B,V", [(3000, 3001), (1000, 20011)])
def test_broad_rows_have_no_bias(dev, dtype, scale, B, V):
    """Rows whose weight is spread over logits near their maximum, at a temperature
    that fp32 holds to 3e-9: the bounds of test_ordinary_tokens."""
    import torch

    g = torch.Generator(device=dev).manual_seed(V)
    x = (torch.randn(B, V, generator=g, device=dev) * scale).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    t = torch.randint(0, V, (B,), generator=g, device=dev, dtype=torch.int32)
    check(x, t, 1.25, mean=2.5e-8 + 1.83 * 3.2e-9 + 3 * 5e-8 / np.sqrt(B))
