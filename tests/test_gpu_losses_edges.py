"""Losses at the edges of their definitions: ratios and KL terms far from 1,
rows that a weight hides, values that are not finite beside tokens that are not
kept. Against the fp64 oracle; the tolerances are test_gpu_losses' own (ABS of
logp, so ABS of an exponential of it relatively)."""

import numpy as np
import pytest

from oracle import dentropy, dlogp, policy_row
from parity_helpers import to_device
from test_gpu_losses import ABS, F32_ROUND, dev, make_rows, near, near_grad, near_rows, put, softmaxes  # noqa: F401

pytestmark = pytest.mark.gpu

FORMS = [("f32", 0, 300), ("bf16", 0, 300), ("f32", 12, 300), ("bf16", 0, 40000), ("f32", 12, 40000)]


def policy(dev, x, dtype, tokens, mask, old, ref, adv, w, kl=0.0, ent=0.0, lo=0.2, hi=0.3, gl=None):
    """qrita_policy_loss against the oracle; returns the call's result."""
    import top_selection_row_gb300 as q

    f = np.float32
    B = len(tokens)
    old, adv, w = (np.asarray(v, f) for v in (old, adv, w))
    ref = None if ref is None else np.asarray(ref, f)
    got = q.qrita_policy_loss(to_device(x, dtype, dev), put(dev, tokens), put(dev, old), put(dev, adv), ref_logp=put(dev, ref),
                              weights=put(dev, w), mask=put(dev, mask), clip_low=lo, clip_high=hi, kl_coef=kl, entropy_coef=ent,
                              grad_loss=None if gl is None else put(dev, [gl], f))
    soft = softmaxes(x, dtype, mask, tokens)
    rows, kls, a, h, size = (np.zeros(B) for _ in range(5))
    for r, s in enumerate(soft):
        rows[r], kls[r], da, dh = policy_row(s, float(old[r]), None if ref is None else float(ref[r]), float(adv[r]), lo, hi, kl, ent)
        if s.joins:
            wr = float(w[r]) * (1.0 if gl is None else gl)
            a[r], h[r] = wr * da, wr * dh
            eq = 0.0 if ref is None else kl * float(np.exp(float(ref[r]) - s.logp))
            size[r] = abs(float(adv[r])) * float(np.exp(s.logp - float(old[r]))) + eq + kl + abs(ent)
    with np.errstate(over="ignore"):
        rows32, kl32 = rows.astype(f), kls.astype(f)  # (a value beyond fp32 is an infinity)
    near(got.row_loss.cpu().numpy(), np.where(np.isinf(rows32), rows32, rows), 2 * ABS * size + 2 * F32_ROUND * np.abs(rows), "row loss")
    kl_size = np.array([1 + (0.0 if ref is None or not s.joins else np.exp(float(ref[r]) - s.logp)) for r, s in enumerate(soft)])
    # (the output's own rounding: half a step of 699 is 3e-5)
    near(got.kl.cpu().numpy(), np.where(np.isinf(kl32), kl32, kls), 2 * ABS * kl_size + 2 * F32_ROUND * np.abs(np.where(np.isinf(kl32), 0, kls)), "kl")
    used = w != 0
    loss = float((w[used].astype(np.float64) * rows[used]).sum())
    near(float(got.loss), loss, float((np.abs(w[used]) * 2 * ABS * (size + np.abs(rows))[used]).sum()) + 2 * F32_ROUND * abs(loss), "loss")
    near_grad(got.grad, dtype, soft, tokens, a, h, np.abs(w * (1.0 if gl is None else gl)) * 2 * ABS * size, 1.0)
    return got


def rows_of(seed, B, V, dtype, keep):
    rng, x, tokens, mask = make_rows(seed, B, V, dtype, keep)
    if mask is not None:
        mask[1, tokens[1]] = 1  # (make_rows leaves these two without their token)
        mask[2, tokens[2]] = 1
    tokens[:] = np.where((tokens < 0) | (tokens >= V), 1, tokens)
    if mask is not None:
        mask[np.arange(B), tokens] = 1
    base = np.array([s.logp for s in softmaxes(x, dtype, mask, tokens)])
    return rng, x, tokens, mask, base


@pytest.mark.parametrize("dtype,keep,V", FORMS)
def test_an_advantage_of_zero_takes_nothing_from_any_ratio(dev, dtype, keep, V):
    """rho = e^d leaves fp32 above d = 88.7; 0 times it is 0, not NaN."""
    _, x, tokens, mask, base = rows_of(11, 9, V, dtype, keep)
    far = np.array([0.0, 79.0, 81.0, 88.5, 89.0, 120.0, 180.0, 360.0, 650.0])
    adv = np.zeros(9)
    adv[0] = 1.0
    got = policy(dev, x, dtype, tokens, mask, base - far, None, adv, np.ones(9), ent=0.01)
    assert np.isfinite(float(got.loss))
    assert not policy(dev, x, dtype, tokens, mask, base - far, None, adv, np.ones(9)).grad[1:].any()


@pytest.mark.parametrize("dtype,keep,V", FORMS)
def test_large_ratios_times_small_advantages(dev, dtype, keep, V):
    """-A rho is within fp32 where rho alone is not; so is its gradient, and
    the one that a weight brings back."""
    _, x, tokens, mask, base = rows_of(12, 8, V, dtype, keep)
    far = np.array([70.0, 81.0, 85.0, 90.0, 100.0, 110.0, 95.0, 88.0])
    adv = -np.array([1e-3, 1e-3, 1e-2, 1e-10, 1e-20, 1e-25, 1e-30, 1.0])
    w = np.array([1.0, 0.5, 1e-3, 1e-3, 1.0, 1e-4, 1e-6, 1e-6])
    policy(dev, x, dtype, tokens, mask, base - far, None, adv, w)


@pytest.mark.parametrize("dtype,keep,V", FORMS)
def test_large_kl_terms(dev, dtype, keep, V):
    """kl_coef e^q is within fp32 where e^q alone is not."""
    _, x, tokens, mask, base = rows_of(13, 8, V, dtype, keep)
    q = np.array([-700.0, -90.0, 0.0, 79.0, 81.0, 88.0, 90.0, 93.0])
    policy(dev, x, dtype, tokens, mask, base, base + q, np.ones(8), np.full(8, 0.01), kl=1e-4)


@pytest.mark.parametrize("dtype,keep,V", FORMS)
def test_gradients_of_rows_with_a_weight_of_zero(dev, dtype, keep, V):
    """A padded batch: rows of weight 0 whose tokens and reference values are
    fillers, so that their ratios and KL terms leave fp32, have no gradient."""
    import top_selection_row_gb300 as q

    rng, x, tokens, mask, base = rows_of(14, 8, V, dtype, keep)
    f = np.float32
    old, ref, w = base.copy(), base.copy(), np.ones(8)
    w[3:] = 0.0
    old[3:], ref[3:] = base[3:] - 150.0, base[3:] + 150.0
    adv = rng.standard_normal(8)
    got = q.qrita_policy_loss(to_device(x, dtype, dev), put(dev, tokens), put(dev, old, f), put(dev, adv, f), ref_logp=put(dev, ref, f),
                              weights=put(dev, w, f), mask=put(dev, mask), kl_coef=0.1)
    assert not got.grad[3:].any() and got.grad[[0, 2]].any(dim=1).all()  # (row 1 keeps its token alone: 0)


@pytest.mark.parametrize("dtype,keep,V", FORMS)
def test_losses_of_rows_with_a_weight_of_zero(dev, dtype, keep, V):
    """The same batch's loss is that of the rows that count; with a NaN among the
    kept logits of a row of weight 0 it is NaN, as the row contract says."""
    rng, x, tokens, mask, base = rows_of(15, 8, V, dtype, keep)
    old, ref, w = base - 0.1, base + 0.2, np.ones(8)
    w[3:] = 0.0
    old[3:], ref[3:] = base[3:] - 150.0, base[3:] + 150.0
    adv = rng.standard_normal(8)
    adv[4] = -1.0  # (no clip: its row loss is beyond fp32 by its ratio too)
    got = policy(dev, x, dtype, tokens, mask, old, ref, adv, w, kl=0.1)
    assert np.isinf(got.row_loss[3:].cpu().numpy()).all() and np.isfinite(float(got.loss))
    x[5, tokens[5]] = 0x7FC0 if dtype == "bf16" else np.nan
    import top_selection_row_gb300 as q

    f = np.float32
    got = q.qrita_policy_loss(to_device(x, dtype, dev), put(dev, tokens), put(dev, old, f), put(dev, adv, f), ref_logp=put(dev, ref, f),
                              weights=put(dev, w, f), mask=put(dev, mask), kl_coef=0.1)
    assert np.isnan(float(got.loss)) and got.grad[5].isnan().any()


def test_preference_pairs_with_a_weight_of_zero(dev):
    """A pair whose loss leaves fp32 and has no weight adds nothing."""
    import torch

    import top_selection_row_gb300 as q

    _, x, tokens, _, _ = rows_of(16, 4, 300, "f32", 0)
    xd, td, starts = put(dev, x), put(dev, tokens), put(dev, np.arange(5, dtype=np.int32))
    far = np.zeros(4, np.float32)
    far[2], far[3] = 3e38, -3e38
    kw = dict(ref_logp=put(dev, far), beta=10.0)
    got = q.qrita_preference_loss(xd, td, starts, weights=put(dev, np.array([1, 0], np.float32)), **kw)
    one = q.qrita_preference_loss(xd[:2], td[:2], starts[:3], ref_logp=kw["ref_logp"][:2], weights=put(dev, np.ones(1, np.float32)), beta=10.0)
    assert np.isinf(float(got.pair_loss[1])) and torch.equal(got.loss, one.loss)
    assert torch.equal(got.grad[:2], one.grad) and not got.grad[2:].any()


@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("dtype,V,keep", [("f32", 9, 4), ("bf16", 1003, 40), ("f32", 40000, 300), ("bf16", 40000, 20000)])
def test_nan_or_infinity_beside_a_token_of_no_probability(dev, bad, dtype, V, keep):
    """NaN or +inf among the kept logits makes the row NaN wherever its token
    is: kept, not kept, or at -inf. Row 3 holds it outside the kept set."""
    import top_selection_row_gb300 as q

    rng = np.random.default_rng(V)
    x = (rng.standard_normal((5, V)) * 2).astype(np.float32)
    mask = np.zeros((5, V), np.uint8)
    tokens = np.zeros(5, np.int32)
    for r in range(5):
        ids = rng.permutation(V)[:keep]
        mask[r, ids] = 1
        tokens[r] = ids[0]
        if r < 3:
            x[r, ids[1]] = bad
    mask[0, tokens[0]] = 0
    x[2, tokens[2]] = -np.inf
    mask[3, tokens[3] - 1] = 0
    x[3, tokens[3] - 1] = bad
    mask[4, tokens[4]] = 0
    if dtype == "bf16":
        from workloads import f32_to_bf16_bits

        x = f32_to_bf16_bits(x)
    soft = softmaxes(x, dtype, mask, tokens)
    assert np.isnan([s.logp for s in soft[:3]]).all() and np.isfinite(soft[3].logp) and soft[4].logp == -np.inf
    xd, td, md = to_device(x, dtype, dev), put(dev, tokens), put(dev, mask)
    logp, ent = q.qrita_token_logprobs(xd, td, mask=md, entropy=True)
    near_rows(logp.cpu().numpy(), [s.logp for s in soft], "logp")
    near_rows(ent.cpu().numpy(), [s.entropy for s in soft], "entropy", extra=ABS)
    near_rows(q.qrita_token_logprobs(xd, td, mask=md)[0].cpu().numpy(), [s.logp for s in soft], "logp alone")
    a, h = rng.standard_normal(5).astype(np.float32), rng.standard_normal(5).astype(np.float32)
    got = q.qrita_token_logprobs_grad(xd, td, put(dev, a), put(dev, h), mask=md)
    near_grad(got, dtype, soft, tokens, a, h, np.zeros(5), 1.0)
    step = q.qrita_policy_loss(xd, td, None, put(dev, a), mask=md)
    rows = step.row_loss.cpu().numpy()
    assert np.isnan(rows[:3]).all() and np.isfinite(rows[3:]).all() and np.isnan(float(step.loss))
    near_grad(step.grad, dtype, soft, tokens, -a / 5, np.zeros(5), np.zeros(5), 1.0)


@pytest.mark.parametrize("shape", [(6,), (3, 2), (1, 6), (6, 1)])
def test_outputs_have_their_own_shape(dev, shape):
    """[B], whatever the shape of the B values given."""
    import torch

    import top_selection_row_gb300 as q

    rng, x, tokens, _ = make_rows(33, 6, 300, "f32")
    v = put(dev, rng.standard_normal(6).astype(np.float32))
    xd, td = put(dev, x), put(dev, tokens)
    want = q.qrita_policy_loss(xd, td, v, v, ref_logp=v, weights=v, entropy=True)
    w = v.view(shape)
    got = q.qrita_policy_loss(xd, td.view(shape), w, w, ref_logp=w, weights=w, entropy=True)
    for a, b in zip(got, want):
        assert a.shape == b.shape and torch.equal(a, b)
    assert [tuple(t.shape) for t in got] == [(), (6, 300), (6,), (6,), (6,), (6,)]
    logp, ent = q.qrita_token_logprobs(xd, td.view(shape), entropy=True)
    assert logp.shape == ent.shape == (6,)
    starts = torch.arange(0, 7, 3, device=dev, dtype=torch.int32)
    got = q.qrita_preference_loss(xd, td.view(shape), starts.view(3, 1), ref_logp=v[:2].view(1, 2), weights=v[:1].view(1, 1))
    assert [tuple(t.shape) for t in got] == [(), (6, 300), (1,), (1,), (2,), (6,)]
    one = q.qrita_policy_loss(xd[:1], td[0], v[0], v[0])  # (values without a dimension are B = 1)
    assert [tuple(t.shape) for t in one[2:5]] == [(1,), (1,), (1,)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ent", [0.0, 0.05])
@pytest.mark.parametrize("B,V,ld", [(64, 200000, 200000), (150, 262144, 262144), (40, 262141, 262149), (20, 1000, 1000)])
def test_tensor_memory_given_back_early(dev, dtype, ent, B, V, ld):
    """A CTA whose cluster's sums are late gives its tensor memory back and reads
    that part of its row again for the gradient: the same bits, beside the logits,
    over them, and while another call does the same on another stream. (Rows of one
    CTA, and of shares that shared memory holds, have nothing to give back.)"""
    import torch

    import top_selection_row_gb300 as q

    if dtype == "f32":
        V, ld = V // 2, ld // 2 + 1
    g = torch.Generator(device=dev).manual_seed(B)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    wide = torch.randn(B, ld, generator=g, device=dev).to(dt)
    x = wide[:, :V]
    t = torch.randint(0, V, (B,), generator=g, device=dev, dtype=torch.int32)
    t[3] = -1
    adv = torch.randn(B, generator=g, device=dev)
    flag = dict(flags=q.LOSS_FLAG_TEST_GIVE_BACK)

    def call(v, **k):
        return q.qrita_policy_loss(v, t, None, adv, entropy_coef=ent, entropy=True, **k)

    want = call(x)
    got = call(x, **flag)
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    over = wide.clone()
    got = call(over[:, :V], out_grad=over[:, :V], **flag)
    assert torch.equal(over[:, :V], want.grad) and torch.equal(over[:, V:], wide[:, V:]) and torch.equal(got.loss, want.loss)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        here, there = call(x, **flag), call(x, stream=side, **flag)
        also = call(x)
        torch.cuda.synchronize()
        for got in (here, there, also):
            assert torch.equal(got.grad, want.grad) and torch.equal(got.loss, want.loss)
    soft = softmaxes(x[:2].float().cpu().numpy(), "f32", None, t[:2].cpu().numpy())
    near_grad(got.grad[:2], dtype, soft, t[:2].cpu().numpy(), -adv[:2].cpu().numpy() / B, np.full(2, -ent / B), np.zeros(2), 1.0)


def test_unknown_flags_are_refused(dev):
    import torch

    import top_selection_row_gb300 as q

    x, t, f = torch.zeros(3, 10, device=dev), torch.zeros(3, dtype=torch.int32, device=dev), torch.zeros(3, device=dev)
    with pytest.raises(q.QritaError) as err:
        q.qrita_policy_loss(x, t, f, f, flags=2)
    assert err.value.code == q.EINVAL


@pytest.mark.parametrize("inv_t", [1e-30, 1e-10, 1e4, 1e10, 1e30])
@pytest.mark.parametrize("dtype,V", [("f32", 300), ("bf16", 300), ("f32", 40000)])
def test_extreme_temperatures(dev, dtype, V, inv_t):
    """Weights all equal, or one token's alone, over rows with masked places of
    -1e9, -1e29 and -inf among them; tokens on such places too."""
    import top_selection_row_gb300 as q

    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, V)).astype(np.float32)
    for r, low in ((1, -1e9), (2, -1e29), (3, -np.inf), (4, -1e9), (5, -1e29)):
        x[r, 50:] = low
    tokens = np.array([3, 2, 1, 4, 70, 80], np.int32)
    if dtype == "bf16":
        from workloads import f32_to_bf16_bits

        x = f32_to_bf16_bits(x)
    soft = softmaxes(x, dtype, None, tokens, inv_t)
    xd, td = to_device(x, dtype, dev), put(dev, tokens)
    with np.errstate(over="ignore"):
        want = np.array([s.logp for s in soft]).astype(np.float32)
    for ent in (False, True):
        logp, H = q.qrita_token_logprobs(xd, td, inv_temperature=inv_t, entropy=ent)
        near_rows(logp.cpu().numpy(), want, "logp")
    near_rows(H.cpu().numpy(), [s.entropy for s in soft], "entropy", extra=ABS)
    a = rng.standard_normal(6).astype(np.float32) * np.float32(1e-2)
    got = q.qrita_token_logprobs_grad(xd, td, put(dev, a), inv_temperature=inv_t)
    keep = [0, 1, 2, 3]  # (a logp beyond fp32 is -inf, and its row then has no gradient)
    near_grad(got[keep], dtype, [soft[r] for r in keep], tokens[keep], a[keep], np.zeros(4), np.zeros(4), inv_t)
    assert np.isfinite(got.float().cpu().numpy()).all()
