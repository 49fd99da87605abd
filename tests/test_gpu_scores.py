"""GPU parity of the scores of given tokens, their rank and alternatives, and of
their gradient, through the binding, against the fp64 oracle
(oracle/qrita_scores.py).

Values: ABS of tests/test_gpu_losses.py bounds log S, and with it logp and H,
before their rounding (fp32: 2^-24 of the value). Gradients: a probability is off
by REL of itself; an entry inv_t (G - p (a + h (log p + H))) by REL of the
magnitudes of its terms, plus the fp32 sum of K gradients (K 2^-24 of their
magnitudes, below REL for K <= 256) and one rounding to the type. Ranks and ids
are whole numbers: equal.
"""

import numpy as np
import pytest

from oracle import scores_grad_row, scores_row
from parity_helpers import to_device
from test_gpu_losses import ABS, BF16_ROUND, F32_ROUND, REL, dev, make_rows, near, padded, put, widened  # noqa: F401
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu


def given(rng, tokens, V, M):
    """[B, M]: the drawn token first, then others, some of them padding or twice."""
    t = rng.integers(0, V, (len(tokens), M)).astype(np.int32)
    t[:, 0] = tokens
    t[rng.random(t.shape) < 0.1] = -1
    if M > 2:
        t[:, 2] = t[:, 0]
    return t


def check(dev, x, dtype, t, mask, top, inv_t=1.0, entropy=True, ld=None, **how):
    import top_selection_row_gb300 as q

    xd = to_device(x, dtype, dev)
    if ld:
        xd = padded(xd, ld, 9e4)[:, : x.shape[1]]
    got = q.qrita_token_scores(xd, put(dev, t), top=top, mask=put(dev, mask), inv_temperature=inv_t, entropy=entropy, rank=True, **how)
    xs = widened(x, dtype)
    want = [scores_row(xs[r], None if mask is None else mask[r], t[r], inv_t, top) for r in range(len(t))]
    both = lambda w: ABS + F32_ROUND * np.abs(np.where(np.isfinite(w), w, 0))  # noqa: E731
    lp = np.array([w[0] for w in want])
    near(got.logp.cpu().numpy(), lp, both(lp), "logp")
    assert np.array_equal(got.rank.cpu().numpy(), [w[1] for w in want])
    if entropy:
        H = np.array([w[2] for w in want])
        near(got.entropy.cpu().numpy(), H, 2 * both(H), "entropy")
    if top:
        assert np.array_equal(got.top_ids.cpu().numpy(), np.array([w[3] for w in want]))
        lp = np.array([w[4] for w in want])
        near(got.top_logp.cpu().numpy(), lp, both(lp), "top logp")
    return got


# rows of one logit, less than a unit, a block, a step and some, several CTAs, several steps a CTA
SHAPES = [(1, 1, "f32"), (3, 5, "bf16"), (2, 17, "f32"), (5, 1000, "bf16"), (7, 4099, "f32"), (3, 50021, "bf16"),
          (2, 70001, "f32"), (700, 2500, "bf16")]


@pytest.mark.parametrize("keep", [0, 30])
@pytest.mark.parametrize("B,V,dtype", SHAPES)
@pytest.mark.parametrize("M,top", [(1, 5), (9, 128)])
def test_scores(dev, B, V, dtype, keep, M, top):
    rng, x, tokens, mask = make_rows(B + V + M, B, V, dtype, keep)
    check(dev, x, dtype, given(rng, tokens, V, M), mask, top, inv_t=0.8, entropy=top > 5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_rows(dev, dtype):
    """One CTA a row with many groups of several steps, and clusters of 16."""
    rng, x, tokens, mask = make_rows(5, 1, 1_500_007, dtype, 40_000)
    t = given(rng, tokens, x.shape[1], 3)
    check(dev, x, dtype, t, None, 100)
    check(dev, x, dtype, t, mask, 128)
    B, V = 640, 33000
    rng, x, tokens, mask = make_rows(6, 2, V, dtype, 9000)
    r = rng.integers(0, 2, B)
    check(dev, x[r], dtype, given(rng, tokens[r], V, 2), mask[r], 20)
    check(dev, x[r], dtype, given(rng, tokens[r], V, 2), None, 20)


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("top", [1, 20, 128])
@pytest.mark.parametrize("kind", ["equal", "levels", "rising", "falling", "stripe", "lowest", "zeros"])
def test_ties_and_orders(dev, kind, top, keep):
    """Rows whose largest logits are many equal ones, or all lie in one thread's
    units: the list overflows and the slow path has to give the same order."""
    V = 40000
    rng = np.random.default_rng(top)
    x = {"equal": np.full(V, 1.5), "levels": rng.integers(0, 3, V).astype(float), "rising": np.arange(V) / 64.0,
         "falling": -np.arange(V) / 64.0, "stripe": np.where(np.arange(V) // 8 % 256 == 3, 5.0 + np.arange(V) / V, 0.0),
         "lowest": np.where(np.arange(V) % 1000 == 7, 1.0, -3.4028234663852886e38), "zeros": np.where(np.arange(V) % 2, -0.0, 0.0)}[kind]
    x = np.stack([x, x[::-1], x]).astype(np.float32)
    mask = (rng.random(x.shape) < 0.7).astype(np.uint8) if keep else None
    t = np.array([[V - 1], [V // 2], [0]], np.int32)
    if keep:
        mask[np.arange(3), t[:, 0]] = 1
    for dtype in ("f32", "bf16"):
        xs = f32_to_bf16_bits(x) if dtype == "bf16" else x
        check(dev, xs, dtype, t, mask, top)
        # many rows: one CTA a row
        check(dev, np.tile(xs, (100, 1)), dtype, np.tile(t, (100, 1)), None if mask is None else np.tile(mask, (100, 1)), top, entropy=False)


@pytest.mark.parametrize("keep", [0, 40])
def test_specials_alignment_and_padding(dev, keep):
    """NaN and infinities in and out of the kept set, rows of odd leading
    dimensions, masked places that hold anything."""
    B, V = 9, 3001
    for dtype in ("f32", "bf16"):
        rng, x, tokens, mask = make_rows(11, B, V, "f32", keep)
        tokens = np.clip(tokens, 0, V - 1)
        x[5, 7] = np.nan
        x[6, V - 1] = np.inf
        x[7, : V // 2] = -np.inf
        x[8] = -np.inf
        if keep:
            mask[:, [7, V - 1]] = 0
            mask[5, 7] = 1
        if dtype == "bf16":
            x = f32_to_bf16_bits(x)
        t = given(rng, tokens, V, 4)
        t[7, 1] = 3
        for ld in (V, V + 1, V + 5, V + 8):
            check(dev, x, dtype, t, mask, 8, ld=ld)
            check(dev, x[1:], dtype, t[1:], None if mask is None else mask[1:], 8, ld=ld)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_of_many_logits_of_minus_infinity(dev, dtype):
    """Whole steps of the sums whose exponents have no finite lowest one."""
    V = 40003
    rng, x, tokens, _ = make_rows(13, 4, V, "f32")
    x[:, rng.random(V) < 0.5] = -np.inf
    x[1, :20000] = -np.inf
    x[2, 8:] = -np.inf
    x[3] = np.where(np.arange(V) % 512 == 5, -3.0e38, x[3])
    if dtype == "bf16":
        x = f32_to_bf16_bits(x)
    t = given(rng, np.clip(tokens, 0, V - 1), V, 3)
    check(dev, x, dtype, t, None, 16)
    check(dev, np.tile(x, (160, 1)), dtype, np.tile(t, (160, 1)), None, 16)  # one CTA a row


def test_only_some_outputs_and_reuse(dev):
    import torch

    import top_selection_row_gb300 as q

    rng, x, tokens, _ = make_rows(3, 6, 900, "f32")
    xd, t = put(dev, x), put(dev, given(rng, tokens, 900, 3))
    whole = q.qrita_token_scores(xd, t, top=7, entropy=True, rank=True)
    assert q.qrita_token_scores(xd, top=7)[:3] == (None, None, None)
    assert torch.equal(q.qrita_token_scores(xd, top=7).top_ids, whole.top_ids)
    assert torch.equal(q.qrita_token_scores(xd, entropy=True).entropy, whole.entropy)
    assert torch.equal(q.qrita_token_scores(xd, t).logp, whole.logp)
    out = q.TokenScores(*(torch.zeros_like(v) for v in whole))
    again = q.qrita_token_scores(xd, t, top=7, entropy=True, rank=True, out=out)
    assert all(a.data_ptr() == o.data_ptr() and torch.equal(a, w) for a, o, w in zip(again, out, whole))
    # the token's own selection says the same order
    ids, _ = q.qrita_topk_ids(xd, torch.full((6,), 7, dtype=torch.int32, device=dev), 7)
    assert torch.equal(ids, whole.top_ids)
    # and the one-token entry the same value, to the bit
    assert torch.equal(q.qrita_token_logprobs(xd, t[:, 0].contiguous())[0], whole.logp[:, 0])
    none = q.qrita_token_scores(xd[:0], t[:0], top=7, rank=True)
    assert none.logp.shape == (0, 3) and none.top_ids.shape == (0, 7)
    for bad in (dict(top=129), dict(top=-1), dict(top=0, rank=True)):
        with pytest.raises((ValueError, q.QritaError)):
            q.qrita_token_scores(xd, **bad)
    with pytest.raises(ValueError):
        q.qrita_token_scores(xd, t[:, 0])


def check_grad(dev, x, dtype, ids, g, h, mask, inv_t=1.0, ld=None, inplace=False):
    import top_selection_row_gb300 as q

    V = x.shape[1]
    xd = to_device(x, dtype, dev)
    buf = None
    if ld:
        buf = padded(xd, ld, 7.0)
        xd = buf[:, :V]
    out = q.qrita_token_scores_grad(xd, put(dev, ids), put(dev, g), put(dev, h), mask=put(dev, mask), inv_temperature=inv_t,
                                    out_grad=xd if inplace else None)
    if inplace and buf is not None and ld > V:
        assert bool((buf[:, V:] == 7.0).all())
    got = out.float().cpu().numpy().astype(np.float64)
    xs = widened(x, dtype)
    half = BF16_ROUND if dtype == "bf16" else F32_ROUND
    for r in range(len(ids)):
        want, size = scores_grad_row(xs[r], None if mask is None else mask[r], ids[r], np.zeros(ids.shape[1]) if g is None else g[r],
                                     0.0 if h is None else h[r], inv_t)
        # (a bf16 or fp32 result below the type's normal range is rounded by its smallest step, or taken as 0)
        near(got[r], want, REL * size + half * np.abs(np.nan_to_num(want)) + 2.0 ** -125, f"row {r}")


@pytest.mark.parametrize("keep", [0, 30])
@pytest.mark.parametrize("B,V,dtype", SHAPES + [(1, 300_001, "bf16"), (1, 1_200_003, "f32")])
@pytest.mark.parametrize("K", [1, 20, 256])
def test_gradient(dev, B, V, dtype, keep, K):
    if B > 100 and K > 20:
        B = 40
    rng, x, tokens, mask = make_rows(B + V + K, B, V, dtype, keep)
    ids = given(rng, tokens, V, K)
    g = (rng.standard_normal(ids.shape) / B).astype(np.float32)
    g[0] = 0 if K == 20 else g[0]
    h = (rng.standard_normal(B) / B).astype(np.float32)
    check_grad(dev, x, dtype, ids, g, None, mask, 0.75)
    check_grad(dev, x, dtype, ids, g, h, mask)
    check_grad(dev, x, dtype, ids, g, h, mask, ld=V + 3, inplace=True)
    if K == 1:
        check_grad(dev, x, dtype, ids, None, h, mask)


def test_gradient_specials(dev):
    B, V = 7, 2000
    for dtype in ("f32", "bf16"):
        for keep in (0, 50):
            rng, x, tokens, mask = make_rows(21, B, V, "f32", keep)
            x[1, 7] = np.nan
            x[2, 5] = np.inf
            x[3] = -np.inf
            x[4, 100:] = -np.inf
            if keep:
                mask[1, 7] = mask[2, 5] = 1
            if dtype == "bf16":
                x = f32_to_bf16_bits(x)
            ids = given(rng, np.clip(tokens, 0, V - 1), V, 6)
            g = rng.standard_normal(ids.shape).astype(np.float32)
            g[5, :] = 0
            g[6, 1] = -g[6, 0]
            check_grad(dev, x, dtype, ids, g, rng.standard_normal(B).astype(np.float32) * 0, mask)


def test_gradient_against_differences_of_the_call(dev):
    """Central differences of the forward call's own values: off by its errors (ABS
    each, over the step) and the step's square times a third derivative below 4."""
    import top_selection_row_gb300 as q

    rng, x, tokens, _ = make_rows(31, 2, 40, "f32")
    ids = np.stack([rng.permutation(40)[:5] for _ in range(2)]).astype(np.int32)
    g, h = rng.standard_normal((2, 5)).astype(np.float32), rng.standard_normal(2).astype(np.float32)

    def f(x):
        s = q.qrita_token_scores(put(dev, x.astype(np.float32)), put(dev, ids), entropy=True)
        return (s.logp.double().cpu().numpy() * g).sum(1) + s.entropy.double().cpu().numpy() * h

    got = q.qrita_token_scores_grad(put(dev, x), put(dev, ids), put(dev, g), put(dev, h)).cpu().numpy()
    step = 1.0 / 64
    weight = np.abs(g).sum(1) + 2 * np.abs(h)
    # (the step is exact in fp32 only up to the logits' rounding: x +- step is rounded by 2^-24 |x|)
    tol = weight * (2 * ABS / step + 4 * step**2 + 2.0 ** -20)
    for j in range(40):
        d = np.zeros_like(x)
        d[:, j] = step
        diff = (f(x + d) - f(x - d)) / (2 * step)
        assert (np.abs(diff - got[:, j]) <= tol).all(), j


def test_a_run_together_captured_and_on_another_stream(dev):
    """A teacher's alternatives, the student's scores of them and their gradient, as
    a distillation step makes them: eager, on another stream, and replayed."""
    import torch

    import top_selection_row_gb300 as q

    _, a, _, _ = make_rows(41, 12, 32000, "bf16")
    _, b, _, _ = make_rows(42, 12, 32000, "bf16")
    teacher, student = to_device(a, "bf16", dev), to_device(b, "bf16", dev)

    def step(**how):
        alt = q.qrita_token_scores(teacher, top=20, **how)
        got = q.qrita_token_scores(student, alt.top_ids, entropy=True, **how)
        p = alt.top_logp.exp() if not how else torch.empty_like(alt.top_logp)
        if how:
            with torch.cuda.stream(how["stream"]):
                p = alt.top_logp.exp()
                w = -p
        else:
            w = -p
        return alt.top_ids, got.logp, q.qrita_token_scores_grad(student, alt.top_ids, w, **how)

    want = [v.clone() for v in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side)
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(2):
        for v in held:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(held, want))
    # the rows' gradient sums to nothing: softmax is free of a constant
    assert float(want[2].float().sum(1).abs().max()) < 0.05
