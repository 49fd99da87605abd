"""Scores and their gradient where values leave what fp32 holds, against the fp64
oracle; tolerances as tests/test_gpu_scores.py unless said."""

import numpy as np
import pytest

from oracle import scores_grad_row, scores_row
from test_gpu_losses import ABS, BF16_ROUND, F32_ROUND, dev, make_rows, near, put, widened  # noqa: F401
from parity_helpers import to_device
from test_gpu_scores import check_grad, given
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu

LOWEST = {"f32": -3.4028234663852886e38, "bf16": -3.3895313892515355e38}


def with_lowest(seed, B, V, dtype, keep):
    """Rows with the type's lowest value (a common way to mask) in a third of their
    places, some of them given: tokens first, then six others."""
    rng, x, tokens, mask = make_rows(seed, B, V, "f32", keep)
    low = rng.random((B, V)) < 0.34
    low[np.arange(B), np.argmax(x, axis=1)] = False
    x[low] = LOWEST[dtype]
    ids = given(rng, np.clip(tokens, 0, V - 1), V, 7)
    ids[:, 3] = [np.flatnonzero(low[r])[0] for r in range(B)]
    ids[:, 4] = [np.flatnonzero(low[r])[-1] for r in range(B)]
    if mask is not None:
        mask[np.arange(B)[:, None], ids[:, 3:5]] = 1
        mask[1] = 0
    return rng, f32_to_bf16_bits(x) if dtype == "bf16" else x, ids, mask


# rows that wait on the SM, rows too long for it, kept sets that are listed and walked
@pytest.mark.parametrize("B,V,keep", [(5, 4000, 0), (2, 70001, 0), (1, 2_400_001, 0), (5, 4000, 40), (3, 70001, 30000)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("inv_t,size", [(1.25, 0.5), (1.0, 3.0)])
def test_gradients_of_tokens_of_the_lowest_value(dev, B, V, keep, dtype, inv_t, size):  # noqa: F811
    """Their log-probabilities, or these times an entropy's gradient, leave fp32; their
    probabilities are 0."""
    rng, x, ids, mask = with_lowest(V + keep, B, V, dtype, keep)
    g = rng.standard_normal(ids.shape).astype(np.float32)
    g[:, 4] = 0
    h = (size * (1 + rng.random(B))).astype(np.float32)
    check_grad(dev, x, dtype, ids, g, h, mask, inv_t)


@pytest.mark.parametrize("B,V,keep", [(3, 4000, 0), (1, 1_200_003, 0), (3, 4000, 100)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_of_one_token_listed_often(dev, B, V, keep, dtype):  # noqa: F811
    """A token of nearly all the probability, listed 250 times with gradients that
    nearly cancel, beside six others. Its entry is G (1 - p) - p R, G its own
    gradients' sum and R the others'. Sums are fp64 (256 2^-53 of their magnitudes), an
    id's own pairs of fp32 (256 roundings of a low part of 2^-20 of the magnitudes: below
    2^-37 of them, 2e-7 here), and rounded once; log p is off by 2^-22 + 2^-24 (10 + E), E < 1 here, and so are 1 - p and
    p; each of the two products' four operations rounds by 2^-24, expm1 and exp by two
    such steps."""
    import top_selection_row_gb300 as q

    rng = np.random.default_rng(V)
    x = rng.standard_normal((B, V)).astype(np.float32)
    x[:, 17] = 10 + np.log(V)
    mask = None
    if keep:
        mask = np.zeros((B, V), np.uint8)
        mask[:, :keep] = 1
    ids = np.full((B, 256), 17, np.int32)
    others = rng.permutation(256)[:6]
    ids[:, others] = 20 + np.arange(6)
    g = (rng.choice([-1, 1], ids.shape) * rng.uniform(90, 110, ids.shape)).astype(np.float32)
    g[:, others] = rng.uniform(-1, 1, (B, 6))
    own = ids == 17
    last = np.flatnonzero(own[0])[-1]
    g[:, last] = 3 - np.where(own, g, 0).astype(np.float64).sum(1) + g[:, last]
    if dtype == "bf16":
        x = f32_to_bf16_bits(x)
    got = q.qrita_token_scores_grad(to_device(x, dtype, dev), put(dev, ids), put(dev, g), mask=put(dev, mask))
    got = got[:, 17].float().cpu().numpy().astype(np.float64)
    xs = widened(x, dtype)
    for r in range(B):
        want = scores_grad_row(xs[r], None if mask is None else mask[r], ids[r], g[r])[0][17]
        G, R = (np.where(w, g[r], 0).astype(np.float64).sum() for w in (own[r], ~own[r]))
        tol = (abs(G) + abs(R)) * (2.0**-22 + 11 * 2.0**-24 + 6 * 2.0**-24) + 256 * 2.0**-53 * np.abs(g[r]).sum()
        near(got[r], want, tol + (BF16_ROUND if dtype == "bf16" else F32_ROUND) * abs(want), f"row {r}")


@pytest.mark.parametrize("B,V,keep", [(5, 4000, 0), (2, 70001, 0), (700, 3000, 0), (5, 4000, 40)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ranks_of_tokens_of_the_lowest_value(dev, B, V, keep, dtype):  # noqa: F811
    """Log-probabilities beyond fp32 are -inf there; ranks and alternatives are those of
    the order, which has them."""
    import top_selection_row_gb300 as q

    _, x, ids, mask = with_lowest(V + keep, min(B, 5), V, dtype, keep)
    ids = ids[:, 3:]
    some = np.arange(B) % len(ids)
    x, ids, mask = x[some], ids[some], None if mask is None else mask[some]
    got = q.qrita_token_scores(to_device(x, dtype, dev), put(dev, ids), top=60, mask=put(dev, mask), inv_temperature=1.25, rank=True)
    xs = widened(x, dtype)
    want = [scores_row(xs[r], None if mask is None else mask[r], ids[r], 1.25, 60) for r in range(min(B, 5))]
    assert np.array_equal(got.rank.cpu().numpy(), np.array([w[1] for w in want])[some])
    assert np.array_equal(got.top_ids.cpu().numpy(), np.array([w[3] for w in want])[some])
    below = np.array([w[0] for w in want])[some] < -3.5e38
    assert below[:, 0].any() and np.isneginf(got.logp.cpu().numpy()[below]).all()


def test_scores_of_nothing_and_of_as_many_as_there_can_be(dev):  # noqa: F811
    """No rows; 8192 given tokens with 128 alternatives; more alternatives than logits in
    more rows than a wave."""
    import torch

    import top_selection_row_gb300 as q

    x = torch.randn(0, 50, device=dev)
    none = torch.zeros(0, 3, dtype=torch.int32, device=dev)
    assert q.qrita_token_scores(x, none, top=4, entropy=True, rank=True).top_logp.shape == (0, 4)
    assert q.qrita_token_scores_grad(x, none, torch.zeros(0, 3, device=dev)).shape == (0, 50)
    rng = np.random.default_rng(2)
    for B, V, M, top in ((2, 30000, 8192, 128), (2, 200_000, 8192, 128), (20000, 100, 3, 128)):
        xs = rng.standard_normal((min(B, 7), V)).astype(np.float32)
        t = rng.integers(-1, V + 1, (len(xs), M)).astype(np.int32)
        some = np.arange(B) % len(xs)
        got = q.qrita_token_scores(put(dev, xs[some]), put(dev, t[some]), top=top, entropy=True, rank=True)
        want = [scores_row(xs[r].astype(np.float64), None, t[r], 1.0, top) for r in range(len(xs))]
        assert np.array_equal(got.top_ids.cpu().numpy(), np.array([w[3] for w in want])[some])
        assert np.array_equal(got.rank.cpu().numpy(), np.array([w[1] for w in want])[some])
        near(got.logp.cpu().numpy(), np.array([w[0] for w in want])[some], ABS + F32_ROUND * 30, "logp")
