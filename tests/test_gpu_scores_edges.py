"""Scores and their gradient where values leave what fp32 holds, against the fp64
oracle; tolerances as tests/test_gpu_scores.py unless said."""

import numpy as np
import pytest

from test_gpu_losses import REL, dev, make_rows, put  # noqa: F401
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
