"""The cache's calls at the edges of what they allow, against the fp64 oracle or the
same call made plainly; tolerances as tests/test_gpu_cache.py unless said."""

import numpy as np
import pytest

from test_gpu_losses import dev  # noqa: F401

pytestmark = pytest.mark.gpu


def small_cache(dev, B=3, H=2, S=60, D=32):  # noqa: F811
    import torch

    g = torch.Generator(device=dev).manual_seed(S)
    k, v = (torch.randn(B, H, S, D, generator=g, device=dev).bfloat16() for _ in range(2))
    w = torch.rand(B, H, S, generator=g, device=dev)
    n = torch.tensor([S, S - 7, 0][:B], dtype=torch.int32, device=dev)
    at = torch.arange(S, dtype=torch.int32, device=dev).expand(B, H, S).contiguous()
    return k, v, w, n, at


def test_vectors_that_are_read_and_written(dev):  # noqa: F811
    """Lengths given as the lengths' output, and the like: refused, nothing written."""
    import torch

    import top_selection_row_gb300 as q

    k, v, w, n, at = small_cache(dev)
    seen = n + 5
    out = q.qrita_cache_evict(k, v, w, n, 20, positions=at, seen=seen)
    new = torch.zeros(3, 2, 32, dtype=torch.bfloat16, device=dev)
    held = [t.clone() for t in (k, v, w, n, at, seen)]
    for bad in (dict(lengths=n), dict(lengths=seen), dict(slots=out.positions), dict(values=out.keys)):
        with pytest.raises(q.QritaError):
            q.qrita_cache_evict(k, v, w, n, 20, positions=at, seen=seen, out=out._replace(**bad))
    for args in ((k, v, w, at, n, n), (k, k, w, at, n, seen)):
        with pytest.raises(q.QritaError):
            q.qrita_cache_insert(*args, new, new, 60)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((k, v, w, n, at, seen), held))


def test_keys_and_values_side_by_side(dev):  # noqa: F811
    """Both in one tensor, read and written: the same as apart."""
    import torch

    import top_selection_row_gb300 as q

    k, v, w, n, at = small_cache(dev)
    want = q.qrita_cache_evict(k, v, w, n, 20, recent=3)
    both, cut = torch.cat((k, v), dim=3), torch.zeros(3, 2, 20, 64, dtype=torch.bfloat16, device=dev)
    out = want._replace(keys=cut[..., :32], values=cut[..., 32:], **{f: torch.empty_like(getattr(want, f)) for f in want._fields[2:]})
    got = q.qrita_cache_evict(both[..., :32], both[..., 32:], w, n, 20, recent=3, out=out)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    new, seen = torch.randn(2, 3, 2, 32, device=dev).bfloat16(), n.clone()
    a = [t.clone() for t in (want.keys, want.values, want.weights, want.positions, want.lengths, seen)]
    b = [got.keys, got.values, *(t.clone() for t in (want.weights, want.positions, want.lengths, seen))]
    for c in (a, b):
        q.qrita_cache_insert(*c, *new, 20)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
