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


@pytest.mark.parametrize("B,H,G,T,S,D", [(2, 2, 4, 16, 3000, 128), (160, 2, 1, 40, 700, 64), (1, 3, 2, 100, 2500, 200)])
@pytest.mark.parametrize("late", [False, True])
def test_a_window_whose_wait_gives_up(dev, B, H, G, T, S, D, late):  # noqa: F811
    """Sums without their scores make every weight NaN that a query of theirs sees, in
    every share of the slots; weights without them are NaN by themselves. The other heads,
    and the calls after, are as ever."""
    import torch

    import top_selection_row_gb300 as q

    g = torch.Generator(device=dev).manual_seed(B)
    k = torch.randn(B, H, S, D, generator=g, device=dev).bfloat16()
    query = torch.randn(B, T, H * G, D, generator=g, device=dev).bfloat16()
    w = torch.rand(B, H, S, generator=g, device=dev)
    n = torch.full((B,), S, dtype=torch.int32, device=dev)
    n[-1] = S // 2
    want = q.qrita_cache_weights(query, k, w.clone(), n)
    flag = q.CACHE_FLAG_TEST_GIVE_UP_WEIGHTS if late else q.CACHE_FLAG_TEST_GIVE_UP_SUMS
    for _ in range(3):
        got = q.qrita_cache_weights(query, k, w.clone(), n, flags=flag)
        assert torch.equal(got[:, 1:], want[:, 1:])
        first, right = got[:, 0], want[:, 0]
        lost = first.isnan()
        for b in range(B):
            m = int(n[b])
            # the first share of a head: 128 slots, or as many of eight CTAs (all of one's)
            part = m if not late or B * H > 152 else max(128, (m + 7) // 8)
            assert bool(lost[b, :part].all()) and not bool(lost[b, m:].any()), b
        assert torch.equal(first[~lost], right[~lost])
        assert torch.equal(q.qrita_cache_weights(query, k, w.clone(), n), want)


@pytest.mark.parametrize("D", [(32, 64), (8, 512)])
@pytest.mark.parametrize("apart", [False, True])
def test_an_eviction_whose_waits_give_up(dev, D, apart):  # noqa: F811
    """Rows whose bulk copies are not waited for are moved all the same, together and (in
    a wider tensor) one by one."""
    import torch

    import top_selection_row_gb300 as q

    _, _, w, n, at = small_cache(dev, S=500)
    k, v = (torch.randn(3, 2, 500, d, device=dev).bfloat16() for d in D)
    want = q.qrita_cache_evict(k, v, w, n, 200, sink=2, recent=9, positions=at, seen=n)
    z = [torch.full_like(t, 9) for t in want]
    if apart:
        z[0] = torch.full((3, 2, 200, D[0] + 8), 9, dtype=k.dtype, device=dev)[..., : D[0]]
        z[1] = torch.full((3, 200, 2, D[1]), 9, dtype=k.dtype, device=dev).transpose(1, 2)
    for _ in range(3):
        got = q.qrita_cache_evict(k, v, w, n, 200, sink=2, recent=9, positions=at, seen=n, out=q.EvictedCache(*z), flags=q.CACHE_FLAG_TEST_GIVE_UP_ROWS)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_the_largest_budget(dev):  # noqa: F811
    """2^31 - 1 slots for a hundred tokens (28 GB): kept whole, and filled to the end."""
    import torch

    import top_selection_row_gb300 as q

    budget = 2**31 - 1
    k, v = (torch.randint(-100, 100, (1, 1, 100, 1), device=dev).to(torch.int8) for _ in range(2))
    w = torch.rand(1, 1, 100, device=dev)
    n = torch.tensor([90], dtype=torch.int32, device=dev)
    got = q.qrita_cache_evict(k, v, w, n, budget)
    assert torch.equal(got.keys[:, :, :90], k[:, :, :90]) and torch.equal(got.values[:, :, :90], v[:, :, :90])
    assert torch.equal(got.weights[:, :, :90], w[:, :, :90]) and got.lengths.tolist() == [90]
    assert torch.equal(got.slots[0, 0, :90], torch.arange(90, dtype=torch.int32, device=dev))
    for t, fill in ((got.keys, 0), (got.values, 0), (got.weights, 0), (got.positions, -1), (got.slots, -1)):
        rest = t.flatten()[90:]
        assert rest.numel() == budget - 90
        for part in rest.split(2**28):  # (views: no copy of it all)
            assert bool((part == fill).all())
    del got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("bad", [dict(budget=2**32 + 5), dict(budget=2**31), dict(sink=2**32), dict(sink=2**31), dict(recent=2**32 + 1),
                                 dict(recent=2**40), dict(recent=-(2**32)), dict(sink=1.5)])
def test_numbers_beyond_32_bits(dev, bad):  # noqa: F811
    """Refused, not cut to their low 32 bits."""
    import torch

    import top_selection_row_gb300 as q

    k, v, w, n, at = small_cache(dev)
    seen, new = n + 5, torch.zeros(3, 2, 32, dtype=torch.bfloat16, device=dev)
    held = [t.clone() for t in (k, v, w, n, at, seen)]
    how = dict(budget=20, sink=1, recent=2) | bad
    out = q.qrita_cache_evict(k, v, w, n, 20, positions=at, seen=seen)
    for call in (lambda: q.qrita_cache_insert(k, v, w, at, n, seen, new, new, **how),
                 lambda: q.qrita_cache_evict(k, v, w, n, positions=at, seen=seen, out=out, **how)):
        with pytest.raises((ValueError, TypeError)):
            call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((k, v, w, n, at, seen), held))
    one = np.int64(3)  # numpy's whole numbers are taken
    q.qrita_cache_evict(k, v, w, n, np.int32(20), sink=one, recent=one)
