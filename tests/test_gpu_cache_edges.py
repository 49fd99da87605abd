"""The cache's calls at the edges of what they allow, against the fp64 oracle or the
same call made plainly; tolerances as tests/test_gpu_cache.py unless said."""

import numpy as np
import pytest

from oracle import cache_weights
from test_gpu_cache import check_weights, rounded, tensor
from test_gpu_losses import dev, put  # noqa: F401

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
    for bad in (dict(lengths=n), dict(lengths=seen), dict(slots=out.positions)):
        with pytest.raises(q.QritaError):
            q.qrita_cache_evict(k, v, w, n, 20, positions=at, seen=seen, out=out._replace(**bad))
    with pytest.raises(q.QritaError):
        q.qrita_cache_insert(k, v, w, at, n, n, new, new, 60)
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


@pytest.mark.parametrize("part", [16, 24, 5])
def test_values_that_are_a_part_of_the_keys(dev, part):  # noqa: F811
    """A cache of latent vectors, evicted into another one and put into: as with values
    of their own."""
    import torch

    import top_selection_row_gb300 as q

    k, _, w, n, at = small_cache(dev)
    want = q.qrita_cache_evict(k, k[..., :part].clone(), w, n, 20, recent=3)
    rows = torch.zeros_like(want.keys)
    out = want._replace(keys=rows, values=rows[..., :part], **{f: torch.empty_like(getattr(want, f)) for f in want._fields[2:]})
    got = q.qrita_cache_evict(k, k[..., :part], w, n, 20, recent=3, out=out)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    new, seen = torch.randn(3, 2, 32, device=dev).bfloat16(), [n.clone(), n.clone()]
    for c, s in zip((want, got), seen):
        q.qrita_cache_insert(c.keys, c.values, c.weights, c.positions, c.lengths, s, new, new[..., :part], 20)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(*seen)


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


@pytest.mark.parametrize("G,T", [(1, 1), (4, 1), (4, 4), (3, 7), (8, 20), (1, 130)])
@pytest.mark.parametrize("evicted", [False, True])
def test_weights_of_heads_of_192_dimensions(dev, G, T, evicted):  # noqa: F811
    check_weights(dev, G * T, 4, 2, G, T, 500, 192, "bf16", evicted)
    check_weights(dev, G * T + 1, 1, 3, G, T, 1300, 192, "bf16", evicted, layout=2)


@pytest.mark.parametrize("D", [32, 64, 96, 128, 192, 256, 72])
@pytest.mark.parametrize("G,T,S", [(1, 17, 100), (4, 8, 900), (8, 9, 3000), (130, 1, 400), (150, 3, 260)])
def test_weights_of_many_rows_that_no_window_takes(dev, D, G, T, S):  # noqa: F811
    """Expanded heads (one cache read by all) have no tensor map, and more than 128
    heads of a group do not fit its lanes: 32 rows at a time. Tolerances as
    tests/test_gpu_cache.py's weights."""
    import torch

    import top_selection_row_gb300 as q

    rng = np.random.default_rng(D + S)
    B, H, expanded = 2, 2, G < 128
    k = rng.standard_normal((B, 1 if expanded else H, S, D)).astype(np.float32)
    qq = (1.5 * rng.standard_normal((B, T, H * G, D))).astype(np.float32)
    w = rng.random((B, H, S)).astype(np.float32)
    n = np.array([S, S - 31], np.int32)
    kd = tensor(dev, k, "bf16").expand(B, H, S, D)
    got = q.qrita_cache_weights(tensor(dev, qq, "bf16"), kd, put(dev, w), put(dev, n), decay=0.75).cpu().numpy().astype(np.float64)
    k64, q64 = np.broadcast_to(rounded(k, "bf16"), (B, H, S, D)), rounded(qq, "bf16")
    for b in range(B):
        for h in range(H):
            m, mine = int(n[b]), q64[b, :, h * G : (h + 1) * G]
            add = cache_weights(mine, k64[b, h], np.arange(S), m, m, D**-0.5)
            want = w[b, h].astype(np.float64)
            want[:m] = want[:m] * 0.75 + add
            A = (np.abs(k64[b, h, :m]) @ np.abs(mine).reshape(T * G, D).T).max() * D**-0.5
            tol = 2 * (2 * (D * 2.0**-22 + 2.0**-23) * A + 2.0**-21 + S * 2.0**-24) * np.r_[add, np.zeros(S - m)] + 2.0**-22 * want
            tol[m:] = 0
            assert (np.abs(got[b, h] - want) <= tol).all(), (b, h)


@pytest.mark.parametrize("B,H,G,T,S,D,dtype,size", [(2, 2, 4, 1, 20000, 128, "bf16", 1.0), (2, 2, 4, 32, 20000, 128, "bf16", 1.0),
                                                     (1, 2, 8, 2, 9000, 64, "bf16", 1.0), (10, 8, 1, 17, 65536, 64, "bf16", 0.01),
                                                     (160, 2, 4, 1, 16384, 64, "bf16", 0.01), (2, 2, 4, 4, 9000, 128, "f32", 1.0)])
def test_accuracy_of_weights(dev, B, H, G, T, S, D, dtype, size):  # noqa: F811
    """The root mean square error of what is added, relative to its own. Scores of normal
    queries and keys are near 1, and near 2 where the square of their weight is. One is a sum
    of n steps (16 products a step on the tensor cores, D multiply-adds in fp32), each of
    which loses 0.58 of 2^-23 (cut off there) or 2^-24 of what is summed, sqrt(n / 3) of
    them in all; scaled and taken from the maximum it is rounded twice more by 0.58 2^-24
    of 2; the exponential is off by 6e-8, a row's sum by 1.2e-7 (512 additions by each of 8
    chains, one row in the window's worst case): 3e-7 on the tensor cores, 5e-7 in fp32.
    (Scores near 0 leave less.)"""
    import torch

    import top_selection_row_gb300 as q

    g = torch.Generator(device=dev).manual_seed(S)
    k = torch.randn(B, H, S, D, generator=g, device=dev)
    qq = size * torch.randn(B, T, H * G, D, generator=g, device=dev)
    if dtype == "bf16":
        k, qq = k.bfloat16(), qq.bfloat16()
    n = torch.full((B,), S, dtype=torch.int32, device=dev)
    got = q.qrita_cache_weights(qq, k, torch.zeros(B, H, S, device=dev), n)
    for b, h in ((0, 0), (B - 1, H - 1)):
        x = (qq[b, :, h * G : (h + 1) * G].reshape(T * G, D).double() @ k[b, h].double().T) / D**0.5
        after = torch.arange(S, device=dev) > S - T + torch.arange(T, device=dev).repeat_interleave(G)[:, None]
        want = x.masked_fill(after, -torch.inf).softmax(dim=1).sum(dim=0)
        err = float((got[b, h].double() - want).norm() / want.norm())
        assert err < (5e-7 if dtype == "f32" else 3e-7), (b, h, err)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,T", [(1, 1), (4, 2), (4, 30), (1, 40), (150, 1)])
def test_weights_of_scores_far_from_zero(dev, G, T, dtype):  # noqa: F811
    """Whole scores times 2^40: each row's largest ones share its weight (sums of at most
    S equal terms: exact; a quotient and R sums of 2^-23 each), the others have none."""
    import torch

    import top_selection_row_gb300 as q

    rng = np.random.default_rng(G * T)
    H, S, D = 2, 700, 64
    k = rng.integers(-1, 2, (1, H, S, D)).astype(np.float32)
    qq = rng.integers(-1, 2, (1, T, H * G, D)).astype(np.float32)
    n = torch.tensor([S], dtype=torch.int32, device=dev)
    got = q.qrita_cache_weights(tensor(dev, qq, dtype), tensor(dev, k, dtype), torch.zeros(1, H, S, device=dev), n, scale=2.0**40)
    for h in range(H):
        want = cache_weights(qq[0, :, h * G : (h + 1) * G], k[0, h], np.arange(S), S, S, 2.0**40)
        assert (np.abs(got[0, h].cpu().numpy() - want) <= G * T * 2.0**-23 * want).all()


@pytest.mark.parametrize("G,T", [(1, 1), (4, 3), (4, 40), (1, 60), (150, 1)])
def test_weights_of_rows_that_see_the_lowest_value_alone(dev, G, T):  # noqa: F811
    """Keys of the type's lowest value, as masked slots have: the queries that see
    nothing else see them alike, the others not at all. The rest as tests/test_gpu_cache.py."""
    import torch

    import top_selection_row_gb300 as q

    rng = np.random.default_rng(T)
    H, S, D = 2, 64, 64
    k = rng.standard_normal((1, H, S, D)).astype(np.float32)
    few = S if T == 1 else 15
    k[:, :, :few] = 0
    k[:, :, :few, 0] = -3.3895313892515355e38
    qq = rng.standard_normal((1, T, H * G, D)).astype(np.float32)
    qq[..., 0] = 1
    n = torch.tensor([S], dtype=torch.int32, device=dev)
    got = q.qrita_cache_weights(tensor(dev, qq, "bf16"), tensor(dev, k, "bf16"), torch.zeros(1, H, S, device=dev), n).cpu().numpy()
    k64, q64 = rounded(k, "bf16"), rounded(qq, "bf16")
    for h in range(H):
        mine = q64[0, :, h * G : (h + 1) * G]
        with np.errstate(over="ignore"):
            want = cache_weights(mine, k64[0, h], np.arange(S), S, S, D**-0.5)
        A = (np.abs(k64[0, h, few:]) @ np.abs(mine).reshape(T * G, D).T).max(initial=0) * D**-0.5
        tol = 2 * (2 * (D * 2.0**-22 + 2.0**-23) * A + 2.0**-21 + S * 2.0**-24) * want + 2.0**-22 * want
        assert (np.abs(got[0, h] - want) <= tol).all(), h


@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-37, 1.3e-38])
@pytest.mark.parametrize("G,T", [(1, 1), (4, 40), (1, 60)])
def test_weights_of_a_scale_of_nothing(dev, G, T, scale):  # noqa: F811
    """Scores of 0, or of 34 and 4 at most, whatever the keys hold. (A row's sum of S terms
    and its quotient, the sum of R rows: 2^-23 a term; the rounding of a score of 34, of its
    difference and of that times log2 e: 2^-18 each; the exponential 2^-21.)"""
    import torch

    import top_selection_row_gb300 as q

    rng = np.random.default_rng(T)
    H, S, D = 2, 200, 64
    k = np.zeros((1, H, S, D), np.float32)
    k[..., 0] = rng.standard_normal((1, H, S))
    k[:, :, ::3, 0] = -3.3895313892515355e38
    qq = rng.standard_normal((1, T, H * G, D)).astype(np.float32)
    qq[..., 0] = 1
    n = torch.tensor([S], dtype=torch.int32, device=dev)
    got = q.qrita_cache_weights(tensor(dev, qq, "bf16"), tensor(dev, k, "bf16"), torch.zeros(1, H, S, device=dev), n, scale=scale).cpu().numpy()
    k64, q64 = rounded(k, "bf16"), rounded(qq, "bf16")
    size = np.float64(np.float32(scale))
    for h in range(H):
        want = cache_weights(q64[0, :, h * G : (h + 1) * G], k64[0, h], np.arange(S), S, S, size)
        assert (np.abs(got[0, h] - want) <= ((G * T + S) * 2.0**-23 + 3 * 2.0**-18 + 2.0**-21) * want).all(), h


def test_batches_of_nothing(dev):  # noqa: F811
    import torch

    import top_selection_row_gb300 as q

    k, v, w, n, at = (t[:0] for t in small_cache(dev))
    new, seen, query = torch.zeros(0, 2, 32, dtype=torch.bfloat16, device=dev), n.clone(), torch.zeros(0, 3, 8, 32, dtype=torch.bfloat16, device=dev)
    assert q.qrita_cache_weights(query, k, w, n).shape == (0, 2, 60)
    assert [tuple(t.shape) for t in q.qrita_cache_evict(k, v, w, n, 7)] == [(0, 2, 7, 32)] * 2 + [(0, 2, 7)] * 3 + [(0,)]
    assert q.qrita_cache_insert(k, v, w, at, n, seen, new, new, 60).shape == (0, 2)


@pytest.mark.parametrize("off", [1, 2, 3])
def test_vectors_and_rows_off_their_boundaries(dev, off):  # noqa: F811
    """Everything `off` elements behind a boundary: the same as on it (weights: with fp32
    products by the same kernel, so equal too)."""
    import torch

    import top_selection_row_gb300 as q

    def shifted(t):
        buf = torch.zeros(t.numel() + off, dtype=t.dtype, device=dev)
        buf[off:] = t.flatten()
        return buf[off:].view(t.shape)

    for S in (60, 5001):
        k, v, w, n, at = small_cache(dev, S=S)
        seen = n + 3
        args = [k, v, w, n]
        want = q.qrita_cache_evict(*args, 31, sink=1, recent=4, positions=at, seen=seen)
        out = q.EvictedCache(*(shifted(torch.full_like(t, 7)) for t in want))
        got = q.qrita_cache_evict(*(shifted(t) for t in args), 31, sink=1, recent=4, positions=shifted(at), seen=shifted(seen), out=out)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        new = torch.randn(2, 3, 2, 32, device=dev).bfloat16()
        a = [t.clone() for t in (k, v, w, at, n, seen)]
        b = [shifted(t) for t in a]
        one = q.qrita_cache_insert(*a, *new, S, recent=4)
        assert torch.equal(q.qrita_cache_insert(*b, *(shifted(t) for t in new), S, recent=4), one)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        query = torch.randn(3, 2, 4, 32, device=dev)
        x = q.qrita_cache_weights(query, k.float(), w.clone(), n, positions=at, seen=seen)
        y = q.qrita_cache_weights(shifted(query), shifted(k.float()), shifted(w), shifted(n), positions=shifted(at), seen=shifted(seen))
        assert torch.allclose(x, y, rtol=2**-18, atol=0)  # (another order of a sum of 32 products)


def test_two_streams_at_once(dev):  # noqa: F811
    """Windows (each takes whole SMs), evictions and insertions of two streams, side by
    side and replayed: nothing is shared between calls."""
    import torch

    import top_selection_row_gb300 as q

    g = torch.Generator(device=dev).manual_seed(9)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev).bfloat16()  # noqa: E731
    sets = []
    for S in (3000, 4100):
        k, v, query, new = rand(3, 4, S, 64), rand(3, 4, S, 64), rand(3, 24, 16, 64), rand(3, 4, 64)
        n = torch.tensor([S, S // 3, S - 1], dtype=torch.int32, device=dev)
        w0 = torch.rand(3, 4, S, generator=g, device=dev)

        def run(k=k, v=v, query=query, new=new, n=n, w0=w0):
            w, seen = w0.clone(), n.clone()
            q.qrita_cache_weights(query, k, w, n)
            c = q.qrita_cache_evict(k, v, w, n, 500, sink=2, recent=50)
            slots = q.qrita_cache_insert(c.keys, c.values, c.weights, c.positions, c.lengths, seen, new, new, 500, recent=50)
            return [w, *c, seen, slots]

        sets.append((run, [t.clone() for t in run()]))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for s, (run, _) in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(run())
        torch.cuda.synchronize()
        for held, (_, want) in zip(got, sets):
            assert all(torch.equal(a, b) for a, b in zip(held, want))
    graphs = []
    for run, _ in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = run()
        graphs.append((graph, held))
    for _ in range(5):
        for s, (graph, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for (_, held), (_, want) in zip(graphs, sets):
            assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_many_short_sequences(dev):  # noqa: F811
    """More heads than a wave of CTAs by far: each as by itself."""
    import torch

    import top_selection_row_gb300 as q

    g = torch.Generator(device=dev).manual_seed(1)
    B, H, S, D = 5000, 3, 20, 32
    k, w = torch.randn(B, H, S, D, generator=g, device=dev).bfloat16(), torch.rand(B, H, S, generator=g, device=dev)
    n = torch.randint(-1, S + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    for T in (1, 9):
        query = torch.randn(B, T, 2 * H, D, generator=g, device=dev).bfloat16()
        got = q.qrita_cache_weights(query, k, w.clone(), n)
        for b in (0, 1234, B - 1):
            assert torch.allclose(got[b], q.qrita_cache_weights(query[b:b + 1], k[b:b + 1], w[b:b + 1].clone(), n[b:b + 1])[0], rtol=2**-20)
    cut = q.qrita_cache_evict(k, k, w, n, 6, recent=2)
    for b in (0, 1234, B - 1):
        assert all(torch.equal(x[b], y[0]) for x, y in zip(cut, q.qrita_cache_evict(k[b:b + 1], k[b:b + 1], w[b:b + 1], n[b:b + 1], 6, recent=2)))
    seen, lengths, new = n.clamp(min=0), cut.lengths.clone(), torch.randn(B, H, D, generator=g, device=dev).bfloat16()
    one = [t[7:8].clone() for t in (cut.keys, cut.values, cut.weights, cut.positions, lengths, seen)]
    q.qrita_cache_insert(cut.keys, cut.values, cut.weights, cut.positions, lengths, seen, new, new, 6, recent=2)
    q.qrita_cache_insert(*one, new[7:8], new[7:8], 6, recent=2)
    assert all(torch.equal(x[7:8], y) for x, y in zip((cut.keys, cut.values, cut.weights, cut.positions, lengths, seen), one))
