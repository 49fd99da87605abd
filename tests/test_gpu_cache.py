"""GPU tests of a key-value cache's slots: attention weights gathered, the slots a
budget keeps, one token put into a full cache, against the fp64 oracle
(oracle/qrita_scores.py).

Weights: a score is an fp32 sum of D exact products (the tensor cores add with at
most 2^-22 of the partial sums' magnitude lost a step: D 2^-22 of the sum of the
products' magnitudes A), is scaled (2^-24) and its difference from the row's maximum
rounded (2^-23 of the largest score X): an exponent is off by
d = 2 (D 2^-22 A scale + 2^-23 X), doubled for the maximum's own. The exponential
itself is within 2^-21, fp32 sums of S terms within S 2^-24, so a weight is off by
(d + 2^-21 + S 2^-24) of itself, twice for the sum it is divided by; what is
accumulated is rounded by 2^-24 of itself a step. Slots, positions and rows are whole:
equal.
"""

import numpy as np
import pytest

from oracle import bf16_bits_to_f64, cache_weights, kept_order
from test_gpu_losses import dev, put  # noqa: F401
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu


def tensor(dev, x, dtype):
    import torch

    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dev)
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def rounded(x, dtype):
    x = np.asarray(x, np.float32)
    return bf16_bits_to_f64(f32_to_bf16_bits(x)).reshape(x.shape) if dtype == "bf16" else x.astype(np.float64)


def cache(rng, B, H, S, evicted):
    """lengths (a full one, an empty one, an idle one among several), and positions
    and seen of caches that have evicted before."""
    n = rng.integers(S // 2, S + 1, B).astype(np.int32)
    n[0] = S
    if B > 3:
        n[1], n[2] = 0, -1
    if not evicted:
        return n, None, None
    seen = (np.maximum(n, 0) + rng.integers(0, S + 1, B)).astype(np.int32)
    at = np.full((B, H, S), -7, np.int32)
    for b in range(B):
        for h in range(H):
            if n[b] > 0:
                at[b, h, : n[b]] = rng.permutation(rng.choice(seen[b], n[b], replace=False))
    return n, at, seen


def check_weights(dev, seed, B, H, G, T, S, D, dtype, evicted=False, decay=0.9, scale=None, layout=0, special=False):
    import torch

    import top_selection_row_gb300 as q

    rng = np.random.default_rng(seed)
    n, at, seen = cache(rng, B, H, S, evicted)
    k = rng.standard_normal((B, H, S, D)).astype(np.float32)
    qq = (1.5 * rng.standard_normal((B, T, H * G, D))).astype(np.float32)
    w = rng.random((B, H, S)).astype(np.float32)
    if special:
        k[0, 0, S - 1] = np.nan  # the newest token's: seen by the last query alone (no positions)
        if B > 3:
            k[3, 0, n[3]:] = np.inf  # behind the length
            k[3, :, 0, 0] = np.inf
    kd, qd, wd = tensor(dev, k, dtype), tensor(dev, qq, dtype), put(dev, w)
    if layout == 1:  # slots before heads, rows padded by an odd number of elements
        buf = torch.zeros((B, S, H, D + 3), dtype=kd.dtype, device=dev)
        buf[..., :D] = kd.transpose(1, 2)
        kd = buf.transpose(1, 2)[..., :D]
        qd = qd.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == 2:  # slots before heads, aligned
        kd = kd.transpose(1, 2).contiguous().transpose(1, 2)
    sc = D ** -0.5 if scale is None else scale
    got = q.qrita_cache_weights(qd, kd, wd, put(dev, n), positions=put(dev, at), seen=put(dev, seen), decay=decay, scale=scale)
    assert got.data_ptr() == wd.data_ptr()
    got = got.cpu().numpy().astype(np.float64)
    k64, q64 = rounded(k, dtype), rounded(qq, dtype)
    with np.errstate(invalid="ignore", over="ignore"):
        for b in range(B):
            m = max(int(n[b]), 0)
            for h in range(H):
                want = w[b, h].astype(np.float64)
                add = cache_weights(q64[b, :, h * G:(h + 1) * G], k64[b, h], np.arange(S) if at is None else at[b, h], m,
                                    m if seen is None else int(seen[b]), sc)
                want[:m] = want[:m] * decay + add
                fin = np.nan_to_num(k64[b, h, :m], nan=0.0, posinf=0.0, neginf=0.0)
                A = np.abs(fin) @ np.abs(q64[b, :, h * G:(h + 1) * G]).reshape(T * G, D).T if m else np.zeros((1, 1))
                A = A.max() * abs(sc)
                d = 2 * (D * 2.0**-22 * A + 2.0**-23 * A)
                tol = 2 * (d + 2.0**-21 + S * 2.0**-24) * np.abs(np.r_[np.nan_to_num(add), np.zeros(S - m)]) + 2.0**-22 * np.abs(np.nan_to_num(want))
                tol[m:] = 0
                g = got[b, h]
                assert np.array_equal(np.isnan(g), np.isnan(want)), (b, h)
                bad = ~(np.abs(g - want) <= tol) & ~np.isnan(want)
                assert not bad.any(), (b, h, np.flatnonzero(bad)[:4], g[bad][:4], want[bad][:4])


# one slot, part of a tile, several tiles a warp, clusters; more slots than scores are kept for
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("bf16", 40), ("f32", 64), ("f32", 33), ("bf16", 256), ("bf16", 96)])
@pytest.mark.parametrize("S", [1, 15, 200, 1037])
def test_weights_of_one_query(dev, dtype, D, S):
    check_weights(dev, S + D, 5, 2, 4, 1, S, D, dtype, evicted=S % 2 == 1)


@pytest.mark.parametrize("G,T", [(1, 1), (3, 1), (8, 2), (1, 33), (4, 32), (5, 21)])
@pytest.mark.parametrize("evicted", [False, True])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 32), ("bf16", 32)])
def test_weights_of_windows(dev, G, T, evicted, dtype, D):
    """Several queries: some before the first slot (short sequences), all causal."""
    check_weights(dev, G * T, 4, 2, G, T, 300, D, dtype, evicted)
    check_weights(dev, G * T + 1, 1, 1, G, T, max(2, T // 2), D, dtype)


@pytest.mark.parametrize("layout", [0, 1, 2])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_of_strided_caches_and_decays(dev, layout, dtype):
    for decay in (1.0, 0.0):
        check_weights(dev, 3 + layout, 4, 3, 2, 3, 130, 64, dtype, layout=layout, decay=decay, scale=0.3)


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("f32", 20)])
@pytest.mark.parametrize("T", [1, 9])
def test_weights_of_nan_and_infinite_keys(dev, dtype, D, T):
    check_weights(dev, 17, 4, 2, 2, T, 140, D, dtype, special=True)


def test_weights_of_long_caches(dev):
    check_weights(dev, 5, 1, 1, 2, 1, 70001, 64, "bf16")
    check_weights(dev, 6, 1, 1, 8, 5, 33000, 64, "bf16", evicted=True)
    check_weights(dev, 7, 20, 9, 1, 2, 500, 32, "bf16")
    check_weights(dev, 8, 1, 1, 16, 1, 40000, 32, "bf16")  # clusters of 16 with most of an SM's memory each
    check_weights(dev, 9, 1, 1, 16, 1, 70000, 32, "bf16")  # scores that fit nowhere


def test_weights_of_windows_over_several_tiles(dev):
    """One CTA a kv head (many of them), and shares of several tiles."""
    check_weights(dev, 11, 160, 2, 1, 40, 700, 64, "bf16", evicted=True)
    check_weights(dev, 12, 1, 2, 8, 40, 5000, 72, "bf16", scale=-0.1)
    check_weights(dev, 13, 2, 1, 4, 9, 3000, 200, "bf16", evicted=True, scale=0.0)
    check_weights(dev, 14, 4, 2, 40, 5, 600, 128, "bf16", special=True)
    check_weights(dev, 15, 2, 3, 7, 7, 900, 128, "bf16", layout=2)
    check_weights(dev, 16, 3, 2, 128, 2, 300, 64, "bf16", layout=1)


def test_weights_decay_zero_reads_nothing(dev):
    import torch

    import top_selection_row_gb300 as q

    k, qq = torch.randn(1, 1, 40, 64, device=dev), torch.randn(1, 1, 2, 64, device=dev)
    w = torch.full((1, 1, 40), float("nan"), device=dev)
    n = torch.tensor([30], dtype=torch.int32, device=dev)
    got = q.qrita_cache_weights(qq, k, w, n, decay=0.0)
    assert bool(got[0, 0, :30].isfinite().all()) and bool(got[0, 0, 30:].isnan().all())
    # two heads' softmax weights add up to two (sums of 30 terms of fp32, each within 2^-20)
    assert abs(float(got[0, 0, :30].sum()) - 2.0) < 2.0 * 31 * 2.0**-20


def check_evict(dev, seed, B, H, S, budget, sink, recent, dtype, evicted, D=(24, 16), levels=None, more=0, special=False, layout=0):
    import torch

    import top_selection_row_gb300 as q

    rng = np.random.default_rng(seed)
    n, at, seen = cache(rng, B, H, S, evicted)
    w = rng.random((B, H, S)).astype(np.float32) if levels is None else rng.integers(0, levels, (B, H, S)).astype(np.float32)
    if special:
        w[:, :, ::5] = np.nan
        w[:, :, 1::7] = np.inf
        w[:, :, 2::7] = -np.inf
        w[:, :, 3::11] = -0.0
        w[:, :, 4::11] = -1.0
    make = lambda d: torch.randint(0, 100, (B, H, S, d), device=dev).to(dtype)  # noqa: E731
    k, v = make(D[0]), make(D[1])
    if layout:
        k = k.transpose(1, 2).contiguous().transpose(1, 2)
        pad = torch.zeros((B, H, S, D[1] + 1), dtype=dtype, device=dev)
        pad[..., :-1] = v
        v = pad[..., :-1]
    out = None
    if more:
        z = lambda *s, dt=torch.int32: torch.full(s, 9, dtype=dt, device=dev)  # noqa: E731
        out = q.EvictedCache(z(B, H, budget + more, D[0], dt=dtype), z(B, H, budget + more, D[1], dt=dtype), z(B, H, budget + more, dt=torch.float32),
                             z(B, H, budget + more), z(B, H, budget), z(B))
    got = q.qrita_cache_evict(k, v, put(dev, w), put(dev, n), budget, sink, recent, positions=put(dev, at), seen=put(dev, seen), out=out)
    ks, vs = k.float().cpu().numpy(), v.float().cpu().numpy()
    gk, gv, gw, gp, gs, gl = (t.float().cpu().numpy() if t.dtype.itemsize < 4 or t.dtype.is_floating_point else t.cpu().numpy() for t in got)
    keep = np.minimum(np.maximum(n, 0), budget)
    assert np.array_equal(gl, keep)
    for b in range(B):
        m = max(int(n[b]), 0)
        for h in range(H):
            pos = np.arange(S) if at is None else at[b, h]
            order = kept_order(w[b, h], pos, m, m if seen is None else int(seen[b]), sink, recent)
            slots = np.array(sorted(order[: keep[b]]), int)
            pad = budget - len(slots)
            assert np.array_equal(gs[b, h], np.r_[slots, [-1] * pad]), (b, h)
            assert np.array_equal(gp[b, h, :budget], np.r_[pos[slots], [-1] * pad])
            assert np.array_equal(gw[b, h, :budget], np.r_[w[b, h][slots], [0.0] * pad], equal_nan=True)
            for g, x in ((gk, ks), (gv, vs)):
                assert np.array_equal(g[b, h, : len(slots)], x[b, h][slots]) and not g[b, h, len(slots):budget].any()
    if more:
        for g in (gk, gv, gw, gp):
            assert (g[:, :, budget:] == 9).all()


@pytest.mark.parametrize("evicted", [False, True])
@pytest.mark.parametrize("S,budget,sink,recent", [(1, 1, 0, 0), (40, 60, 2, 3), (200, 200, 0, 0), (333, 100, 4, 16), (1000, 1, 0, 0), (1000, 999, 1, 1),
                                                  (3001, 700, 3, 650), (20000, 5000, 4, 64), (500, 64, 40, 40), (700, 130, 0, 699)])
def test_evict(dev, S, budget, sink, recent, evicted):
    import torch

    B = 4 if S < 5000 else 2
    check_evict(dev, S + budget, B, 3, S, budget, sink, recent, torch.bfloat16, evicted)
    check_evict(dev, S + budget + 1, B, 2, S, budget, sink, recent, torch.uint8, evicted, levels=3, D=(5, 7))


@pytest.mark.parametrize("layout", [0, 1])
def test_evict_types_layouts_and_special_weights(dev, layout):
    import torch

    for i, dt in enumerate((torch.float32, torch.float16, torch.bfloat16, torch.int8, torch.float64)):
        check_evict(dev, i, 4, 2, 300, 77, 3, 9, dt, i % 2 == 0, special=i != 1, layout=layout, more=0 if i % 2 else 5, D=((24, 16), (8, 64), (1, 3))[i % 3])


def test_evict_long_and_many(dev):
    import torch

    check_evict(dev, 1, 1, 1, 120_001, 30_000, 4, 100, torch.int8, False, D=(4, 16))
    check_evict(dev, 2, 1, 2, 1_000_003, 1000, 4, 100, torch.int8, False, D=(1, 1), levels=50)
    check_evict(dev, 3, 30, 20, 300, 50, 1, 5, torch.float16, True)


@pytest.mark.parametrize("H,S,budget,sink,recent", [(1, 8, 8, 0, 0), (3, 50, 33, 2, 5), (8, 700, 700, 4, 64), (20, 40, 40, 0, 39), (2, 3000, 3000, 10, 2000),
                                                    (2, 30, 30, 40, 40)])
def test_insert(dev, H, S, budget, sink, recent):
    """Several tokens one after another into short, empty, full and idle sequences."""
    import torch

    import top_selection_row_gb300 as q

    rng = np.random.default_rng(S)
    B, D = 6, (24, 10)
    n = np.array([budget, budget - 1, 0, -1, budget, S], np.int32)
    seen = np.where(n < 0, 3, np.minimum(n, budget) + rng.integers(0, 50, B) * (n >= budget)).astype(np.int32)
    at = np.full((B, H, S), -7, np.int32)
    for b in range(B):
        m = min(max(n[b], 0), budget)
        for h in range(H):
            at[b, h, :m] = rng.permutation(rng.choice(max(seen[b], 1), m, replace=False)) if m else at[b, h, :0]
    w = np.where(rng.random((B, H, S)) < 0.3, 0.0, rng.random((B, H, S))).astype(np.float32)
    w[0, 0, 1::3] = np.nan
    k, v = torch.randn(B, H, S, D[0], device=dev).bfloat16(), torch.randn(B, S, H, D[1], device=dev).half().transpose(1, 2)
    wd, pd, nd, sd = (put(dev, x.copy()) for x in (w, at, n, seen))
    wk, wv = k.clone(), v.clone()
    for step in range(3):
        nk, nv = torch.randn(B, H, D[0], device=dev).bfloat16(), torch.randn(H, B, D[1], device=dev).half().transpose(0, 1)
        got = q.qrita_cache_insert(k, v, wd, pd, nd, sd, nk, nv, budget, sink, recent).cpu().numpy()
        for b in range(B):
            if n[b] < 0:
                assert (got[b] == -1).all()
                continue
            m = min(int(n[b]), budget)
            for h in range(H):
                s = m if m < budget else kept_order(w[b, h], at[b, h], m, int(seen[b]), sink, recent)[-1]
                assert got[b, h] == s, (step, b, h)
                w[b, h, s], at[b, h, s] = 0, seen[b]
                wk[b, h, s], wv[b, h, s] = nk[b, h], nv[b, h]
            n[b] = min(m + 1, budget)
            seen[b] += 1
        assert torch.equal(k, wk) and torch.equal(v, wv)
        for d, x in ((wd, w), (pd, at), (nd, n), (sd, seen)):
            assert np.array_equal(d.cpu().numpy(), x, equal_nan=True), step


def decode(dev, steps=4):
    """A prompt's weights, its eviction into a cache with room, then tokens put in and
    the weights that their queries add: outputs of every step."""
    import torch

    import top_selection_row_gb300 as q

    g = torch.Generator(device=dev).manual_seed(3)
    B, H, G, S, D, budget = 3, 2, 4, 400, 64, 100
    rand = lambda *s: torch.randn(*s, generator=g, device=dev).bfloat16()  # noqa: E731
    k, v, n = rand(B, H, S, D), rand(B, H, S, D), torch.tensor([400, 90, 250], dtype=torch.int32, device=dev)
    tokens = [(rand(B, H, D), rand(B, H, D), rand(B, 1, H * G, D)) for _ in range(steps)]
    window = rand(B, 16, H * G, D)

    def run():
        w = torch.zeros(B, H, S, device=dev)
        q.qrita_cache_weights(window, k, w, n)
        c = q.qrita_cache_evict(k, v, w, n, budget, sink=4, recent=16)
        seen, slots = n.clone(), []
        for nk, nv, qq in tokens:
            slots.append(q.qrita_cache_insert(c.keys, c.values, c.weights, c.positions, c.lengths, seen, nk, nv, budget, sink=4, recent=16))
            q.qrita_cache_weights(qq, c.keys, c.weights, c.lengths, positions=c.positions, seen=seen, decay=0.95)
        return [*c, seen, *slots]

    return run


def test_a_run_together_captured_and_on_another_stream(dev):
    import torch

    run = decode(dev)
    want = [t.clone() for t in run()]
    assert want[5].tolist() == [100, 94, 100] and want[6].tolist() == [404, 94, 254]
    # protected positions are there: the sinks, and the last sixteen
    at = want[3].cpu().numpy()
    for b, s in enumerate((404, 94, 254)):
        for h in range(2):
            held = set(at[b, h].tolist())
            assert {0, 1, 2, 3} | set(range(s - 16, s)) <= held and len(held - {-1}) == min(100, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for _ in range(2):
        for t in held:
            t.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_stream_argument(dev):
    import torch

    import top_selection_row_gb300 as q

    side = torch.cuda.Stream()
    k = torch.randn(2, 2, 50, 32, device=dev)
    w, n = torch.rand(2, 2, 50, device=dev), torch.tensor([50, 20], dtype=torch.int32, device=dev)
    qq = torch.randn(2, 1, 4, 32, device=dev)
    want = q.qrita_cache_evict(k, k, q.qrita_cache_weights(qq, k, w.clone(), n), n, 10)
    torch.cuda.synchronize()
    w2 = q.qrita_cache_weights(qq, k, w, n, stream=side)
    got = q.qrita_cache_evict(k, k, w2, n, 10, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals_of_the_binding(dev):
    import torch

    import top_selection_row_gb300 as q

    k = torch.zeros(2, 2, 10, 32, device=dev)
    w, n = torch.zeros(2, 2, 10, device=dev), torch.zeros(2, dtype=torch.int32, device=dev)
    at, nk, qq = torch.zeros(2, 2, 10, dtype=torch.int32, device=dev), torch.zeros(2, 2, 32, device=dev), torch.zeros(2, 1, 4, 32, device=dev)
    bad = [lambda: q.qrita_cache_weights(qq[:, :, :3], k, w, n), lambda: q.qrita_cache_weights(qq.bfloat16(), k, w, n),
           lambda: q.qrita_cache_weights(qq.half(), k.half(), w, n), lambda: q.qrita_cache_weights(qq, k, w[:, :, :9], n),
           lambda: q.qrita_cache_weights(qq, k, w, n, positions=at), lambda: q.qrita_cache_weights(qq, k, w, n.long()),
           lambda: q.qrita_cache_weights(qq, k, w, n, decay=2.0), lambda: q.qrita_cache_weights(qq, k.transpose(2, 3), w, n),
           lambda: q.qrita_cache_weights(qq[:1], k, w, n),
           lambda: q.qrita_cache_evict(k, k[:, :, :9], w, n, 4), lambda: q.qrita_cache_evict(k, k, w, n, 0),
           lambda: q.qrita_cache_evict(k, k, w, n, 4, out=(k, k, w, at, at, n)), lambda: q.qrita_cache_evict(k, k, w, n, 4, sink=-1),
           lambda: q.qrita_cache_insert(k, k, w, at, n, n, nk, nk, 11), lambda: q.qrita_cache_insert(k, k, w, None, n, n, nk, nk, 5),
           lambda: q.qrita_cache_insert(k, k, w, at, n, n, nk.half(), nk, 5), lambda: q.qrita_cache_insert(k, k, w, at, n, n, nk[:, :1], nk, 5),
           lambda: q.qrita_cache_insert(k[:, :1].expand(2, 2, 10, 32), k, w, at, n, n, nk, nk, 5)]
    for call in bad:
        with pytest.raises((ValueError, TypeError, q.QritaError)):
            call()
    # an expanded head is read as it is
    one = torch.randn(2, 1, 10, 32, device=dev)
    n.fill_(10)
    a = q.qrita_cache_weights(qq + 1, one.expand(2, 2, 10, 32), w.clone(), n)
    assert torch.equal(a, q.qrita_cache_weights(qq + 1, one.expand(2, 2, 10, 32).contiguous(), w.clone(), n))


def test_offsets_past_32_bits(dev):
    """Heads of a cache, and rows of logits, more than 2^31 elements apart: the same as
    side by side."""
    import torch

    import top_selection_row_gb300 as q

    far = 2**31 + 64
    buf = torch.empty(far + 2**16, dtype=torch.bfloat16, device=dev)
    gen = torch.Generator(device=dev).manual_seed(4)
    near = torch.randn(1, 2, 300, 64, generator=gen, device=dev).bfloat16()
    k = buf.as_strided((1, 2, 300, 64), (2 * far, far, 64, 1))
    k.copy_(near)
    n = torch.tensor([290], dtype=torch.int32, device=dev)
    w = torch.rand(1, 2, 300, generator=gen, device=dev)
    for T in (1, 40):
        qq = torch.randn(1, T, 8, 64, generator=gen, device=dev).bfloat16()
        assert torch.equal(q.qrita_cache_weights(qq, k, w.clone(), n), q.qrita_cache_weights(qq, near, w.clone(), n))
    assert all(torch.equal(a, b) for a, b in zip(q.qrita_cache_evict(k, k, w, n, 50), q.qrita_cache_evict(near, near, w, n, 50)))
    out = q.qrita_cache_evict(near, near, w, n, 50)
    far_out = out._replace(keys=buf.as_strided((1, 2, 50, 64), (2 * far, far, 64, 1)), values=torch.empty_like(out.values))
    got = q.qrita_cache_evict(near, near, w, n, 50, out=far_out)
    assert torch.equal(got.keys, q.qrita_cache_evict(near, near, w, n, 50).keys)
    k.copy_(near)
    state = [[w.clone(), torch.arange(300, dtype=torch.int32, device=dev).expand(1, 2, 300).contiguous(), n + 10, n + 10] for _ in range(2)]
    new = torch.randn(1, 2, 64, generator=gen, device=dev).bfloat16()
    slots = [q.qrita_cache_insert(c, c.clone() if c is near else near.clone(), *s, new, new, 300) for c, s in zip((k, near), state)]
    assert torch.equal(*slots) and torch.equal(k, near)
    x = torch.randn(2, 9000, generator=gen, device=dev).bfloat16()
    rows = buf.as_strided((2, 9000), (far, 1))
    rows.copy_(x)
    ids = torch.randint(0, 9000, (2, 4), generator=gen, device=dev, dtype=torch.int32)
    a, b = (q.qrita_token_scores(v, ids, top=9, entropy=True, rank=True) for v in (rows, x))
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    g = torch.randn(2, 4, generator=gen, device=dev)
    want = q.qrita_token_scores_grad(x, ids, g)
    assert torch.equal(q.qrita_token_scores_grad(rows, ids, g, out_grad=rows), want)
