"""Scores and cache calls on another stream than the current one, and what autograd
sees of tensors that they write."""

import numpy as np
import pytest

from parity_helpers import to_device
from test_gpu_losses import dev, make_rows, put  # noqa: F401
from test_gpu_losses_streams import backlog, same

pytestmark = pytest.mark.gpu

B, V = 16, 32000


def cases(dev, seed):
    import torch

    import top_selection_row_gb300 as q

    rng, x, tokens, mask = make_rows(seed, B, V, "bf16", keep=40)
    x, m = to_device(x, "bf16", dev), put(dev, mask)
    t = put(dev, rng.integers(0, V, (B, 5)).astype(np.int32))
    g = put(dev, rng.standard_normal((B, 5)).astype(np.float32))
    gen = torch.Generator(device=dev).manual_seed(seed)
    k = torch.randn(2, 2, 500, 64, generator=gen, device=dev).bfloat16()
    w = torch.rand(2, 2, 500, generator=gen, device=dev)
    n = torch.tensor([500, 300], dtype=torch.int32, device=dev)
    return [lambda **kw: q.qrita_token_scores(x, t, top=20, mask=m, entropy=True, rank=True, **kw),
            lambda **kw: (q.qrita_token_scores_grad(x, t, g, **kw),),
            lambda **kw: q.qrita_cache_evict(k, k, w, n, 64, recent=8, **kw)]


@pytest.mark.parametrize("which", range(3))
def test_outputs_are_no_block_that_the_current_stream_still_uses(dev, which):  # noqa: F811
    import torch

    call = cases(dev, 3)[which]
    want = call()
    side, busy = torch.cuda.Stream(), backlog(torch, dev)
    call(stream=side)
    torch.cuda.synchronize()
    for _ in range(3):
        busy()
        for t in want:
            torch.full_like(t, 9)
        got = call(stream=side)
        torch.cuda.synchronize()
        assert same(got, want)


@pytest.mark.parametrize("which", range(3))
def test_a_call_on_a_captured_side_stream(dev, which):  # noqa: F811
    import torch

    call = cases(dev, 5)[which]
    want = call()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        held = call(stream=side)
        main.wait_stream(side)
    for _ in range(3):
        for t in held:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert same(held, want)


def test_beside_gradients_that_hold_tensor_memory(dev):  # noqa: F811
    """A window's weights (all of an SM's tensor memory) beside another stream's
    gradients, which keep parts of their rows in it."""
    import torch

    import top_selection_row_gb300 as q

    gen = torch.Generator(device=dev).manual_seed(1)
    k = torch.randn(4, 8, 4096, 128, generator=gen, device=dev).bfloat16()
    qq = torch.randn(4, 32, 32, 128, generator=gen, device=dev).bfloat16()
    n = torch.full((4,), 4096, dtype=torch.int32, device=dev)
    x = torch.randn(300, 100000, generator=gen, device=dev).bfloat16()
    ids = torch.randint(0, 100000, (300, 20), generator=gen, device=dev, dtype=torch.int32)
    g = torch.randn(300, 20, generator=gen, device=dev)
    weights = lambda **kw: q.qrita_cache_weights(qq, k, torch.zeros(4, 8, 4096, device=dev), n, **kw)  # noqa: E731
    want = weights(), q.qrita_token_scores_grad(x, ids, g)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a, b = [], []
        for _ in range(4):
            a.append(q.qrita_token_scores_grad(x, ids, g, stream=side))
            b.append(weights())
        torch.cuda.synchronize()
        assert all(torch.equal(v, want[1]) for v in a) and all(torch.equal(v, want[0]) for v in b)


def test_written_tensors_have_a_new_version(dev):  # noqa: F811
    import torch

    import top_selection_row_gb300 as q

    i32 = torch.int32
    x = torch.randn(3, 100, device=dev)
    k, w = torch.randn(2, 2, 20, 32, device=dev), torch.rand(2, 2, 20, device=dev)
    n, seen = torch.full((2,), 20, dtype=i32, device=dev), torch.full((2,), 20, dtype=i32, device=dev)
    at = torch.arange(20, dtype=i32, device=dev).expand(2, 2, 20).contiguous()
    v, new, one = k.clone(), torch.randn(2, 2, 32, device=dev), torch.randn(2, 1, 4, 32, device=dev)
    ids = torch.zeros(3, 2, dtype=i32, device=dev)
    scores = q.qrita_token_scores(x, ids, top=4, entropy=True, rank=True)
    cut = q.qrita_cache_evict(k, v, w, n, 8)
    slots = torch.empty(2, 2, dtype=i32, device=dev)
    for written, call in ((tuple(scores), lambda: q.qrita_token_scores(x, ids, top=4, entropy=True, rank=True, out=scores)),
                          ((x,), lambda: q.qrita_token_scores_grad(x, ids, torch.ones(3, 2, device=dev), out_grad=x)),
                          (tuple(cut), lambda: q.qrita_cache_evict(k, v, w, n, 8, out=cut)),
                          ((w,), lambda: q.qrita_cache_weights(one, k, w, n)),
                          ((k, v, w, at, n, seen, slots), lambda: q.qrita_cache_insert(k, v, w, at, n, seen, new, new, 20, out=slots))):
        before = [t._version for t in written]
        call()
        assert all(t._version > b for t, b in zip(written, before))
