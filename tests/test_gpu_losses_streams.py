"""Losses on another stream than the current one: what a call allocates, reads
and returns is ordered with that stream, not with the current one's backlog."""

import numpy as np
import pytest

from parity_helpers import to_device
from test_gpu_losses import dev, make_rows, put  # noqa: F401

pytestmark = pytest.mark.gpu

B, V = 16, 32000


def backlog(torch, dev):
    """A few milliseconds of work on the current stream."""
    work = torch.ones(4096, 4096, device=dev)

    def run():
        for _ in range(20):
            work @ work

    run()
    torch.cuda.synchronize()
    return run


def cases(dev, seed):
    import top_selection_row_gb300 as q

    rng, x, tokens, mask = make_rows(seed, B, V, "bf16", keep=40)
    x, t, m = to_device(x, "bf16", dev), put(dev, tokens), put(dev, mask)
    adv = put(dev, rng.standard_normal(B).astype(np.float32))
    starts = put(dev, np.array([0, 3, 8, 12, B], np.int32))
    return [lambda **k: q.qrita_token_logprobs(x, t, entropy=True, **k),
            lambda **k: (q.qrita_token_logprobs_grad(x, t, adv, **k),),
            lambda **k: q.qrita_policy_loss(x, t, None, adv, mask=m, entropy_coef=0.1, **k),
            lambda **k: q.qrita_preference_loss(x, t, starts, **k)]


def same(got, want):
    return all(u.data_ptr() != v.data_ptr() and u.equal(v) for u, v in zip(got, want))


@pytest.mark.parametrize("which", range(4))
def test_outputs_are_no_block_that_the_current_stream_still_uses(dev, which):
    """Temporaries of the outputs' sizes are dropped while the current stream has
    yet to write them; a call on an idle stream must not be given their memory."""
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


@pytest.mark.parametrize("which", range(4))
def test_a_call_on_a_busy_stream_and_one_on_an_idle_stream(dev, which):
    """The first call's workspace is dropped while its kernels wait; the second
    one, on other logits, must not write into it."""
    import torch

    first, second = cases(dev, 4)[which], cases(dev, 5)[which]
    want = first(), second()
    side, busy = torch.cuda.Stream(), backlog(torch, dev)
    for _ in range(4):
        busy()
        a = first()
        b = second(stream=side)
        torch.cuda.synchronize()
        assert same(a, want[0]) and same(b, want[1])


@pytest.mark.parametrize("which", range(4))
def test_results_dropped_while_the_current_stream_reads_them(dev, which):
    """Results of a call on another stream are read by the current one, which is
    behind, and dropped; later calls on that stream must leave them alone."""
    import torch

    first, second = cases(dev, 6)[which], cases(dev, 7)[which]
    want = first()
    side, busy = torch.cuda.Stream(), backlog(torch, dev)
    for _ in range(3):
        got = first(stream=side)
        side.synchronize()
        busy()
        read = [t.clone() for t in got]
        del got
        for _ in range(4):
            second(stream=side)
        torch.cuda.synchronize()
        assert same(read, want)


def test_a_stream_of_another_device_is_refused(dev):
    import torch

    import top_selection_row_gb300 as q

    class Elsewhere:
        device = torch.device("cuda", 7)

    x, t = torch.zeros(2, 10, device=dev), torch.zeros(2, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError):
        q.qrita_token_logprobs(x, t, stream=Elsewhere())


def test_a_call_on_a_captured_side_stream(dev):
    """A graph whose capture forks to another stream for the call and joins."""
    import torch

    calls = cases(dev, 8)
    want = [call() for call in calls]
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        held = [call(stream=side) for call in calls]
        main.wait_stream(side)
    for _ in range(3):
        for group in held:
            for t in group:
                t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(held, want):
            assert same(got, w)
