"""Selection, ranked ids and candidate lists on another stream than the current
one: their outputs, and the fills of unused entries, are that stream's."""

import numpy as np
import pytest

from test_gpu_losses import dev  # noqa: F401
from test_gpu_losses_streams import backlog, same

pytestmark = pytest.mark.gpu

B, V = 16, 32000


def cases(dev, seed):
    import torch

    import top_selection_row_gb300 as q

    rng = np.random.default_rng(seed)
    x = torch.from_numpy((rng.standard_normal((B, V)) * 2).astype(np.float32)).to(dev)
    k = torch.full((B,), 50, dtype=torch.int32, device=dev)
    p = torch.full((B,), 0.9, device=dev)
    u = torch.from_numpy(rng.random(B).astype(np.float32)).to(dev)
    mask = q.qrita_select(x, k, p)
    host = x.cpu().pin_memory()
    return [lambda **s: (q.qrita_select(x, k, p, **s),),
            lambda **s: q.qrita_select_ex(x, k, p, row_status=True, row_info=True, **s)[:2],
            lambda **s: q.qrita_topk_ids(x, k, 64, **s),
            lambda **s: q.qrita_candidates(x, mask, 64, u=u, **s),
            lambda **s: (q.qrita_select_host(host, k.cpu(), p.cpu(), **s),)]


@pytest.mark.parametrize("which", range(5))
def test_on_an_idle_stream_beside_a_busy_current_one(dev, which):
    """Temporaries of the outputs' sizes, not written yet when they are dropped;
    the call's outputs hold no block of theirs, and nothing fills them late."""
    import torch

    call, other = cases(dev, 3)[which], cases(dev, 4)[which]
    want = call()
    side, busy = torch.cuda.Stream(), backlog(torch, dev)
    call(stream=side)
    torch.cuda.synchronize()
    for _ in range(3):
        busy()
        for t in want:
            torch.full_like(t, 1, device=dev)
        got = call(stream=side)
        torch.cuda.synchronize()
        assert same(got, want)
    for _ in range(3):  # results dropped while the current stream has yet to read them
        got = call(stream=side)
        side.synchronize()
        busy()
        read = [t.clone() for t in got]
        del got
        for _ in range(4):
            other(stream=side)
        torch.cuda.synchronize()
        assert same(read, want)
