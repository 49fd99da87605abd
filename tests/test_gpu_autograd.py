"""Tensors that the caller gives for outputs are written in place: autograd sees
it, and refuses a backward pass that would read an overwritten value."""

import numpy as np
import pytest

from test_gpu_losses import dev, put  # noqa: F401

pytestmark = pytest.mark.gpu

B, V = 6, 1000


def inputs(dev):
    import torch

    g = torch.Generator(device=dev).manual_seed(2)
    h = torch.randn(B, 32, generator=g, device=dev)
    w = torch.randn(32, V, generator=g, device=dev).requires_grad_()
    t = torch.randint(0, V, (B,), generator=g, device=dev, dtype=torch.int32)
    adv = torch.randn(B, generator=g, device=dev)
    return h, w, t, adv, put(dev, np.array([0, 2, 6], np.int32))


CALLS = [lambda q, x, t, adv, s, **k: q.qrita_token_logprobs_grad(x, t, adv, **k),
         lambda q, x, t, adv, s, **k: q.qrita_policy_loss(x, t, None, adv, **k).grad,
         lambda q, x, t, adv, s, **k: q.qrita_preference_loss(x, t, s, **k).grad]


@pytest.mark.parametrize("call", CALLS)
def test_a_producer_that_saved_its_logits_is_told(dev, call):
    import torch

    import top_selection_row_gb300 as q

    h, w, t, adv, s = inputs(dev)
    x = torch.tanh(h @ w)  # (its backward pass reads what it gave out)
    want = call(q, x, t, adv, s)
    x.backward(want, retain_graph=True)
    got = call(q, x, t, adv, s, out_grad=x.detach())
    assert torch.equal(got, want) and got.data_ptr() == x.data_ptr()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        x.backward(got)


@pytest.mark.parametrize("call", CALLS)
def test_a_producer_that_did_not_takes_the_gradient(dev, call):
    import torch

    import top_selection_row_gb300 as q

    h, w, t, adv, s = inputs(dev)
    x = h @ w
    x.backward(call(q, x, t, adv, s))
    want, w.grad = w.grad, None
    x = h @ w
    x.backward(call(q, x, t, adv, s, out_grad=x.detach()))
    assert torch.equal(w.grad, want)


def test_every_given_tensor_has_a_new_version(dev):
    import torch

    import top_selection_row_gb300 as q

    h, w, t, adv, s = inputs(dev)
    x = (h @ w).detach()
    k, p, u = torch.full((B,), 20, dtype=torch.int32, device=dev), torch.full((B,), 0.9, device=dev), torch.full((B,), 0.5, device=dev)
    mask = q.qrita_select(x, k, p)
    ids, probs, count, token = q.qrita_candidates(x, mask, 32, u=u)
    calls = [(lambda out: q.qrita_token_logprobs(x, t, entropy=True, out=out), q.qrita_token_logprobs(x, t, entropy=True)),
             (lambda out: q.qrita_policy_loss(x, t, None, adv, entropy=True, out=out), q.qrita_policy_loss(x, t, None, adv, entropy=True)),
             (lambda out: q.qrita_preference_loss(x, t, s, out=out), q.qrita_preference_loss(x, t, s)),
             (lambda out: q.qrita_select(x, k, p, out=out[0]), (mask,)),
             (lambda out: q.qrita_topk_ids(x, k, 32, out_mask=out[0], out_ids=out[1]), (mask, ids)),
             (lambda out: q.qrita_candidates(x, mask, 32, u=u, out=out), (ids, probs, count, token)),
             (lambda out: q.qrita_select_host(x.cpu(), k.cpu(), p.cpu(), out=out[0]), (mask.cpu(),))]
    for call, out in calls:
        before = [v._version for v in out]
        call(out)
        assert all(v._version > n for v, n in zip(out, before))
    with torch.inference_mode():  # (tensors without versions are written as they are)
        y = x + 1
        q.qrita_policy_loss(y, t, None, adv, out_grad=y)
    assert q.qrita_token_logprobs_grad(y, t, adv, out_grad=y).data_ptr() == y.data_ptr()
