"""Refusals of the loss entry points: every bad argument is answered before
any device work (no GPU here; pointers are never dereferenced)."""

import ctypes
import math
import os

import pytest

from top_selection_row_gb300.build import LIB_PATH, build_library

VP = ctypes.c_void_p
NULL = VP(0)
X, G, T, F, W = VP(0x100000), VP(0x900000), VP(0x2000000), VP(0x3000000), VP(0x4000000)
EINVAL = 1
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(LIB_PATH):
        build_library()
    import top_selection_row_gb300 as q

    return q.lib()


ROWS = dict(logits=X, dtype=1, B=4, V=100, ld=100, mask=NULL, tokens=T, inv_t=1.0)
GRAD = dict(out_grad=G, ld_grad=100)


def _rows(a):
    return [a[k] for k in ("logits", "dtype", "B", "V", "ld", "mask", "tokens", "inv_t")]


def logprobs(L, **kw):
    a = {**ROWS, "out_logp": F, "out_entropy": NULL, **kw}
    return L.qrita_token_logprobs(*_rows(a), a["out_logp"], a["out_entropy"], NULL)


def logprobs_grad(L, **kw):
    a = {**ROWS, **GRAD, "g": F, "h": NULL, **kw}
    return L.qrita_token_logprobs_grad(*_rows(a), a["g"], a["h"], a["out_grad"], a["ld_grad"], NULL)


def policy(L, **kw):
    a = {**ROWS, **GRAD, "adv": F, "lo": 0.2, "hi": 0.2, "kl": 0.0, "ent": 0.0, "loss": F, "row_loss": F, **kw}
    return L.qrita_policy_loss(*_rows(a), NULL, NULL, a["adv"], NULL, a["lo"], a["hi"], a["kl"], a["ent"], NULL, a["loss"],
                               a["row_loss"], NULL, NULL, NULL, a["out_grad"], a["ld_grad"], NULL)


def preference(L, **kw):
    a = {**ROWS, **GRAD, "starts": T, "P": 2, "beta": 0.1, "ls": 0.0, "margin": 0.0, "norm": 0, "loss": F, "pair": F,
         "ratio": F, "seq": F, "ws": W, "wsn": 1 << 20, **kw}
    return L.qrita_preference_loss(a["logits"], a["dtype"], a["B"], a["V"], a["ld"], a["tokens"], a["inv_t"], a["starts"],
                                   a["P"], NULL, NULL, a["beta"], a["ls"], a["margin"], a["norm"], NULL, a["loss"],
                                   a["pair"], a["ratio"], a["seq"], NULL, a["out_grad"], a["ld_grad"], a["ws"],
                                   ctypes.c_size_t(a["wsn"]), NULL)


BAD_ROWS = [
    dict(dtype=2), dict(B=-1), dict(B=2**31), dict(V=0), dict(V=2**31, ld=2**31), dict(ld=99), dict(logits=NULL),
    dict(tokens=NULL), dict(logits=VP(0x100001)), dict(inv_t=0.0), dict(inv_t=-1.0), dict(inv_t=INF), dict(inv_t=NAN),
    dict(inv_t=1e-45), dict(inv_t=1e300), dict(ld=2**62),
]


@pytest.mark.parametrize("call", [logprobs, logprobs_grad, policy, preference])
@pytest.mark.parametrize("bad", BAD_ROWS, ids=lambda b: " ".join(f"{k}={v}" for k, v in b.items()))
def test_bad_rows(L, call, bad):
    assert call(L, **bad) == EINVAL


@pytest.mark.parametrize("call", [logprobs_grad, policy, preference])
@pytest.mark.parametrize("bad", [
    dict(ld_grad=99), dict(out_grad=VP(0x900001)), dict(ld_grad=2**62),
    dict(out_grad=VP(0x100000), ld_grad=104),       # the logits' buffer with another leading dimension
    dict(out_grad=VP(0x100000 + 64)),               # a shifted overlap
    dict(out_grad=VP(0x100000 - 64)),
    dict(out_grad=VP(0x100000 + (3 * 100 + 99) * 2)),  # the last element
])
def test_bad_gradients(L, call, bad):
    assert call(L, **bad) == EINVAL


@pytest.mark.parametrize("shift", [1, 99, 157, 256 + 99, 256 + 157])
def test_gradients_beside_the_logits_that_share_elements(L, shift):
    # V = 100 in rows of 256: a gradient that starts 100 .. 156 elements on shares none
    assert policy(L, ld=256, ld_grad=256, out_grad=VP(0x100000 + 2 * shift)) == EINVAL


def test_missing_pointers(L):
    assert logprobs(L, out_logp=NULL) == EINVAL
    assert logprobs_grad(L, out_grad=NULL) == EINVAL
    assert logprobs_grad(L, g=NULL, h=NULL) == EINVAL
    assert policy(L, adv=NULL) == EINVAL
    assert policy(L, loss=NULL) == EINVAL
    assert policy(L, row_loss=NULL) == EINVAL
    for k in ("starts", "loss", "pair", "ratio", "seq", "ws"):
        assert preference(L, **{k: NULL}) == EINVAL


@pytest.mark.parametrize("bad", [dict(lo=-0.1), dict(lo=1.1), dict(lo=NAN), dict(hi=-0.1), dict(hi=NAN), dict(kl=-1.0),
                                 dict(kl=INF), dict(kl=NAN), dict(ent=INF), dict(ent=NAN)])
def test_bad_policy_scalars(L, bad):
    assert policy(L, **bad) == EINVAL


@pytest.mark.parametrize("bad", [dict(beta=0.0), dict(beta=-1.0), dict(beta=INF), dict(beta=NAN), dict(ls=-0.1), dict(ls=1.1),
                                 dict(ls=NAN), dict(margin=INF), dict(margin=NAN), dict(norm=2), dict(norm=-1), dict(P=-1),
                                 dict(P=2**30), dict(ws=VP(0x4000008)), dict(wsn=16)])
def test_bad_preference_arguments(L, bad):
    assert preference(L, **bad) == EINVAL


def test_workspace_bytes(L):
    f = L.qrita_preference_workspace_bytes
    assert f(-1, 1) == f(1, -1) == f(2**31, 1) == f(1, 2**30) == 0
    assert f(0, 0) == 256
    for B, P in ((1, 1), (1000, 7), (2**31 - 1, 2**30 - 1)):
        n = f(B, P)
        assert n % 256 == 0 and n >= 16 * B + 16 * P


def test_empty_batches_launch_nothing(L):
    assert logprobs(L, B=0, logits=NULL, tokens=NULL, out_logp=NULL) == 0
    assert logprobs_grad(L, B=0, logits=NULL, tokens=NULL, out_grad=NULL, g=NULL) == 0


def test_binding_refuses_before_any_device_work():
    torch = pytest.importorskip("torch")
    import top_selection_row_gb300 as q

    x, t, f = torch.zeros(3, 10), torch.zeros(3, dtype=torch.int32), torch.zeros(3)
    for call in (lambda: q.qrita_token_logprobs(x, t), lambda: q.qrita_token_logprobs_grad(x, t, f),
                 lambda: q.qrita_policy_loss(x, t, f, f), lambda: q.qrita_preference_loss(x, t, t)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
