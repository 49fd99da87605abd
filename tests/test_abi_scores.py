"""Refusals of the scores' entry points: every bad argument is answered before any
device work (no GPU here; pointers are never dereferenced)."""

import pytest

from test_abi_losses import BAD_ROWS, EINVAL, F, GRAD, NULL, ROWS, T, VP, L, _rows  # noqa: F401


def scores(L, **kw):
    a = {**ROWS, "M": 2, "N": 5, "logp": F, "rank": NULL, "H": NULL, "ids": T, "top": F, **kw}
    r = _rows(a)
    return L.qrita_token_scores(*r[:7], a["M"], a["N"], r[7], a["logp"], a["rank"], a["H"], a["ids"], a["top"], NULL)


def scores_grad(L, **kw):
    a = {**ROWS, **GRAD, "K": 3, "g": F, "h": NULL, **kw}
    r = _rows(a)
    return L.qrita_token_scores_grad(*r[:7], a["K"], r[7], a["g"], a["h"], a["out_grad"], a["ld_grad"], NULL)


@pytest.mark.parametrize("call", [scores, scores_grad])
@pytest.mark.parametrize("bad", BAD_ROWS, ids=lambda b: " ".join(f"{k}={v}" for k, v in b.items()))
def test_bad_rows(L, call, bad):  # noqa: F811
    assert call(L, **bad) == EINVAL


@pytest.mark.parametrize("bad", [dict(M=-1), dict(M=8193), dict(N=-1), dict(N=129), dict(M=0, rank=T), dict(M=0, N=0),
                                 dict(logp=NULL), dict(ids=NULL), dict(top=NULL)],
                         ids=lambda b: " ".join(f"{k}={v}" for k, v in b.items()))
def test_bad_scores(L, bad):  # noqa: F811
    assert scores(L, **bad) == EINVAL


@pytest.mark.parametrize("bad", [dict(K=0), dict(K=257), dict(g=NULL), dict(out_grad=NULL), dict(ld_grad=99),
                                 dict(out_grad=VP(0x900001)), dict(out_grad=VP(0x100000 + 64))],
                         ids=lambda b: " ".join(f"{k}={v}" for k, v in b.items()))
def test_bad_gradients(L, bad):  # noqa: F811
    assert scores_grad(L, **bad) == EINVAL


def test_nothing_to_do(L):  # noqa: F811
    assert scores(L, B=0, logits=NULL, tokens=NULL) == 0
    assert scores_grad(L, B=0, logits=NULL, tokens=NULL, out_grad=NULL) == 0
