"""qrita_policy_loss_ex: the same refusals as without flags, and unknown flags (no
GPU here; pointers are never dereferenced)."""

import ctypes

import pytest

from test_abi_losses import BAD_ROWS, EINVAL, F, GRAD, L, NULL, ROWS, _rows  # noqa: F401


def policy_ex(L, flags=0, **kw):
    a = {**ROWS, **GRAD, "adv": F, "loss": F, "row_loss": F, **kw}
    return L.qrita_policy_loss_ex(*_rows(a), NULL, NULL, a["adv"], NULL, 0.2, 0.2, 0.0, 0.0, NULL, a["loss"], a["row_loss"],
                                  NULL, NULL, NULL, a["out_grad"], a["ld_grad"], ctypes.c_uint32(flags), NULL)


@pytest.mark.parametrize("bad", BAD_ROWS + [dict(adv=NULL), dict(loss=NULL), dict(row_loss=NULL), dict(ld_grad=99)],
                         ids=lambda b: " ".join(f"{k}={v}" for k, v in b.items()))
@pytest.mark.parametrize("flags", [0, 1])
def test_bad_arguments(L, bad, flags):
    assert policy_ex(L, flags, **bad) == EINVAL


@pytest.mark.parametrize("flags", [2, 3, 0x1000, 0x80000000])
def test_unknown_flags(L, flags):
    assert policy_ex(L, flags) == EINVAL


@pytest.mark.parametrize("inv_t", [9e-31, 1.1e30, 1e-38, 1e38])
def test_temperatures_outside_the_stated_range(L, inv_t):
    assert policy_ex(L, inv_t=inv_t) == EINVAL
    assert L.qrita_token_logprobs(*_rows({**ROWS, "inv_t": inv_t}), F, NULL, NULL) == EINVAL
