"""The cache's entry points with flags: the same refusals as without, and unknown flags
(no GPU here; pointers are never dereferenced, and no call here is a valid one)."""

import ctypes

import pytest

from test_abi_cache import BASE, CACHE, K, OK_, OV, V, strides
from test_abi_cache_overlap import OUT, READ
from test_abi_losses import EINVAL, NULL, L  # noqa: F401


def weights_ex(L, flags=0, **kw):  # noqa: F811
    a = {**BASE, "q": V, "dtype": 1, "T": 2, "G": 2, "D": 64, "qs": strides(1024, 512, 64), "keys": K,
         "ks": strides(25600, 6400, 64), "scale": 0.125, "decay": 1.0, **kw}
    return L.qrita_cache_weights_ex(a["B"], a["H"], a["S"], a["q"], a["dtype"], a["T"], a["G"], a["D"], a["qs"], a["keys"], a["ks"],
                                    a["scale"], a["decay"], a["lengths"], a["positions"], a["seen"], a["weights"],
                                    ctypes.c_uint32(flags), NULL)


def evict_ex(L, flags=0, **kw):  # noqa: F811
    a = {**BASE, **CACHE, **READ, **OUT, "ok": OK_, "oks": strides(5120, 1280, 128), "ov": OV, "ovs": strides(2560, 640, 64), "oS": 10, **kw}
    return L.qrita_cache_evict_ex(a["B"], a["H"], a["S"], a["lengths"], a["weights"], a["positions"], a["seen"], a["budget"], a["sink"],
                                  a["recent"], a["keys"], a["kb"], a["ks"], a["values"], a["vb"], a["vs"], a["ok"], a["oks"], a["ov"],
                                  a["ovs"], a["oS"], a["ow"], a["op"], a["os"], a["ol"], ctypes.c_uint32(flags), NULL)


@pytest.mark.parametrize("call,flags", [(weights_ex, 4), (evict_ex, 1), (evict_ex, 2)] + [(c, f) for c in (weights_ex, evict_ex) for f in (8, 0x1000, 0x80000001)])
def test_unknown_flags(L, call, flags):  # noqa: F811
    assert call(L, flags) == EINVAL


@pytest.mark.parametrize("flags", [0, 4])
@pytest.mark.parametrize("bad", [dict(budget=0), dict(oS=9), dict(ok=NULL), dict(ok=K), dict(ol=READ["lengths"]), dict(S=0)], ids=str)
def test_bad_evictions(L, bad, flags):  # noqa: F811
    assert evict_ex(L, flags, **bad) == EINVAL


@pytest.mark.parametrize("flags", [0, 1, 2, 3])
@pytest.mark.parametrize("bad", [dict(dtype=2), dict(T=0), dict(D=1025), dict(q=NULL), dict(keys=NULL), dict(decay=1.1), dict(S=0), dict(lengths=NULL)],
                         ids=str)
def test_bad_weights(L, bad, flags):  # noqa: F811
    assert weights_ex(L, flags, **bad) == EINVAL


def test_flags_match_the_header():
    import os
    import re

    import top_selection_row_gb300 as q

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "qrita.h")) as f:
        flags = re.findall(r"#define QRITA_(CACHE_FLAG_\w+) (0x\w+)u", f.read())
    assert len(flags) == 3
    for name, value in flags:
        assert getattr(q, name) == int(value, 16), name
