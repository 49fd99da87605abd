"""Refusals of the cache's entry points: every bad argument is answered before any
device work (no GPU here; pointers are never dereferenced)."""

import ctypes
import math

import pytest

from test_abi_losses import EINVAL, NULL, VP, L  # noqa: F401

K, V, OK_, OV = VP(0x10000000), VP(0x20000000), VP(0x30000000), VP(0x40000000)
F, I = VP(0x50000000), VP(0x60000000)  # noqa: E741
BASE = dict(B=2, H=4, S=100, lengths=I, weights=F, positions=NULL, seen=NULL)


def strides(*v):
    return (ctypes.c_int64 * 3)(*v)


def weights(L, **kw):  # noqa: F811
    a = {**BASE, "q": V, "dtype": 1, "T": 2, "G": 2, "D": 64, "qs": strides(1024, 512, 64), "keys": K,
         "ks": strides(25600, 6400, 64), "scale": 0.125, "decay": 1.0, **kw}
    return L.qrita_cache_weights(a["B"], a["H"], a["S"], a["q"], a["dtype"], a["T"], a["G"], a["D"], a["qs"], a["keys"], a["ks"],
                                 a["scale"], a["decay"], a["lengths"], a["positions"], a["seen"], a["weights"], NULL)


CACHE = dict(budget=10, sink=1, recent=2, keys=K, kb=128, ks=strides(51200, 12800, 128), values=V, vb=64, vs=strides(25600, 6400, 64))


def evict(L, **kw):  # noqa: F811
    a = {**BASE, **CACHE, "ok": OK_, "oks": strides(5120, 1280, 128), "ov": OV, "ovs": strides(2560, 640, 64), "oS": 10, "ow": VP(0x70000000),
         "op": I, "os": I, "ol": I, **kw}
    return L.qrita_cache_evict(a["B"], a["H"], a["S"], a["lengths"], a["weights"], a["positions"], a["seen"], a["budget"], a["sink"],
                               a["recent"], a["keys"], a["kb"], a["ks"], a["values"], a["vb"], a["vs"], a["ok"], a["oks"], a["ov"],
                               a["ovs"], a["oS"], a["ow"], a["op"], a["os"], a["ol"], NULL)


def insert(L, **kw):  # noqa: F811
    a = {**BASE, **CACHE, "positions": I, "seen": I, "nk": OK_, "nks": strides(512, 128), "nv": OV, "nvs": strides(256, 64), "os": I, **kw}
    return L.qrita_cache_insert(a["B"], a["H"], a["S"], a["lengths"], a["seen"], a["weights"], a["positions"], a["budget"], a["sink"],
                                a["recent"], a["keys"], a["kb"], a["ks"], a["values"], a["vb"], a["vs"], a["nk"], a["nks"], a["nv"],
                                a["nvs"], a["os"], NULL)


def _id(b):
    return " ".join(f"{k}={v if isinstance(v, (int, float)) else getattr(v, 'value', list(v) if hasattr(v, '__len__') else v)}" for k, v in b.items())


@pytest.mark.parametrize("call", [weights, evict, insert])
@pytest.mark.parametrize("bad", [dict(B=-1), dict(H=0), dict(S=0), dict(S=2**31), dict(B=2**31), dict(lengths=NULL), dict(weights=NULL),
                                 dict(keys=NULL)], ids=_id)
def test_bad_caches(L, call, bad):  # noqa: F811
    assert call(L, **bad) == EINVAL


@pytest.mark.parametrize("call", [weights, evict])
def test_positions_and_seen_come_together(L, call):  # noqa: F811
    assert call(L, positions=I) == EINVAL and call(L, seen=I) == EINVAL


@pytest.mark.parametrize("bad", [dict(dtype=2), dict(T=0), dict(G=0), dict(D=0), dict(D=1025), dict(T=4097), dict(q=NULL), dict(qs=None), dict(ks=None),
                                 dict(scale=math.inf), dict(scale=math.nan), dict(scale=1e39), dict(decay=-0.1), dict(decay=1.1),
                                 dict(decay=math.nan), dict(keys=VP(0x10000001)), dict(q=VP(0x20000001)), dict(ks=strides(-1, 6400, 64)),
                                 dict(qs=strides(1024, 512, 2**57))], ids=_id)
def test_bad_weights(L, bad):  # noqa: F811
    assert weights(L, **bad) == EINVAL


@pytest.mark.parametrize("call", [evict, insert])
@pytest.mark.parametrize("bad", [dict(budget=0), dict(budget=-1), dict(sink=-1), dict(recent=-1), dict(kb=0), dict(vb=2**20 + 1), dict(ks=None),
                                 dict(values=NULL), dict(vs=strides(25600, 6400, 63)), dict(os=NULL)], ids=_id)
def test_bad_rows(L, call, bad):  # noqa: F811
    assert call(L, **bad) == EINVAL


@pytest.mark.parametrize("bad", [dict(oS=9), dict(oS=2**31), dict(ow=NULL), dict(op=NULL), dict(ol=NULL), dict(ok=NULL), dict(ok=K), dict(ov=V), dict(ov=K), dict(ow=F),
                                 dict(ok=VP(0x10000000 + 51200)), dict(ok=VP(0x10000000 - 128))], ids=_id)
def test_bad_evictions(L, bad):  # noqa: F811
    assert evict(L, **bad) == EINVAL


@pytest.mark.parametrize("bad", [dict(budget=101), dict(nk=NULL), dict(nvs=None), dict(positions=NULL, seen=NULL), dict(seen=NULL)], ids=_id)
def test_bad_insertions(L, bad):  # noqa: F811
    assert insert(L, **bad) == EINVAL


def test_nothing_to_do_and_too_much(L):  # noqa: F811
    assert weights(L, B=0, q=NULL, keys=NULL) == evict(L, B=0, keys=NULL) == insert(L, B=0, keys=NULL) == 0
    for call in (weights, evict, insert):
        assert call(L, B=2**30, H=2**10) == 2  # more CTAs than a grid has
