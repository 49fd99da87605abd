"""Vectors of the cache's entry points that overlap where one of them is written: refused
before any device work (no GPU here; pointers are never dereferenced, and no call here
is a valid one)."""

import pytest

from test_abi_cache import K, V, evict, insert, strides, weights
from test_abi_losses import EINVAL, NULL, VP, L  # noqa: F401

# vectors apart from each other: 2 x 4 x 100 weights and positions of 4 bytes, 2 lengths, 2 x 4 x 10 slots
W, AT, N, SEEN, OW, OAT, OS, ON = (VP(0x50000000 + i * 0x100000) for i in range(8))
READ = dict(lengths=N, weights=W, positions=AT, seen=SEEN)
OUT = dict(ow=OW, op=OAT, os=OS, ol=ON)


def behind(p, n):
    return VP(p.value + n)


CASES = [
    (evict, dict(ol=N)), (evict, dict(ol=SEEN)), (evict, dict(ol=behind(N, 4))), (evict, dict(ol=behind(W, 3196))),
    (evict, dict(ow=W)), (evict, dict(ow=behind(W, 3196))), (evict, dict(ow=AT)), (evict, dict(op=AT)), (evict, dict(op=W)),
    (evict, dict(os=AT)), (evict, dict(os=N)), (evict, dict(os=W)), (evict, dict(os=OAT)), (evict, dict(os=OW)), (evict, dict(ol=OS)),
    (evict, dict(op=OW)), (evict, dict(ol=N, positions=NULL, seen=NULL)),
    (insert, dict(seen=N)), (insert, dict(lengths=behind(SEEN, 4))), (insert, dict(weights=AT)), (insert, dict(os=N)),
    (insert, dict(os=W)), (insert, dict(os=behind(AT, 3196))), (insert, dict(lengths=W)),
    (weights, dict(weights=AT)), (weights, dict(weights=N)), (weights, dict(weights=behind(SEEN, 4))),
]


@pytest.mark.parametrize("call,over", CASES, ids=lambda v: v.__name__ if callable(v) else " ".join(f"{k}={p.value or 0:#x}" for k, p in v.items()))
def test_overlapping_vectors(L, call, over):  # noqa: F811
    assert call(L, **{**READ, **({} if call is weights else {**OUT} if call is evict else dict(os=OS)), **over}) == EINVAL


# the refusals of tests/test_abi_cache.py, where nothing else is amiss
@pytest.mark.parametrize("bad", [dict(budget=0), dict(budget=-1), dict(sink=-1), dict(recent=-1), dict(kb=0), dict(vb=2**20 + 1), dict(ks=None),
                                 dict(values=NULL), dict(vs=strides(25600, 6400, 63)), dict(os=NULL), dict(S=0), dict(lengths=NULL),
                                 dict(weights=NULL), dict(keys=NULL)], ids=str)
@pytest.mark.parametrize("call", [evict, insert])
def test_bad_arguments_of_vectors_apart(L, call, bad):  # noqa: F811
    assert call(L, **{**READ, **(OUT if call is evict else dict(os=OS)), **bad}) == EINVAL


@pytest.mark.parametrize("bad", [dict(oS=9), dict(oS=2**31), dict(ow=NULL), dict(op=NULL), dict(ol=NULL), dict(ok=NULL), dict(ok=K), dict(ov=V),
                                 dict(ov=K), dict(ok=VP(0x10000000 + 51200)), dict(ok=VP(0x10000000 - 128)), dict(seen=NULL)], ids=str)
def test_bad_evictions_of_vectors_apart(L, bad):  # noqa: F811
    assert evict(L, **{**READ, **OUT, **bad}) == EINVAL


@pytest.mark.parametrize("bad", [dict(budget=101), dict(nk=NULL), dict(nvs=None), dict(positions=NULL, seen=NULL), dict(seen=NULL)], ids=str)
def test_bad_insertions_of_vectors_apart(L, bad):  # noqa: F811
    assert insert(L, **{**READ, "os": OS, **bad}) == EINVAL
