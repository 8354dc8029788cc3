"""Prompt attention and its gradients when a CTA's bounded wait runs out (a testing hook ends its loads
after one tile): KVB_DERR_TIMEOUT is set, what the CTA had not written keeps what it held, nothing else is
off, and the next call is right again."""
import functools

import numpy as np
import pytest

import memory_bounded_kv_b200 as kvb
from memory_bounded_kv_b200 import _lib
import prefill_bounds as bounds
from test_gpu_prefill import backward, f64, forward, make

pytestmark = pytest.mark.gpu
LIMIT = 20_000_000   # ns: well above what any wait of these calls takes
LONG = ([0, 2000], 8, 2)                                # one document: key blocks cut into pieces
MANY = (np.r_[0, np.cumsum([300, 129, 256, 77] * 5)].tolist(), 8, 8)   # whole key blocks, several a CTA
FORMS = [(64, True, 0.0), (64, False, 0.0), (64, True, 20.0), (128, True, 0.0), (128, False, 0.0), (128, True, 20.0)]


@functools.lru_cache(maxsize=None)
def case(kind, d, beta, softcap):
    cu, Hq, Hkv = dict(long=LONG, many=MANY)[kind]
    c = make(80, cu, cu[-1], Hq, Hkv, d, beta, grads=True)
    a = [f64(c[n]) for n in ("q", "k", "v", "lb")]
    return c, dict(o=bounds.forward(*a, cu, None, softcap), **bounds.gradients(*a, cu, f64(c["d_o"]), None, None, softcap))


def all_within(got, want, lost=None):
    """Every value within its bound, or where lost(name, value) says so still 7."""
    for n, x in got.items():
        if x is None:
            continue
        x, (w, bound) = f64(x), want[n]
        if lost is not None:
            gone = lost(n, x)
            assert 0 < gone.sum() < gone.size, n
            w, bound = np.where(gone, 7.0, w), np.where(gone, 0.0, bound)
        bounds.within(x, w, bound, n)


@pytest.mark.parametrize("kind,cta", [("long", 0), ("long", 5), ("many", 3)])
@pytest.mark.parametrize("d,beta,softcap", FORMS)
def test_forward(d, beta, softcap, kind, cta):
    c, want = case(kind, d, beta, softcap)
    kvb.kvb_test_withhold_next_prefill(0, cta, LIMIT)
    o, lse = forward(c, None, softcap)
    assert kvb.kvb_get_error() == _lib.DERR_TIMEOUT
    all_within(dict(o=o), want, lambda n, x: np.broadcast_to((x == 7).all(-1, keepdims=True), x.shape))
    assert bool((lse[(o == 7).all(-1)] == 7).all())
    o, lse = forward(c, None, softcap)
    all_within(dict(o=o), want)
    assert kvb.kvb_get_error() == 0


@pytest.mark.parametrize("kind", ["long", "many"])
@pytest.mark.parametrize("d,beta,softcap", FORMS)
def test_gradients_by_query_rows(d, beta, softcap, kind):
    """Without all deltas there are no gradients by keys."""
    c, want = case(kind, d, beta, softcap)
    o, lse = forward(c, None, softcap)
    kvb.kvb_test_withhold_next_prefill(1, 2, LIMIT)
    g = backward(c, o, lse, None, softcap)
    assert kvb.kvb_get_error() == _lib.DERR_TIMEOUT
    for n in ("dk", "dv", "d_log_beta"):
        assert g[n] is None or bool((g[n] == 7).all()), n
    all_within(dict(dq=g["dq"]), want, lambda n, x: np.broadcast_to((x == 7).all(-1, keepdims=True), x.shape))
    all_within(backward(c, o, lse, None, softcap), want)
    assert kvb.kvb_get_error() == 0


@pytest.mark.parametrize("kind,cta", [("long", 0), ("long", 1), ("long", 40), ("many", 3)])
@pytest.mark.parametrize("d,beta,softcap", FORMS)
def test_gradients_by_keys(d, beta, softcap, kind, cta):
    """Key blocks that the CTA has a part in keep what they held; no sum takes in what was never written."""
    c, want = case(kind, d, beta, softcap)
    cu = c["cu"].tolist()
    o, lse = forward(c, None, softcap)
    kvb.kvb_test_withhold_next_prefill(2, cta, LIMIT)
    g = backward(c, o, lse, None, softcap)
    assert kvb.kvb_get_error() == _lib.DERR_TIMEOUT
    all_within(dict(dq=g.pop("dq")), want)

    def whole_blocks(n, x):
        gone = np.zeros(x.shape, bool)
        for s0, e in zip(cu[:-1], cu[1:]):
            for s in range(s0, e, 128):
                for h in range(x.shape[1]):
                    gone[s:min(s + 128, e), h] = (x[s:min(s + 128, e), h] == 7).all()
        return gone
    all_within(g, want, whole_blocks)
    all_within(backward(c, o, lse, None, softcap), want)
    assert kvb.kvb_get_error() == 0


def test_a_hook_for_another_kernel_waits():
    """The hook is taken by the kernel it names alone, once."""
    c, want = case("long", 64, True, 0.0)
    kvb.kvb_test_withhold_next_prefill(2, 0, LIMIT)
    o, lse = forward(c)
    assert kvb.kvb_get_error() == 0
    backward(c, o, lse)
    assert kvb.kvb_get_error() == _lib.DERR_TIMEOUT
    all_within(backward(c, o, lse), want)
    assert kvb.kvb_get_error() == 0
