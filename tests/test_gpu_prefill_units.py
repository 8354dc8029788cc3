"""Prompt attention where every CTA runs several units one after the other: stages and parities go on
from unit to unit. Each value of o is held to its own bound (prefill_bounds.py), so that a few lost
rows of V show; lse as in test_gpu_prefill.py."""
import numpy as np
import pytest
import torch

import memory_bounded_kv_b200 as kvb
from gpu_util import host
import prefill_bounds as bounds
from test_gpu_prefill import backward, f64, forward, make, reference

pytestmark = pytest.mark.gpu

# documents that end on a tile after as many tiles as the loads' stages, between ones that end inside a tile
LENGTHS = [256, 256, 70, 256, 100, 512, 64, 130, 256, 1, 200, 129, 256, 255, 385, 512, 90, 127, 256, 65, 128, 3, 257, 448,
           256, 191, 640, 31, 256, 77]


def starts(n, seed):
    return np.r_[0, np.cumsum(np.random.default_rng(seed).permutation(n))].tolist()


@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("beta", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d", [(16, 16, 128), (32, 8, 128), (16, 16, 64), (32, 8, 64)])
def test_several_units_a_cta(Hq, Hkv, d, beta, softcap):
    cu = starts(LENGTHS, d + Hq)
    c = make(60, cu, cu[-1], Hq, Hkv, d, beta)
    args = [f64(c[n]) for n in ("q", "k", "v", "lb")]
    want, bound = bounds.forward(*args, cu, None, softcap)
    lse_want = reference(c, None, softcap)["lse"]
    for _ in range(4):
        o, lse = forward(c, None, softcap)
        bounds.within(f64(o), want, bound, "o")
        np.testing.assert_allclose(f64(lse), lse_want, rtol=2e-6, atol=4e-6)
    assert kvb.kvb_get_error() == 0


@pytest.mark.parametrize("beta", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_a_neighbours_nan_in_v_between_units(d, beta):
    """Every second document's V is NaN: it reaches its own rows alone, whatever a stage held before."""
    Hq = Hkv = 16
    cu = starts(LENGTHS, 61)
    c = make(61, cu, cu[-1], Hq, Hkv, d, beta)
    want, bound = bounds.forward(*[f64(c[n]) for n in ("q", "k", "v", "lb")], cu)
    for s, e in list(zip(cu[:-1], cu[1:]))[::2]:
        c["v"][s:e] = float("nan")
        want[s:e] = np.nan
    for _ in range(4):
        o, _ = forward(c)
        bounds.within(f64(o), want, bound, "o")
    assert kvb.kvb_get_error() == 0 and host(c["cu"])[-1] == cu[-1]


@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("beta", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d", [(16, 16, 128), (16, 8, 64)])
def test_gradients_of_several_units_a_cta(Hq, Hkv, d, beta, softcap):
    """Units of one tile and of several in turn, with rows that have one key above half the weight: every value
    within its bound, and the same bits each time."""
    cu = starts(LENGTHS, 62 + d)
    c = make(62, cu, cu[-1], Hq, Hkv, d, beta, grads=True, d_lse=True)
    if beta:
        c["lb"][:, ::2] -= 3
    a = [f64(c[n]) for n in ("q", "k", "v", "lb")]
    want = bounds.gradients(*a, cu, f64(c["d_o"]), f64(c["d_lse"]), None, softcap)
    o, lse = forward(c, None, softcap)
    first = backward(c, o, lse, None, softcap)
    for n, x in first.items():
        if x is not None:
            bounds.within(f64(x), *want[n], n)
    for _ in range(6):
        again = backward(c, o, lse, None, softcap)
        assert all(x is None or torch.equal(x, again[n]) for n, x in first.items())
    assert kvb.kvb_get_error() == 0


@pytest.mark.parametrize("beta", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_a_neighbours_nan_in_the_gradients_of_several_units(d, beta):
    """Every second document is NaN throughout: the others' gradients are theirs."""
    cu = starts(LENGTHS, 63)
    c = make(63, cu, cu[-1], 16, 8, d, beta, grads=True)
    want = bounds.gradients(*[f64(c[n]) for n in ("q", "k", "v", "lb")], cu, f64(c["d_o"]))
    for s, e in list(zip(cu[:-1], cu[1:]))[::2]:
        for n in ("q", "k", "v", "d_o"):
            c[n][s:e] = float("nan")
        for n in want:
            want[n][0][s:e] = np.nan
    o, lse = forward(c)
    for n, x in backward(c, o, lse).items():
        if x is not None:
            bounds.within(f64(x), *want[n], n)
    assert kvb.kvb_get_error() == 0
