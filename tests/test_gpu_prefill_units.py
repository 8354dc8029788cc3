"""Prompt attention where every CTA runs several units one after the other: stages and parities go on
from unit to unit. Each value of o is held to its own bound (prefill_bounds.py), so that a few lost
rows of V show; lse as in test_gpu_prefill.py."""
import numpy as np
import pytest
import torch

import memory_bounded_kv_b200 as kvb
from gpu_util import host
import prefill_bounds as bounds
from test_gpu_prefill import f64, forward, make, reference

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
