"""Infinities, NaN and the largest finite numbers within a document of the prompt attention.

The kernels compute the weights of different columns in different ways, so each case stands at eight
columns in a row. The bounds are prefill_bounds.py's."""
import pytest
import torch

import memory_bounded_kv_b200 as kvb
import prefill_bounds as bounds
from test_gpu_prefill import backward, f64, forward, make

pytestmark = pytest.mark.gpu
L, Hq, Hkv = 300, 4, 2


def clean(d, seed, grads=False):
    c = make(seed, [0, L], L, Hq, Hkv, d, grads=grads)
    return c, bounds.forward(*[f64(c[n]) for n in ("q", "k", "v", "lb")], [0, L])


def rows_below(j, o, want, bound, what):
    w = want.copy()
    w[j:] = float("nan")
    bounds.within(f64(o), w, bound, what)


@pytest.mark.parametrize("where", ["k", "log_beta", "infinity"])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("d", [64, 128])
def test_nan_of_one_key_reaches_every_row_that_sees_it(d, softcap, where):
    """A score that is NaN (a NaN in k or log beta; q.k of two infinities of opposite sign) makes o, lse and the
    gradients of its row NaN, and no earlier row's o."""
    c, _ = clean(d, 70, True)
    want, bound = bounds.forward(*[f64(c[n]) for n in ("q", "k", "v", "lb")], [0, L], None, softcap)
    for j in range(200, 208):
        b = dict(c, **{n: c[n].clone() for n in ("k", "lb", "q")})
        first = j
        if where == "k":
            b["k"][j, :, 5] = float("nan")
        elif where == "log_beta":
            b["lb"][j] = float("nan")
            first = j + 1               # at distance 0 it has no use
        else:
            b["k"][j, :, 0], b["k"][j, :, 1] = float("inf"), float("-inf")
            b["q"][j:, :, :2] = 1.0
        o, lse = forward(b, None, softcap)
        g = backward(b, o, lse, None, softcap)
        assert torch.isnan(o[first:]).all() and torch.isnan(lse[first:]).all(), j
        assert torch.isnan(g["dq"][first:]).all(), j
        # the last row sees every key
        assert torch.isnan(g["dv"]).all() and torch.isnan(g["d_log_beta"][:-1]).all(), j
        rows_below(j, o, want, bound, "o")
        assert torch.isfinite(lse[:j]).all(), j
    assert kvb.kvb_get_error() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_large_values_of_unseen_tokens_weigh_nothing(d):
    """v_j of 3e38 (and for the gradients 1e36, whose products with d_o stay finite) leaves the rows before j alone."""
    c, (want, bound) = clean(d, 71, True)
    o0, lse0 = forward(c)
    dq0 = backward(c, o0, lse0)["dq"]
    for j in range(200, 208):
        b = dict(c, v=c["v"].clone())
        b["v"][j] = 3e38
        o, lse = forward(b)
        rows_below(j, o, want, bound, "o")
        assert torch.equal(lse, lse0)
        b["v"][j] = 1e36
        o, lse = forward(b)
        assert torch.equal(backward(b, o, lse)["dq"][:j], dq0[:j]), j
    assert kvb.kvb_get_error() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_infinite_scores(d):
    """A score of -inf is a key of weight 0; one of +inf makes its row NaN, as inf - inf in the formula."""
    c, _ = clean(d, 72)
    for j in range(200, 208):
        b = dict(c, **{n: c[n].clone() for n in ("k", "q", "v")})
        b["q"][:, :, 0] = 1.0
        b["k"][j, :, 0] = float("-inf")
        b["k"][j, :, 1:] = 0.0
        b["v"][j] = 3e38
        o, lse = forward(b)
        # the same without the key: its score so low that the weight is exactly 0
        a = dict(b, k=b["k"].clone(), v=b["v"].clone())
        a["k"][j, :, 0], a["v"][j] = -1e30, 0.0
        want, bound = bounds.forward(*[f64(a[n]) for n in ("q", "k", "v", "lb")], [0, L])
        bounds.within(f64(o)[:j], want[:j], bound[:j], "before")
        bounds.within(f64(o)[j + 1:], want[j + 1:], bound[j + 1:], "after")
        assert torch.isfinite(lse[j + 1:]).all()
        b["k"][j, :, 0] = float("inf")
        o, lse = forward(b)
        assert torch.isnan(o[j:]).all() and torch.isnan(lse[j:]).all(), j
        bounds.within(f64(o)[:j], want[:j], bound[:j], "before")
    assert kvb.kvb_get_error() == 0
