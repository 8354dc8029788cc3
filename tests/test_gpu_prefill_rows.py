"""Prompt attention and its gradients, every value held to its own bound (prefill_bounds.py): a norm over a
whole tensor passes with a row of it wrong."""
import numpy as np
import pytest
import torch

import memory_bounded_kv_b200 as kvb
import prefill_bounds as bounds
from test_gpu_prefill import REL, SHAPES, backward, f64, forward, make

pytestmark = pytest.mark.gpu


def check(c, prefix=None, softcap=0.0, scale=0.0):
    cu, d_lse = c["cu"].tolist(), c["d_lse"]
    a = [f64(c[n]) for n in ("q", "k", "v", "lb")]
    o, lse = forward(c, prefix, softcap, scale)
    bounds.within(f64(o), *bounds.forward(*a, cu, prefix, softcap, scale), "o")
    g = backward(c, o, lse, prefix, softcap, scale)
    want = bounds.gradients(*a, cu, f64(c["d_o"]), None if d_lse is None else f64(d_lse), prefix, softcap, scale)
    for n, x in g.items():
        if x is not None:
            bounds.within(f64(x), *want[n], n)
    assert kvb.kvb_get_error() == 0


@pytest.mark.parametrize("beta", [True, False])
@pytest.mark.parametrize("cu,T,Hq,Hkv,d", SHAPES)
def test_values(cu, T, Hq, Hkv, d, beta):
    check(make(100, cu, T, Hq, Hkv, d, beta, grads=True, d_lse=T % 2 == 1))


@pytest.mark.parametrize("beta", [True, False])
@pytest.mark.parametrize("softcap,prefix,scale", [(20.0, None, 0.0), (0.0, [5, 0, 9999, -3], 0.2), (3.0, [129, 40, 1, 200], 0.0)])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (8, 1, 128), (2, 2, 128)])
def test_values_cap_prefix_scale(Hq, Hkv, d, softcap, prefix, scale, beta):
    check(make(101, [0, 260, 300, 420, 800], 805, Hq, Hkv, d, beta, grads=True, d_lse=True), prefix, softcap, scale)


@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (8, 2, 128), (2, 2, 128)])
@pytest.mark.parametrize("low,high", [(-5.0, -3.0), (-20.0, -0.1)])
def test_values_where_decay_leaves_few_keys(low, high, Hq, Hkv, d, softcap):
    """log beta of -3 to -5: a row's weight is almost all at one or two keys, dq and d_log_beta are small
    differences, and an estimate of delta from the stored o (rows past the first 128 keys) would show in dq.
    The whole's error is REL again, as where the weight is spread."""
    c = make(102, [0, 500, 640], 641, Hq, Hkv, d, grads=True, d_lse=True)
    c["lb"] = low + (high - low) * torch.rand(c["lb"].shape, generator=torch.Generator().manual_seed(7)).cuda()
    check(c, None, softcap)
    far = slice(128, 500)
    o, lse = forward(c, None, softcap)
    got = f64(backward(c, o, lse, None, softcap)["dq"])[far]
    want = bounds.gradients(*[f64(c[n]) for n in ("q", "k", "v", "lb")], [0, 500, 640], f64(c["d_o"]), f64(c["d_lse"]), None,
                            softcap)["dq"][0][far]
    assert np.linalg.norm(got - want) <= REL * np.linalg.norm(want)


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (8, 2, 128)])
def test_values_where_one_far_key_takes_all(Hq, Hkv, d):
    """Rows whose weight is at a single far key among many: one key in 200 has a score of about 12, the others one
    of about -4 (below 16, as the bounds want)."""
    L = 1200
    c = make(103, [0, L], L, Hq, Hkv, d, False, grads=True)
    far = (torch.arange(L) % 200 == 0).cuda()[:, None, None]
    c["q"] = (c["q"] * 0.1 + 1).to(torch.bfloat16)
    c["k"] = (c["k"] * 0.1 + torch.where(far, 12.0, -4.0) / d ** 0.5).to(torch.bfloat16)
    check(c)
