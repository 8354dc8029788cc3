"""GPU parity of the prompt's path against the float64 host reference (prefill_ref.py).

Tolerances. o and the bf16 gradients, as relative 2-norms: 2^-8 for the rounding of the result to
bf16 (half a step) and 2^-8 for the softmax weights and their gradients, which enter the second
matrix products as bf16: 2^-7. lse: a logit is an fp32 sum of d products whose partial sums stay
below 16 in these inputs, off by 2^-22 of that (4e-6); the exponentials, their sum and the logarithm
add 2^-22 relative each (with the logits' own: 2e-6 of |lse|). d_log_beta is fp32 throughout: each of
p, d_o . v and delta is off by at most 5e-6 relative (from the logits and lse), three of them and the
sums: 2e-5 as a relative 2-norm."""
import numpy as np
import pytest
import torch

import memory_bounded_kv_b200 as kvb
from memory_bounded_kv_b200 import _lib
from memory_bounded_kv_b200.cache import PagedKVCache
from gpu_util import host
import prefill_ref as ref

pytestmark = pytest.mark.gpu
PAGE = _lib.PAGE_SLOTS
REL = 2.0 ** -7


def make(seed, cu, T, Hq, Hkv, d, beta=True, grads=False, d_lse=False):
    g = torch.Generator().manual_seed(seed)
    bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()   # noqa: E731
    c = dict(q=bf(T, Hq, d), k=bf(T, Hkv, d), v=bf(T, Hkv, d), cu=torch.tensor(cu, dtype=torch.int32).cuda(), lb=None)
    if beta:
        c["lb"] = torch.nn.functional.logsigmoid(torch.randn(T, Hkv, generator=g) * 1.5 + 2).cuda()
    if grads:
        c["d_o"] = bf(T, Hq, d)
        c["d_lse"] = torch.randn(T, Hq, generator=g).cuda() if d_lse else None
    return c


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def forward(c, prefix=None, softcap=0.0, scale=0.0, stream=None):
    T, Hq, d = c["q"].shape
    o = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    p = None if prefix is None else torch.tensor(prefix, dtype=torch.int32).cuda()
    kvb.kvb_prefill_attn(c["q"], c["k"], c["v"], c["lb"], c["cu"], o, lse, prefix_len=p, softcap=softcap, scale=scale,
                         stream=stream)
    return o, lse


def backward(c, o, lse, prefix=None, softcap=0.0, scale=0.0):
    T, Hq, d = c["q"].shape
    Hkv = c["k"].shape[1]
    out = dict(dq=torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda"),
               dk=torch.full((T, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda"),
               dv=torch.full((T, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda"),
               d_log_beta=None if c["lb"] is None else torch.full((T, Hkv), 7.0, device="cuda"))
    ws = torch.full((kvb.kvb_prefill_attn_bwd_workspace_bytes(T, Hq),), 255, dtype=torch.uint8, device="cuda")
    p = None if prefix is None else torch.tensor(prefix, dtype=torch.int32).cuda()
    kvb.kvb_prefill_attn_bwd(c["q"], c["k"], c["v"], c["lb"], c["cu"], o, lse, c["d_o"], c["d_lse"], out["dq"], out["dk"],
                             out["dv"], out["d_log_beta"], ws, prefix_len=p, softcap=softcap, scale=scale)
    return out


def reference(c, prefix=None, softcap=0.0, scale=0.0):
    return ref.attention(f64(c["q"]), f64(c["k"]), f64(c["v"]), f64(c["lb"]), host(c["cu"]), prefix, softcap, scale,
                         f64(c.get("d_o")), f64(c.get("d_lse")))


def rel(x, y):
    n = np.linalg.norm(y)
    return float(np.linalg.norm(x - y) / n) if n else float(np.linalg.norm(x))


def check(got, want, tol, what):
    """Rows of documents within tol; the others as they were (7)."""
    got = f64(got)
    rows = ~np.isnan(want.reshape(want.shape[0], -1)[:, 0]) if want.shape[0] else np.zeros(0, bool)
    assert np.all(got[~rows] == 7.0), f"{what}: a row of no document was written"
    assert np.all(np.isfinite(got)), what
    r = rel(got[rows], want[rows])
    assert r <= tol, f"{what}: {r:.3e} > {tol:.1e}"


def check_state(o, lse, r, what=""):
    check(o, r["o"], REL, what + " o")
    rows = ~np.isnan(r["lse"][:, 0])
    assert np.all(f64(lse)[~rows] == 7.0), what
    w = r["lse"][rows]
    np.testing.assert_allclose(f64(lse)[rows], w, rtol=2e-6, atol=4e-6, err_msg=what + " lse")


def check_grads(got, r, what=""):
    for n in ("dq", "dk", "dv"):
        check(got[n], r[n], REL, f"{what} {n}")
    if got["d_log_beta"] is not None:
        check(got["d_log_beta"], r["d_log_beta"], 2e-5, what + " d_log_beta")


SHAPES = [
    # documents, rows, Hq, Hkv, d
    ([0, 1], 1, 1, 1, 64),
    ([0, 1, 2, 3], 3, 8, 1, 128),
    ([0, 17], 17, 8, 2, 64),
    ([0, 127, 127, 255, 256], 260, 4, 4, 128),
    ([3, 131, 260, 260], 301, 16, 4, 128),
    ([0, 64, 193, 700], 703, 8, 8, 64),
    ([0, 300, 301, 1100], 1100, 8, 1, 128),
    ([0, 1025], 1025, 4, 2, 64),
    ([0, 513, 1100], 1111, 2, 2, 128),
]


@pytest.mark.parametrize("beta", [True, False])
@pytest.mark.parametrize("cu,T,Hq,Hkv,d", SHAPES)
def test_forward(cu, T, Hq, Hkv, d, beta):
    c = make(1, cu, T, Hq, Hkv, d, beta)
    o, lse = forward(c)
    check_state(o, lse, reference(c))
    assert kvb.kvb_get_error() == 0


@pytest.mark.parametrize("softcap,prefix", [(20.0, None), (0.0, [5, 0, 9999, -3]), (3.0, [129, 40, 1, 200])])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (8, 1, 128), (2, 2, 128)])
def test_forward_cap_and_prefix(softcap, prefix, Hq, Hkv, d):
    cu = [0, 260, 300, 420, 800]
    c = make(2, cu, 805, Hq, Hkv, d)
    o, lse = forward(c, prefix, softcap)
    check_state(o, lse, reference(c, prefix, softcap))


@pytest.mark.parametrize("d_lse", [False, True])
@pytest.mark.parametrize("cu,T,Hq,Hkv,d", SHAPES)
def test_gradients(cu, T, Hq, Hkv, d, d_lse):
    c = make(3, cu, T, Hq, Hkv, d, grads=True, d_lse=d_lse)
    o, lse = forward(c)
    check_grads(backward(c, o, lse), reference(c))
    assert kvb.kvb_get_error() == 0


@pytest.mark.parametrize("beta", [True, False])
@pytest.mark.parametrize("softcap,prefix", [(20.0, None), (0.0, [5, 0, 9999, -3]), (3.0, [129, 40, 1, 200])])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (8, 1, 128), (2, 2, 128)])
def test_gradients_cap_and_prefix(softcap, prefix, Hq, Hkv, d, beta):
    cu = [0, 260, 300, 420, 800]
    c = make(4, cu, 805, Hq, Hkv, d, beta, grads=True, d_lse=True)
    o, lse = forward(c, prefix, softcap)
    check_grads(backward(c, o, lse, prefix, softcap), reference(c, prefix, softcap))


def test_gradients_against_differences():
    """d_log_beta and dv against central differences of L = sum o . d_o + lse . d_lse of the reference
    itself (its own gradient formulas are held to the definition here)."""
    g = np.random.default_rng(5)
    T, Hq, Hkv, d = 9, 2, 1, 64
    q, k, v = g.normal(size=(T, Hq, d)), g.normal(size=(T, Hkv, d)), g.normal(size=(T, Hkv, d))
    lb, d_o, d_l = -np.abs(g.normal(size=(T, Hkv))), g.normal(size=(T, Hq, d)), g.normal(size=(T, Hq))
    cu, pre, cap = [0, 6, 9], [3, 0], 2.0

    def loss(**kw):
        a = dict(q=q, k=k, v=v, log_beta=lb)
        a.update(kw)
        r = ref.attention(a["q"], a["k"], a["v"], a["log_beta"], cu, pre, cap)
        return float((r["o"] * d_o).sum() + (r["lse"] * d_l).sum())
    r = ref.attention(q, k, v, lb, cu, pre, cap, 0.0, d_o, d_l)
    h = 1e-5
    for name, x, grad in (("q", q, "dq"), ("k", k, "dk"), ("v", v, "dv"), ("log_beta", lb, "d_log_beta")):
        for at in [tuple(g.integers(0, s) for s in x.shape) for _ in range(6)]:
            up, dn = x.copy(), x.copy()
            up[at] += h
            dn[at] -= h
            num = (loss(**{name: up}) - loss(**{name: dn})) / (2 * h)
            # central differences: h^2 / 6 of the third derivative plus 2^-53 |L| / h
            assert abs(num - r[grad][at]) <= 1e-6 * max(1.0, abs(num)), (name, at, num, r[grad][at])


def test_strided_inputs_and_other_stream():
    T, Hq, Hkv, d = 333, 8, 2, 64
    c = make(6, [0, 100, 333], T, Hq, Hkv, d, grads=True)
    qkv = torch.zeros(T, Hq + 2 * Hkv, d, dtype=torch.bfloat16, device="cuda")   # one fused projection's output
    qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:] = c["q"], c["k"], c["v"]
    e = dict(c, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], lb=c["lb"].t().contiguous().t())
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    o, lse = forward(c)
    s.wait_stream(torch.cuda.current_stream())
    o2 = torch.full_like(o, 7.0)
    lse2 = torch.full_like(lse, 7.0)
    s.wait_stream(torch.cuda.current_stream())
    kvb.kvb_prefill_attn(e["q"], e["k"], e["v"], e["lb"], e["cu"], o2, lse2, stream=s)
    s.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    g1, g2 = backward(c, o, lse), backward(e, o, lse)
    assert all(torch.equal(g1[n], g2[n]) for n in g1)


def test_head_major_inputs():
    T, Hq, Hkv, d = 200, 4, 2, 128
    c = make(7, [0, 200], T, Hq, Hkv, d)
    e = dict(c, **{n: c[n].transpose(0, 1).contiguous().transpose(0, 1) for n in "qkv"})
    for a, b in zip(forward(c), forward(e)):
        assert torch.equal(a, b)


def test_one_log_beta_for_all_tokens():
    """A broadcast log beta (strides 0) is read as such."""
    T, Hq, Hkv, d = 150, 4, 2, 64
    c = make(8, [0, 150], T, Hq, Hkv, d)
    c["lb"] = torch.full((1, 1), -0.25, device="cuda").expand(T, Hkv)
    o, lse = forward(c)
    check_state(o, lse, reference(c))


def test_extreme_log_betas():
    """beta = 0 (log beta -inf, and the type's lowest value) leaves a token to itself; beta = 1 decays nothing."""
    T, Hq, Hkv, d = 300, 4, 1, 64
    c = make(9, [0, 300], T, Hq, Hkv, d, grads=True)
    c["lb"][::3] = -float("inf")
    c["lb"][1::3] = torch.finfo(torch.float32).min
    c["lb"][2::9] = 0.0
    o, lse = forward(c)
    r = reference(dict(c, lb=c["lb"].clamp(min=-1e30)))
    check_state(o, lse, r)
    check_grads(backward(c, o, lse), r)


def test_large_scores():
    """Scores of +-300: only differences of the logits count."""
    T, Hq, Hkv, d = 260, 2, 1, 128
    c = make(10, [0, 260], T, Hq, Hkv, d)
    c["q"] = (c["q"] * 30).to(torch.bfloat16)
    o, lse = forward(c)
    r = reference(c)
    check(o, r["o"], REL, "o")
    # a score of 300 in fp32 products is off by 2^-22 of it
    np.testing.assert_allclose(f64(lse), r["lse"], rtol=2e-6, atol=1e-4)


@pytest.mark.parametrize("climb", ["scores", "log_beta", "nan"])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 64), (2, 1, 128)])
def test_capped_scores_that_climb_with_the_distance(climb, Hq, Hkv, d):
    """Far keys weigh more than near ones by far more than a tile's reference leaves room for.

    lse: scores of +-60 are off by 2^-22 of 64, a cap of 40 by 2^-21 of it: 1.5e-5 + 1.9e-5."""
    cu, T, cap = [0, 700, 900], 901, 40.0
    c = make(30, cu, T, Hq, Hkv, d)
    if climb == "scores":
        c["q"] = (c["q"] * 0.05 + 1).to(torch.bfloat16)
        sign = torch.where(torch.arange(T) < 300, 1.0, -1.0).cuda()[:, None, None]
        c["k"] = (c["k"] * 0.05 + sign * 60 / d ** 0.5).to(torch.bfloat16)
        c["lb"] = c["lb"] * 1e-3
    else:
        c["lb"][:300] = 0.05                 # up to 35 at 700 tokens
    r = reference(c, None, cap)
    if climb == "nan":
        c["lb"][700:] = float("nan")         # the second document's own
        c["lb"][900:] = -1.0
        o, lse = forward(c, None, cap)
        assert rel(f64(o)[:700], r["o"][:700]) <= REL
        assert torch.isnan(lse[701:900]).all()
    else:
        o, lse = forward(c, None, cap)
        check(o, r["o"], REL, climb)
    np.testing.assert_allclose(f64(lse)[:700], r["lse"][:700], rtol=2e-6, atol=4e-5)


def test_other_documents_and_padding_do_not_leak():
    """NaN and infinities in a neighbour document's rows, and behind the last one, reach nobody else."""
    T, Hq, Hkv, d = 310, 8, 2, 128
    cu = [0, 70, 90, 300]
    c = make(11, cu, T, Hq, Hkv, d, grads=True)
    r = reference(c)
    bad = dict(c, **{n: c[n].clone() for n in ("q", "k", "v", "lb", "d_o")})
    for n in ("q", "k", "v", "lb", "d_o"):
        bad[n][70:90] = float("nan")
        bad[n][300:] = float("inf") if n != "lb" else float("nan")
    o, lse = forward(bad)
    g = backward(bad, o, lse)
    keep = np.r_[0:70, 90:300]
    assert rel(f64(o)[keep], r["o"][keep]) <= REL and np.allclose(f64(lse)[keep], r["lse"][keep], rtol=2e-6, atol=4e-6)
    for n in ("dq", "dk", "dv"):
        assert rel(f64(g[n])[keep], r[n][keep]) <= REL, n
    assert rel(f64(g["d_log_beta"])[keep], r["d_log_beta"][keep]) <= 2e-5
    assert torch.all(o[300:] == 7) and torch.all(g["dq"][300:] == 7) and torch.all(g["d_log_beta"][300:] == 7)


def test_bad_documents_write_nothing():
    for cu in ([0, 50, 40, 60], [-1, 20, 30, 40], [0, 10, 20, 65]):
        c = make(12, cu, 64, 4, 2, 64, grads=True)
        o, lse = forward(c)
        assert kvb.kvb_get_error() == _lib.DERR_RANGE
        g = backward(c, o, lse)
        assert kvb.kvb_get_error() == _lib.DERR_RANGE
        assert all(bool((x == 7).all()) for x in (o, lse, *g.values()))


def test_same_bits_twice_and_in_a_graph():
    T, Hq, Hkv, d = 400, 8, 2, 128
    c = make(13, [0, 150, 400], T, Hq, Hkv, d, grads=True)
    o, lse = forward(c)
    g = backward(c, o, lse)
    o2, lse2 = forward(c)
    g2 = backward(c, o2, lse2)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(g[n], g2[n]) for n in g)
    ws = torch.empty(kvb.kvb_prefill_attn_bwd_workspace_bytes(T, Hq), dtype=torch.uint8, device="cuda")
    out = {n: torch.zeros_like(x) for n, x in g.items()}
    o3, lse3 = torch.zeros_like(o), torch.zeros_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvb.kvb_prefill_attn(c["q"], c["k"], c["v"], c["lb"], c["cu"], o3, lse3)
        kvb.kvb_prefill_attn_bwd(c["q"], c["k"], c["v"], c["lb"], c["cu"], o3, lse3, c["d_o"], None, out["dq"], out["dk"],
                                 out["dv"], out["d_log_beta"], ws)
    # other lengths on replay: the documents are read on the device
    c["cu"].copy_(torch.tensor([0, 33, 399], dtype=torch.int32))
    for _ in range(2):
        graph.replay()
    r = reference(c)
    rows = np.arange(399)
    assert rel(f64(o3)[rows], r["o"][rows]) <= REL
    assert rel(f64(out["d_log_beta"])[rows], r["d_log_beta"][rows]) <= 2e-5
    assert torch.all(o3[399:] == 0)


def test_more_documents_than_a_warp():
    g = np.random.default_rng(14)
    n = g.integers(0, 9, 700)
    cu = np.r_[0, np.cumsum(n)].tolist()
    c = make(14, cu, cu[-1] + 2, 4, 1, 64, grads=True)
    o, lse = forward(c)
    r = reference(c)
    check_state(o, lse, r)
    check_grads(backward(c, o, lse), r)


@pytest.mark.parametrize("softcap,pre", [(0.0, False), (4.0, True)])
def test_many_documents_of_unequal_length(softcap, pre):
    """More key blocks than the device has SMs, so that whole ones are dealt out (few ones are cut)."""
    g = np.random.default_rng(16)
    n = g.integers(0, 400, 60)
    cu = np.r_[1, 1 + np.cumsum(n)].tolist()
    prefix = g.integers(0, 300, 60).tolist() if pre else None
    c = make(16, cu, cu[-1] + 5, 8, 4, 64, grads=True, d_lse=True)
    o, lse = forward(c, prefix, softcap)
    r = reference(c, prefix, softcap)
    check_state(o, lse, r)
    check_grads(backward(c, o, lse, prefix, softcap), r)
    assert kvb.kvb_get_error() == 0


@pytest.mark.parametrize("beta,d,Hq,Hkv,L", [(True, 128, 4, 1, 2500), (False, 64, 2, 2, 2111), (True, 64, 8, 1, 1400)])
def test_long_document(beta, d, Hq, Hkv, L):
    """One document of many tiles: far biases, a moving maximum, key blocks cut into many pieces."""
    c = make(17, [0, L], L, Hq, Hkv, d, beta, grads=True)
    if beta:
        c["lb"][::7] = -1e-4   # tokens that are still seen at the far end
    o, lse = forward(c)
    r = reference(c)
    check_state(o, lse, r)
    check_grads(backward(c, o, lse), r)


def test_growing_weights():
    """log beta > 0 (the far keys weigh most): the running maximum moves in every tile."""
    c = make(18, [0, 700], 700, 4, 2, 128, grads=True)
    c["lb"] = c["lb"].abs() * 0.25
    o, lse = forward(c)
    r = reference(c)
    check(o, r["o"], REL, "o")
    # logits up to some hundreds: an fp32 sum of that size
    np.testing.assert_allclose(f64(lse), r["lse"], rtol=2e-6, atol=1e-4)


@pytest.mark.parametrize("scale", [0.02, 0.6])
def test_given_scale(scale):
    c = make(19, [0, 129, 400], 400, 4, 2, 64, grads=True)
    o, lse = forward(c, scale=scale)
    r = reference(c, scale=scale)
    check(o, r["o"], REL, "o")
    # scores of about 8 * 0.6 / 0.125 partial sums: the tolerance of scores grows with the scale
    np.testing.assert_allclose(f64(lse), r["lse"], rtol=2e-6, atol=4e-6 * max(1.0, scale / 0.125))
    g = backward(c, o, lse, scale=scale)
    for n in ("dq", "dk", "dv"):
        check(g[n], r[n], REL, n)
    check(g["d_log_beta"], r["d_log_beta"], 2e-5 * max(1.0, scale / 0.125), "d_log_beta")


def test_without_lse_and_two_streams_at_once():
    T, Hq, Hkv, d = 900, 8, 2, 128
    a, b = make(20, [0, 400, 900], T, Hq, Hkv, d), make(21, [0, 900], T, Hq, Hkv, d)
    want_a, want_b = forward(a)[0], forward(b)[0]
    oa, ob = torch.zeros_like(want_a), torch.zeros_like(want_b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        kvb.kvb_prefill_attn(a["q"], a["k"], a["v"], a["lb"], a["cu"], oa, stream=s1)
        kvb.kvb_prefill_attn(b["q"], b["k"], b["v"], b["lb"], b["cu"], ob, stream=s2.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(oa, want_a) and torch.equal(ob, want_b)


def test_gradients_on_two_streams_with_a_workspace_each():
    T, Hq, Hkv, d = 600, 8, 2, 64
    cs = [make(22 + k, [0, 250, 600], T, Hq, Hkv, d, grads=True) for k in range(2)]
    states = [forward(c) for c in cs]
    want = [backward(c, *s) for c, s in zip(cs, states)]
    streams = [torch.cuda.Stream() for _ in cs]
    ws = [torch.empty(kvb.kvb_prefill_attn_bwd_workspace_bytes(T, Hq), dtype=torch.uint8, device="cuda") for _ in cs]
    got = [{n: torch.zeros_like(x) for n, x in w.items()} for w in want]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, (o, lse), s, w, g in zip(cs, states, streams, ws, got):
            kvb.kvb_prefill_attn_bwd(c["q"], c["k"], c["v"], c["lb"], c["cu"], o, lse, c["d_o"], None, g["dq"], g["dk"],
                                     g["dv"], g["d_log_beta"], w, stream=s)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w[n], g[n]) for n in w)


def test_single_tokens_have_no_score_gradient():
    """A document of one token: softmax is 1, so dq = dk = d_log_beta = 0 and dv = sum of d_o."""
    T, Hq, Hkv, d = 5, 4, 2, 64
    c = make(24, list(range(T + 1)), T, Hq, Hkv, d, grads=True)
    o, lse = forward(c)
    g = backward(c, o, lse)
    # p = exp(s - lse) is off by 2^-21 relative, so dS by that of dP (at most 40 here), times 40 of k or q
    for n in ("dq", "dk"):
        assert float(g[n].abs().max()) <= 40 * 40 * 2.0 ** -21, n
    assert torch.all(g["d_log_beta"] == 0)
    check(g["dv"], reference(c)["dv"], REL, "dv")


def test_empty_calls():
    c = make(15, [0, 0, 0], 5, 2, 1, 64, grads=True)
    o, lse = forward(c)
    g = backward(c, o, lse)
    assert all(bool((x == 7).all()) for x in (o, lse, *g.values()))
    z = make(15, [0], 0, 2, 1, 64, grads=True)
    o, lse = forward(z)
    assert o.numel() == 0
    assert kvb.kvb_get_error() == 0


# ------------------------------------------------------------------ pages

def filled_pool(seed, B, H, width, num_pages, held, d=64, beta=True):
    """A pool whose sequences hold `held` slots, pages in a shuffled order."""
    g = np.random.default_rng(seed)
    pool = kvb.PagedPool(B, H, d, width, num_pages, beta)
    order = g.permutation(num_pages).astype(np.int32)
    table = np.full((B, H, width), -1, np.int32)
    at = 0
    for b in range(B):
        for h in range(H):
            n = -(-held[b] // PAGE)
            table[b, h, :n] = order[at:at + n]
            at += n
    free = order[at:]
    pool.table.copy_(torch.from_numpy(table))
    pool.len.copy_(torch.tensor([[x] * H for x in held], dtype=torch.int32))
    pool.free_pages[:len(free)] = torch.from_numpy(free).cuda()
    pool.free_count.fill_(len(free))
    return pool


BITS = {"range": _lib.DERR_RANGE, "len": _lib.DERR_LEN, "pages": _lib.DERR_PAGES}


@pytest.mark.parametrize("B,H,held,new,pages,empty_only", [
    (1, 1, [0], [1], 1, False),
    (3, 2, [0, 63, 64], [65, 1, 1], 20, False),
    (4, 2, [10, 0, 0, 5], [0, 200, 0, 300], 40, False),      # sequences without new tokens
    (4, 2, [10, 0, 0, 5], [100, 200, 0, 50], 11, False),     # the free stack runs short
    (4, 1, [0, 30, 0, 0], [10, 10, 0, 70], 20, True),        # a sequence that holds slots already
    (2, 1, [500, 0], [200, 3], 40, False),                   # past the table's width
    (70, 3, [7] * 70, [11] * 70, 500, False),
    (1500, 1, [0] * 1500, [3] * 1500, 1400, False),          # more sequences than a block has threads
])
def test_plan(B, H, held, new, pages, empty_only):
    width = 8
    pool = filled_pool(20, B, H, width, pages, held)
    cu = np.r_[2, 2 + np.cumsum(new)].astype(np.int32)
    T = int(cu[-1]) + 3
    slot_map = torch.full((H, T), -7, dtype=torch.int32, device="cuda")
    want = ref.plan(cu, host(pool.len), host(pool.table), host(pool.free_pages), int(pool.free_count), host(slot_map),
                    pages, PAGE, empty_only)
    ws = torch.empty(kvb.kvb_paged_plan_workspace_bytes(B, H), dtype=torch.uint8, device="cuda")
    kvb.kvb_paged_plan(pool, torch.from_numpy(cu).cuda(), slot_map, ws, empty_only=empty_only)
    bits = kvb.kvb_get_error()
    for got, w in ((slot_map, want[0]), (pool.table, want[1]), (pool.len, want[2])):
        np.testing.assert_array_equal(host(got), w)
    assert int(pool.free_count) == want[3]
    assert bits == sum(BITS[e] for e in want[4])


def test_plan_of_unequal_heads():
    """Heads of one sequence that hold different numbers of slots."""
    pool = filled_pool(21, 2, 2, 6, 30, [0, 0])
    pool.len.copy_(torch.tensor([[70, 3], [0, 64]], dtype=torch.int32))
    table = torch.full((2, 2, 6), -1, dtype=torch.int32)
    table[0, 0, :2], table[0, 1, 0], table[1, 1, 0] = torch.tensor([4, 9], dtype=torch.int32), 2, 17
    pool.table.copy_(table)
    free = np.setdiff1d(np.arange(30), [4, 9, 2, 17]).astype(np.int32)
    pool.free_pages[:26] = torch.from_numpy(free).cuda()
    pool.free_count.fill_(26)
    cu = np.array([0, 130, 195], np.int32)
    slot_map = torch.full((2, 195), -7, dtype=torch.int32, device="cuda")
    want = ref.plan(cu, host(pool.len), host(pool.table), host(pool.free_pages), 26, host(slot_map), 30, PAGE)
    ws = torch.empty(kvb.kvb_paged_plan_workspace_bytes(2, 2), dtype=torch.uint8, device="cuda")
    kvb.kvb_paged_plan(pool, torch.from_numpy(cu).cuda(), slot_map, ws)
    for got, w in ((slot_map, want[0]), (pool.table, want[1]), (pool.len, want[2])):
        np.testing.assert_array_equal(host(got), w)
    assert int(pool.free_count) == want[3] and kvb.kvb_get_error() == 0


def test_plan_with_bad_starts_leaves_the_cache():
    pool = filled_pool(22, 2, 2, 4, 20, [5, 6])
    before = [host(x).copy() for x in (pool.table, pool.len, pool.free_count, pool.free_pages)]
    slot_map = torch.full((2, 40), 3, dtype=torch.int32, device="cuda")
    ws = torch.empty(kvb.kvb_paged_plan_workspace_bytes(2, 2), dtype=torch.uint8, device="cuda")
    kvb.kvb_paged_plan(pool, torch.tensor([0, 30, 20], dtype=torch.int32).cuda(), slot_map, ws)
    assert kvb.kvb_get_error() == _lib.DERR_RANGE
    assert torch.all(slot_map == -1)
    for x, w in zip((pool.table, pool.len, pool.free_count, pool.free_pages), before):
        np.testing.assert_array_equal(host(x), w)


@pytest.mark.parametrize("T,H,d,beta", [(1, 1, 64, True), (61, 2, 64, True), (257, 3, 128, False), (1000, 4, 128, True),
                                        (33, 2, 72, True)])
def test_write(T, H, d, beta):
    g = torch.Generator().manual_seed(30)
    pages = T // 8 + 3
    pool = kvb.PagedPool(1, H, d, 4, pages, beta)
    kv = torch.randn(T, 2 * H, d, generator=g).to(torch.bfloat16).cuda()
    k, v = kv[:, :H], kv[:, H:]
    lb = torch.randn(T, H, generator=g).cuda() if beta else None
    pos = torch.randint(0, 1 << 30, (T,), generator=g).to(torch.int32).cuda()
    rows = torch.randperm(pages * PAGE, generator=g)[:T * H].to(torch.int32).reshape(H, T).cuda()
    rows[:, T // 3] = -1
    if T > 50:
        rows[0, 7], rows[H - 1, 9] = -7, pages * PAGE   # skipped; past the pool
    want = [host(x).copy() for x in (pool.k_pages, pool.v_pages, pool.pos_pages)]
    wlb = None if lb is None else host(pool.log_beta_pages).copy()
    r = host(rows)
    for h in range(H):
        ok = np.flatnonzero((r[h] >= 0) & (r[h] < pages * PAGE))
        want[0].reshape(-1, d)[r[h][ok]] = host(k.contiguous())[ok, h]
        want[1].reshape(-1, d)[r[h][ok]] = host(v.contiguous())[ok, h]
        want[2].reshape(-1)[r[h][ok]] = host(pos)[ok]
        if wlb is not None:
            wlb.reshape(-1)[r[h][ok]] = host(lb)[ok, h]
    kvb.kvb_paged_write(pool, k, v, lb, pos, rows)
    assert kvb.kvb_get_error() == (_lib.DERR_RANGE if T > 50 else 0)
    for x, w in zip((pool.k_pages, pool.v_pages, pool.pos_pages), want):
        np.testing.assert_array_equal(host(x), w)
    if wlb is not None:
        np.testing.assert_array_equal(host(pool.log_beta_pages), wlb)


@pytest.mark.parametrize("beta", [True, False])
def test_prompts_then_decode(beta):
    """Prompts enter a paged cache, then decode steps run on it: the same as prompts one token longer,
    and later joiners leave the others alone."""
    B, Hq, Hkv, d = 3, 8, 2, 64
    cache = PagedKVCache(B, Hq, Hkv, d, max_pages=6, num_pages=30, M=300, with_beta=beta)
    lens = [130, 0, 65]
    cu = [0, 130, 130, 195]
    full = make(40, [0, 131, 131, 197], 197, Hq, Hkv, d, beta)     # each prompt with one token more
    rows = torch.cat([torch.arange(0, 130), torch.arange(131, 196)]).cuda()
    c = {n: full[n][rows].contiguous() for n in "qkv"}
    lb = full["lb"][rows].contiguous() if beta else None
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
    o = torch.zeros(195, Hq, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(195, Hq, device="cuda")
    cache.prefill(c["q"], c["k"], c["v"], lb, torch.tensor(cu, dtype=torch.int32).cuda(), pos, o, lse)
    assert kvb.kvb_get_error() == 0
    want_o, want_lse = forward(full)
    assert torch.equal(o, want_o[rows]) or rel(f64(o), f64(want_o)[rows.cpu()]) <= REL
    assert cache.len.tolist() == [[130] * 2, [0] * 2, [65] * 2]
    assert cache.pages_in_use() == 2 * (3 + 2)
    # the next token of each prompt as a decode step; sequence 1 is inactive
    last = torch.tensor([130, 0, 196]).cuda()
    t = torch.tensor([130, -1, 65], dtype=torch.int32).cuda()
    od, ld = torch.zeros(B, Hq, d, device="cuda"), torch.zeros(B, Hq, device="cuda")
    cache.step(full["q"][last].contiguous(), full["k"][last].contiguous(), full["v"][last].contiguous(),
               full["lb"][last].contiguous() if beta else None, t, od, ld)
    assert kvb.kvb_get_error() == 0
    r = reference(full)
    for b, row in ((0, 130), (2, 196)):
        assert rel(f64(od)[b], r["o"][row]) <= REL
        np.testing.assert_allclose(f64(ld)[b], r["lse"][row], rtol=2e-6, atol=1e-4)
    # sequence 1 joins; the others have no new tokens and keep theirs
    before = host(cache.pool.k_pages).copy()
    j = make(41, [0, 0, 70, 70], 70, Hq, Hkv, d, beta)
    oj = torch.zeros(70, Hq, d, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cache.prefill(j["q"], j["k"], j["v"], j["lb"], j["cu"], torch.arange(70, dtype=torch.int32).cuda(), oj, stream=s)
    s.synchronize()
    assert kvb.kvb_get_error() == 0
    assert cache.len.tolist() == [[131] * 2, [70] * 2, [66] * 2]
    assert rel(f64(oj), reference(j)["o"]) <= REL
    used = host(cache.pool.table)[[0, 2]]
    used = used[used >= 0]
    np.testing.assert_array_equal(host(cache.pool.k_pages)[used], before[used])
    # a sequence that holds tokens does not take another prompt
    cache.prefill(j["q"], j["k"], j["v"], j["lb"], j["cu"], torch.arange(70, dtype=torch.int32).cuda(), oj)
    assert kvb.kvb_get_error() == _lib.DERR_LEN
    assert cache.len.tolist() == [[131] * 2, [70] * 2, [66] * 2]


def test_reset_and_prefill_captured_and_replayed():
    """A graph of reset and prefill: every replay serves the lengths that stand in cu then."""
    B, Hq, Hkv, d, T = 2, 4, 2, 64, 300
    cache = PagedKVCache(B, Hq, Hkv, d, max_pages=6, num_pages=16, M=300)
    c = make(50, [0, 100, 300], T, Hq, Hkv, d)
    pos = torch.cat([torch.arange(100), torch.arange(200)]).to(torch.int32).cuda()
    o, lse = torch.zeros(T, Hq, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, Hq, device="cuda")

    def work():
        cache.reset()
        cache.prefill(c["q"], c["k"], c["v"], c["lb"], c["cu"], pos, o, lse)
    work()
    want = o.clone(), cache.len.clone(), host(cache.pool.k_pages)[host(cache.pool.table)[1, 0, :4]].copy()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for _ in range(2):
        o.zero_()
        graph.replay()
        assert torch.equal(o, want[0]) and torch.equal(cache.len, want[1])
        np.testing.assert_array_equal(host(cache.pool.k_pages)[host(cache.pool.table)[1, 0, :4]], want[2])
    c["cu"].copy_(torch.tensor([0, 100, 260], dtype=torch.int32))
    graph.replay()
    assert cache.len.tolist() == [[100] * 2, [160] * 2] and cache.pages_in_use() == 2 * (2 + 3)
    assert kvb.kvb_get_error() == 0
