"""Bounds, value by value, on what the prompt-path kernels may be off by, in float64 on the host (numpy).

A rounding to bf16 is off by at most 2^-8 of the value. ETA is what a softmax weight may be off by,
relative to itself, before that rounding: 4e-6 from its logit (an fp32 sum of d products whose partial
sums stay below 16), as much from the row's lse or sum, 2.6e-6 from the exponential: below 2^-16."""
import numpy as np

BF16, ETA = 2.0 ** -8, 2.0 ** -16
SLACK = 1.01   # products of two of the errors


def pairs(q, k, log_beta, g, h, s, e, pre, softcap, scale):
    """(p, slope, age) of a document's rows s .. e, query head h of kv head g."""
    i, j = np.arange(e - s)[:, None], np.arange(e - s)[None, :]
    x = scale * (q[s:e, h].astype(np.float64) @ k[s:e, g].astype(np.float64).T)
    slope = np.ones_like(x)
    if softcap:
        t = np.tanh(x / softcap)
        x, slope = softcap * t, 1 - t * t
    age = np.maximum(i - j, 0).astype(np.float64)
    if log_beta is not None:
        x = x + age * log_beta[s:e, g].astype(np.float64)[None, :]
    x = np.where(j < np.maximum(i + 1, pre), x, -np.inf)
    p = np.exp(x - x.max(1, keepdims=True))
    return p / p.sum(1, keepdims=True), slope, age


def documents(cu, prefix):
    for n in range(len(cu) - 1):
        s, e = int(cu[n]), int(cu[n + 1])
        if e > s:
            yield s, e, 0 if prefix is None else min(max(int(prefix[n]), 0), e - s)


def forward(q, k, v, log_beta, cu, prefix=None, softcap=0.0, scale=0.0):
    """o and the bound on its error, [T, Hq, d]; rows of no document are NaN. The weights enter P V as bf16
    (BF16 of p |v| for each key), their sum does not, and o is rounded once."""
    T, Hq, d = q.shape
    G = Hq // k.shape[1]
    o, bound = np.full((T, Hq, d), np.nan), np.full((T, Hq, d), np.nan)
    for s, e, pre in documents(cu, prefix):
        for h in range(Hq):
            g = h // G
            p, _, _ = pairs(q, k, log_beta, g, h, s, e, pre, softcap, scale or d ** -0.5)
            vv = v[s:e, g].astype(np.float64)
            o[s:e, h] = p @ vv
            bound[s:e, h] = SLACK * (BF16 * np.abs(o[s:e, h]) + (BF16 + 2 * ETA) * (p @ np.abs(vv)))
    return o, bound


def gradients(q, k, v, log_beta, cu, d_o, d_lse=None, prefix=None, softcap=0.0, scale=0.0):
    """{name: (gradient, bound on its error)}; rows of no document are NaN. For each pair, with B = sum_c |d_o_c v_c|
    and D its row's mean of B plus |d_lse|: dS = p (d_o.v - delta) is off by 2 ETA p (B + D) (p, the fp32 sums of
    d_o.v and delta), P and dS enter the products as bf16, and dq, dk and dv are rounded once. dq of a row whose
    tile of 128 / G tokens sees more than 128 keys takes delta from o as it was stored, but for a key of weight
    above 1/2 (to fp32). That delta's error (of o, `forward`'s bound, times |d_o|) meets p |k| of the other keys."""
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    scale = scale or d ** -0.5
    _, o_bound = forward(q, k, v, log_beta, cu, prefix, softcap, scale)
    shapes = dict(dq=(T, Hq, d), dk=(T, Hkv, d), dv=(T, Hkv, d), d_log_beta=(T, Hkv))
    val, bnd = ({n: np.full(s, np.nan) for n, s in shapes.items()} for _ in range(2))
    for s, e, pre in documents(cu, prefix):
        first = np.arange(e - s) * G // 128 * 128 // G          # of each row's tile
        far = np.maximum(np.minimum(first + 128 // G, e - s), pre) > 128
        for x in (val, bnd):
            for n in ("dk", "dv", "d_log_beta"):
                x[n][s:e] = 0.0
        for h in range(Hq):
            g = h // G
            p, slope, age = pairs(q, k, log_beta, g, h, s, e, pre, softcap, scale)
            qq, kk, vv, do = (x.astype(np.float64) for x in (q[s:e, h], k[s:e, g], v[s:e, g], d_o[s:e, h]))
            dl = np.zeros(e - s) if d_lse is None else d_lse[s:e, h].astype(np.float64)
            dp = do @ vv.T
            ds = p * (dp - ((p * dp).sum(1) - dl)[:, None])
            b = np.abs(do) @ np.abs(vv).T
            eds = 2 * ETA * p * (b + ((p * b).sum(1) + np.abs(dl))[:, None])
            eps = (np.abs(do) * o_bound[s:e, h]).sum(1)[:, None]
            at = p.argmax(1)[:, None]
            top = np.where(np.take_along_axis(p, at, 1) > 0.5 + 8 * ETA, np.take_along_axis(p * slope, at, 1), 0.0)
            top = top * np.abs(kk)[at[:, 0]]
            estimate = np.where(far[:, None], eps * ((p * slope) @ np.abs(kk) - top)
                                + 4 * ETA * ((p * b).sum(1) + np.abs(dl))[:, None] * top, 0.0)
            val["dq"][s:e, h] = scale * (ds * slope) @ kk
            e16 = (eds + BF16 * np.abs(ds)) * slope             # dS as it enters the products
            bnd["dq"][s:e, h] = scale * (e16 @ np.abs(kk) + estimate)
            val["dk"][s:e, g] += scale * (ds * slope).T @ qq
            bnd["dk"][s:e, g] += scale * e16.T @ np.abs(qq)
            val["dv"][s:e, g] += p.T @ do
            bnd["dv"][s:e, g] += (BF16 + 2 * ETA) * p.T @ np.abs(do)
            val["d_log_beta"][s:e, g] += (ds * age).sum(0)
            bnd["d_log_beta"][s:e, g] += (eds * age).sum(0)
    return {n: (val[n], SLACK * (bnd[n] + (0.0 if n == "d_log_beta" else BF16 * np.abs(val[n])))) for n in shapes}


def within(got, want, bound, what):
    """Every value of the documents' rows within its bound."""
    rows = ~np.isnan(want.reshape(want.shape[0], -1)[:, 0])
    off = np.abs(got[rows] - want[rows]) - bound[rows]
    bad = ~(off <= 0)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} values out of bounds, the first at "
                           f"{tuple(int(x[0]) for x in np.nonzero(bad))} of the documents' rows, by {off[bad].max():.3e}")
