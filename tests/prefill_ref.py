"""The prompt-path operators in float64 on the host (numpy), written from their definitions."""
import numpy as np


def attention(q, k, v, log_beta, cu, prefix=None, softcap=0.0, scale=0.0, d_o=None, d_lse=None):
    """o, lse (and with d_o the gradients dq, dk, dv, d_log_beta) of packed documents, float64; rows of
    no document are NaN. q [T, Hq, d], k, v [T, Hkv, d], log_beta [T, Hkv] or None."""
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    scale = scale or d ** -0.5
    full = lambda *s: np.full(s, np.nan)   # noqa: E731
    r = dict(o=full(T, Hq, d), lse=full(T, Hq), dq=full(T, Hq, d), dk=full(T, Hkv, d), dv=full(T, Hkv, d),
             d_log_beta=full(T, Hkv))
    for n in range(len(cu) - 1):
        s, e = int(cu[n]), int(cu[n + 1])
        L = e - s
        if L == 0:
            continue
        pre = 0 if prefix is None else min(max(int(prefix[n]), 0), L)
        i, j = np.arange(L)[:, None], np.arange(L)[None, :]
        sees = j < np.maximum(i + 1, pre)
        age = np.maximum(i - j, 0).astype(np.float64)
        for g in range(Hkv):
            kk, vv = k[s:e, g].astype(np.float64), v[s:e, g].astype(np.float64)
            dk, dv, db = np.zeros((L, d)), np.zeros((L, d)), np.zeros(L)
            for h in range(g * G, (g + 1) * G):
                qq = q[s:e, h].astype(np.float64)
                x = scale * (qq @ kk.T)
                slope = 1.0
                if softcap:
                    t = np.tanh(x / softcap)
                    x, slope = softcap * t, 1 - t * t
                if log_beta is not None:
                    b = np.broadcast_to(log_beta[s:e, g].astype(np.float64)[None, :], (L, L))
                    x = x + np.where(age > 0, age * np.where(age > 0, b, 0.0), 0.0)
                x = np.where(sees, x, -np.inf)
                m = x.max(1, keepdims=True)
                w = np.exp(x - m)
                z = w.sum(1, keepdims=True)
                p = w / z
                o = p @ vv
                r["o"][s:e, h], r["lse"][s:e, h] = o, (m + np.log(z))[:, 0]
                if d_o is None:
                    continue
                go = d_o[s:e, h].astype(np.float64)
                dx = go @ vv.T - (go * o).sum(1, keepdims=True)
                if d_lse is not None:
                    dx = dx + d_lse[s:e, h].astype(np.float64)[:, None]
                dx = p * dx
                dv += p.T @ go
                db += (dx * age).sum(0)
                ds = dx * slope
                r["dq"][s:e, h] = scale * (ds @ kk)
                dk += scale * (ds.T @ qq)
            if d_o is not None:
                r["dk"][s:e, g], r["dv"][s:e, g], r["d_log_beta"][s:e, g] = dk, dv, db
    return r


def plan(cu, len_, table, free_pages, free_count, slot_map, num_pages, page, empty_only=False):
    """(slot_map, table, len, free_count, error kinds) after a plan, by a loop over the sequences."""
    B, H, width = table.shape
    T = slot_map.shape[1]
    slot_map, table, len_ = slot_map.copy(), table.copy(), len_.copy()
    if cu[0] < 0 or np.any(np.diff(cu) < 0) or cu[-1] > T:
        return np.full_like(slot_map, -1), table, len_, free_count, {"range"}
    errors, want, top = set(), 0, free_count
    for b in range(B):
        new = int(cu[b + 1] - cu[b])
        held = [int(x) for x in len_[b]]
        if any(n < 0 or n + new > width * page or (empty_only and n > 0 and new > 0) for n in held):
            errors.add("len")
            slot_map[:, cu[b]:cu[b + 1]] = -1
            continue
        need = sum(-(-(n + new) // page) - -(-n // page) for n in held)
        want += need
        if need and want > free_count:
            errors.add("pages")
            slot_map[:, cu[b]:cu[b + 1]] = -1
            continue
        for g in range(H):
            n = held[g]
            for jp in range(-(-n // page), -(-(n + new) // page)):
                top -= 1
                table[b, g, jp] = free_pages[top]
            for x in range(new):
                slot_map[g, cu[b] + x] = table[b, g, (n + x) // page] * page + (n + x) % page
            len_[b, g] = n + new
    return slot_map, table, len_, top, errors
