"""Measured cases of the prompt's path into a memory-bounded cache.

Four operators, each with its plain form (elementary torch operations) and the library's call:

  prefill  retention-gated causal attention over packed prompts: for query token i and key token j of
           one document, logit = cap(scale q.k) + max(i - j, 0) log beta_j over the keys j with
           j < max(i + 1, prefix), cap(x) = softcap tanh(x / softcap); gives (o, lse)
  train    the same attention and its gradients with respect to q, k, v and log beta
  plan     pages and a slot map for the new tokens of every sequence of a paged cache
  write    the packed K/V rows, log beta and positions into the pages a slot map names

Every case is a dict of plain values. `lengths` (from the case alone) gives the documents.
"""
import math
import random

import torch

own = False

PAGE = 64          # slots of a page
COST_MOST = 8192 * 8192 * 32   # padded scores (documents x longest^2 x query heads) of the largest attention cases


def listed():
    return [
        # one short question of a chat turn: the latency of a call
        dict(name="prefill_tiny", op="prefill", tokens=17, docs=1, salt=1, pad=0, Hq=8, Hkv=2, d=64, beta=True,
             softcap=0.0, prefix=0.0),
        # a serving batch of prompts of very different lengths, empty ones among them, in a padded buffer
        dict(name="prefill_ragged", op="prefill", tokens=6151, docs=24, salt=2, pad=37, Hq=32, Hkv=8, d=128, beta=True,
             softcap=0.0, prefix=0.0),
        # capped scores and an instruction prefix whose tokens see each other, 64-dim heads in groups of 8
        dict(name="prefill_cap_prefix", op="prefill", tokens=4000, docs=5, salt=3, pad=0, Hq=16, Hkv=2, d=64, beta=True,
             softcap=30.0, prefix=0.3),
        # plain causal attention (beta = 1), one query head per kv head
        dict(name="prefill_plain", op="prefill", tokens=4096, docs=2, salt=4, pad=0, Hq=16, Hkv=16, d=128, beta=False,
             softcap=0.0, prefix=0.0),
        # one long prompt through a layer of 32 query and 8 kv heads
        dict(name="prefill_layer", op="prefill", tokens=8192, docs=1, salt=5, pad=0, Hq=32, Hkv=8, d=128, beta=True,
             softcap=0.0, prefix=0.0),
        # a few short samples of a gate's training step
        dict(name="train_small", op="train", tokens=301, docs=3, salt=6, pad=0, Hq=8, Hkv=2, d=64, beta=True,
             softcap=0.0, prefix=0.0),
        # packed samples with capped scores and a prefix; the state's lse has a gradient as well
        dict(name="train_ragged", op="train", tokens=5003, docs=11, salt=7, pad=21, Hq=16, Hkv=4, d=128, beta=True,
             softcap=50.0, prefix=0.2),
        # the training step of a layer over one long sample
        dict(name="train_layer", op="train", tokens=8192, docs=1, salt=8, pad=0, Hq=32, Hkv=8, d=128, beta=True,
             softcap=0.0, prefix=0.0),
        # a decode batch with a few short prompts joining it
        dict(name="plan_small", op="plan", tokens=200, docs=6, salt=9, pad=0, Hkv=2, held=300),
        # a large batch of prompts admitted at once, behind what its sequences hold already
        dict(name="plan_large", op="plan", tokens=131072, docs=256, salt=10, pad=500, Hkv=8, held=1000),
        # a short prompt's rows
        dict(name="write_small", op="write", tokens=61, docs=2, salt=11, pad=0, Hkv=2, d=64, beta=True),
        # a long batch's rows
        dict(name="write_large", op="write", tokens=32768, docs=40, salt=12, pad=0, Hkv=8, d=128, beta=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "train", "train", "plan", "write"])
    salt = rng.randrange(1 << 20)
    if op == "plan":
        return dict(op=op, tokens=_log_int(rng, 1, 131072), docs=_log_int(rng, 1, 256), salt=salt, pad=rng.choice([0, 3, 100]),
                    Hkv=rng.choice([1, 2, 4, 8]), held=rng.choice([0, 1, 64, 700]))
    if op == "write":
        return dict(op=op, tokens=_log_int(rng, 1, 32768), docs=_log_int(rng, 1, 64), salt=salt, pad=rng.choice([0, 5]),
                    Hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]), beta=rng.random() < 0.7)
    while True:
        c = dict(op=op, tokens=_log_int(rng, 1, 12000), docs=_log_int(rng, 1, 32), salt=salt, pad=rng.choice([0, 11]),
                 Hq=0, Hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]), beta=rng.random() < 0.7,
                 softcap=rng.choice([0.0, 0.0, 20.0, 50.0]), prefix=rng.choice([0.0, 0.0, 0.4]))
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 4, 8])
        if c["docs"] * max(lengths(c)) ** 2 * c["Hq"] <= COST_MOST // 2:
            return c


def lengths(case):
    """The documents' lengths: they sum to `tokens`; with several documents they differ widely and some may be 0."""
    n, total = case["docs"], case["tokens"]
    if n == 1:
        return [total]
    r = random.Random(case["salt"])
    w = [0.0 if r.random() < 0.08 else r.expovariate(1.0) + 0.05 for _ in range(n)]
    s = sum(w)
    if s == 0.0:
        w, s = [1.0] * n, float(n)
    out = [int(total * x / s) for x in w]
    out[max(range(n), key=lambda i: out[i])] += total - sum(out)
    return out


def _prefixes(case):
    r = random.Random(case["salt"] + 1)
    return [int(case["prefix"] * n * r.random() * 2) for n in lengths(case)]


def _starts(case):
    cu = [0]
    for n in lengths(case):
        cu.append(cu[-1] + n)
    return cu


def _pairs(case):
    """Visible (query, key) pairs of one head."""
    total = 0
    for n, p in zip(lengths(case), _prefixes(case)):
        p = min(p, n)
        total += n * (n + 1) // 2 + p * (p - 1) // 2
    return total


def work(case):
    T = case["tokens"]
    if case["op"] == "plan":
        B, H = case["docs"], case["Hkv"]
        pages = sum(-(-(h + n) // PAGE) - -(-h // PAGE) for h, n in zip(_held(case), lengths(case))) * H
        # new slot map and table entries; the pages taken; lengths and starts read, lengths written
        return {"bytes": 4.0 * (T * H + 2 * pages + 2 * B * H + B + 2), "flops": 0.0}
    if case["op"] == "write":
        rows = T * case["Hkv"]
        return {"bytes": 2.0 * rows * (2 * 2 * case["d"] + 4 + (4 if case["beta"] else 0)), "flops": 0.0}
    q, kv = T * case["Hq"] * case["d"] * 2, T * case["Hkv"] * case["d"] * 2
    gate = T * case["Hkv"] * 4 if case["beta"] else 0
    fwd = 2 * q + 2 * kv + gate + T * case["Hq"] * 4
    if case["op"] == "prefill":
        return {"bytes": float(fwd), "flops": 4.0 * case["d"] * case["Hq"] * _pairs(case)}
    # o, lse, dq, dk, dv, dlog_beta written; q, k, v, log_beta and the two gradients of the state read
    return {"bytes": float(fwd + 2 * q + 2 * kv + gate + T * case["Hq"] * 4),
            "flops": 14.0 * case["d"] * case["Hq"] * _pairs(case)}


def _held(case):
    """Slots that each sequence of a plan case holds before the call."""
    r = random.Random(case["salt"] + 2)
    return [r.randrange(case["held"] + 1) if case["held"] else 0 for _ in range(case["docs"])]


def _gate(shape, g):
    """log of a retention score: beta = sigmoid(x), x ~ N(2, 1.5)."""
    x = torch.randn(shape, generator=g, device="cuda") * 1.5 + 2.0
    return torch.nn.functional.logsigmoid(x)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cu_h = _starts(case)
    rows = case["tokens"] + case["pad"]
    s = dict(case=case, cu=torch.tensor(cu_h, dtype=torch.int32, device="cuda"), longest=max(lengths(case)))
    bf = dict(dtype=torch.bfloat16, device="cuda")
    if case["op"] in ("prefill", "train"):
        Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
        s["q"] = torch.randn(rows, Hq, d, generator=g, **bf)
        s["k"] = torch.randn(rows, Hkv, d, generator=g, **bf)
        s["v"] = torch.randn(rows, Hkv, d, generator=g, **bf)
        s["gate"] = _gate((rows, Hkv), g) if case["beta"] else None
        s["prefix"] = torch.tensor(_prefixes(case), dtype=torch.int32, device="cuda") if case["prefix"] else None
        s["o"], s["lse"] = torch.zeros(rows, Hq, d, **bf), torch.zeros(rows, Hq, device="cuda")
        if case["op"] == "train":
            s["d_o"] = torch.randn(rows, Hq, d, generator=g, **bf)
            s["d_lse"] = torch.randn(rows, Hq, generator=g, device="cuda") if case["softcap"] else None
            s["dq"], s["dk"], s["dv"] = (torch.zeros_like(s[x]) for x in "qkv")
            s["d_gate"] = torch.zeros(rows, Hkv, device="cuda") if case["beta"] else None
        return s
    H, held = case["Hkv"], _held(case) if case["op"] == "plan" else [0] * case["docs"]
    B = case["docs"]
    old = [-(-h // PAGE) for h in held]
    new = [-(-(h + n) // PAGE) for h, n in zip(held, lengths(case))]
    # a plan's pool is a little short, so that the last sequences of a crowded batch wait
    pool = sum(new) * H if case["op"] == "write" else sum(old) * H + max(1, (sum(new) - sum(old)) * H * 15 // 16 + 1)
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    taken = (sum(old) if case["op"] == "plan" else sum(new)) * H
    width = max(1, max(new)) + 1
    table = torch.full((B, H, width), -1, dtype=torch.int32)
    order_h, at = order.cpu(), 0
    for b, n in enumerate(old if case["op"] == "plan" else new):
        for h in range(H):
            table[b, h, :n] = order_h[at:at + n]
            at += n
    s.update(table=table.cuda(), free_pages=torch.cat([order[taken:], order[:taken]]).contiguous(),
             free_count=torch.tensor([pool - taken], dtype=torch.int32, device="cuda"), pages=pool,
             len=torch.tensor([[h] * H for h in held], dtype=torch.int32, device="cuda"))
    s["slot_map"] = torch.full((H, rows), -7, dtype=torch.int32, device="cuda")
    if case["op"] == "plan":
        s["len0"], s["free0"] = s["len"].clone(), s["free_count"].clone()
        return s
    d = case["d"]
    s["k"] = torch.randn(rows, H, d, generator=g, **bf)
    s["v"] = torch.randn(rows, H, d, generator=g, **bf)
    s["gate"] = _gate((rows, H), g) if case["beta"] else None
    s["pos"] = torch.cat([torch.arange(n, dtype=torch.int32) for n in lengths(case)] + [torch.zeros(case["pad"], dtype=torch.int32)]).cuda()
    s["slot_map"][:] = -1
    for b, n in enumerate(lengths(case)):
        r = torch.arange(n, device="cuda")
        s["slot_map"][:, cu_h[b]:cu_h[b + 1]] = s["table"][b][:, r // PAGE] * PAGE + (r % PAGE).to(torch.int32)
    s["k_pages"], s["v_pages"] = torch.zeros(pool, PAGE, d, **bf), torch.zeros(pool, PAGE, d, **bf)
    s["gate_pages"] = torch.zeros(pool, PAGE, device="cuda") if case["beta"] else None
    s["pos_pages"] = torch.zeros(pool, PAGE, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms

def _padded(s):
    """Token index [N, L] of every document's rows (clipped) and which of them exist."""
    cu = s["cu"].long()
    r = torch.arange(s["longest"], device="cuda")
    n = (cu[1:] - cu[:-1])[:, None]
    return (cu[:-1, None] + r).clamp(max=s["q"].shape[0] - 1), r < n, n


def _plain_attention(s):
    c = s["case"]
    G, Hkv, d, L = c["Hq"] // c["Hkv"], c["Hkv"], c["d"], s["longest"]
    at, real, n = _padded(s)
    N = at.shape[0]
    q = s["q"][at].float().reshape(N, L, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(N, Hkv, G * L, d)
    k, v = (s[x][at].float().permute(0, 2, 1, 3) for x in "kv")
    x = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).reshape(N, Hkv, G, L, L)
    bent = None
    if c["softcap"]:
        bent = torch.tanh(x.div_(c["softcap"]))
        x = bent * c["softcap"]
    i, j = torch.arange(L, device="cuda")[:, None], torch.arange(L, device="cuda")[None, :]
    dist = (i - j).clamp(min=0).float()
    if c["beta"]:
        x += dist * s["gate"][at].permute(0, 2, 1)[:, :, None, None, :]
    sees = (j <= i)[None] & (j < n[:, :, None])
    if s["prefix"] is not None:
        sees = ((j <= i)[None] | (j[None] < s["prefix"][:, None, None])) & (j < n[:, :, None])
    x.masked_fill_(~sees[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    p /= total
    lse = (m + total.log()).squeeze(-1)
    o = (p.reshape(N, Hkv, G * L, L) @ v).reshape(N, Hkv, G, L, d)
    return dict(at=at, real=real, q=q, k=k, v=v, p=p, bent=bent, dist=dist, o=o, lse=lse)


def _unpad(x, a, like):
    """[N, heads, L, ...] of padded documents -> the packed rows of `like` (rows outside stay 0)."""
    out = torch.zeros_like(like)
    out[a["at"][a["real"]]] = x.transpose(1, 2)[a["real"]].to(like.dtype)
    return out


def _plain_prefill(s):
    a = _plain_attention(s)
    N, Hkv, G, L, d = a["o"].shape
    return {"o": _unpad(a["o"].reshape(N, Hkv * G, L, d), a, s["o"]), "lse": _unpad(a["lse"].reshape(N, Hkv * G, L), a, s["lse"])}


def _plain_train(s):
    a = _plain_attention(s)
    c = s["case"]
    N, Hkv, G, L, d = a["o"].shape
    heads = (N, Hkv, G * L, d)
    d_o = (s["d_o"][a["at"]].float() * a["real"][:, :, None, None]).reshape(N, L, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(heads)
    delta = (d_o * a["o"].reshape(heads)).sum(-1)
    if s["d_lse"] is not None:
        delta = delta - (s["d_lse"][a["at"]] * a["real"][:, :, None]).reshape(N, L, Hkv, G).permute(0, 2, 3, 1).reshape(N, Hkv, G * L)
    dv = a["p"].reshape(N, Hkv, G * L, L).transpose(-1, -2) @ d_o
    ds = (d_o @ a["v"].transpose(-1, -2)).sub_(delta[..., None]).mul_(a["p"].reshape(N, Hkv, G * L, L))
    out = {}
    if c["beta"]:
        d_gate = (ds.reshape(N, Hkv, G, L, L) * a["dist"]).sum((2, 3))
        out["d_gate"] = _unpad(d_gate, a, s["d_gate"])
    if c["softcap"]:
        ds *= 1 - a["bent"].square_().reshape(N, Hkv, G * L, L)
    ds *= 1.0 / math.sqrt(d)
    dq = (ds @ a["k"]).reshape(N, Hkv * G, L, d)
    dk = ds.transpose(-1, -2) @ a["q"]
    out.update(o=_unpad(a["o"].reshape(N, Hkv * G, L, d), a, s["o"]), lse=_unpad(a["lse"].reshape(N, Hkv * G, L), a, s["lse"]),
               dq=_unpad(dq, a, s["dq"]), dk=_unpad(dk, a, s["dk"]), dv=_unpad(dv, a, s["dv"]))
    return out


def _plain_plan(s):
    cu, held, table, free = s["cu"].long(), s["len"].long(), s["table"], s["free_count"].long()
    B, H, width = table.shape
    fresh = (cu[1:] - cu[:-1])[:, None]
    before, after = (held + PAGE - 1) // PAGE, (held + fresh + PAGE - 1) // PAGE
    need = after - before
    upto = need.sum(1).cumsum(0)
    served = (need.sum(1) == 0) | (upto <= free)
    first = (need.reshape(-1).cumsum(0) - need.reshape(-1)).reshape(B, H)   # pages taken by the rows ahead
    col = torch.arange(width, device="cuda")
    takes = (col >= before[..., None]) & (col < after[..., None]) & served[:, None, None]
    page = s["free_pages"][(free - 1 - (first - before)[..., None] - col).clamp(0, s["pages"] - 1)]
    table = torch.where(takes, page, table)
    token = torch.arange(s["slot_map"].shape[1], device="cuda")
    b = (torch.searchsorted(cu, token, right=True) - 1).clamp(max=B - 1)
    slot = held[b].T + (token - cu[b])
    row = table[b[None], torch.arange(H, device="cuda")[:, None], (slot // PAGE).clamp(max=width - 1)].long() * PAGE + slot % PAGE
    row = torch.where(served[b], row, -1).to(torch.int32)
    return {"slot_map": torch.where(token < cu[-1], row, s["slot_map"]), "table": table,
            "len": torch.where(served[:, None], held + fresh, held).to(torch.int32),
            "free_count": (free - (need.sum(1) * served).sum()).to(torch.int32)}


def _plain_write(s):
    H = s["case"]["Hkv"]
    head, token = torch.nonzero(s["slot_map"] >= 0, as_tuple=True)
    row = s["slot_map"][head, token].long()
    for x, pages in (("k", s["k_pages"]), ("v", s["v_pages"])):
        pages.view(-1, pages.shape[-1])[row] = s[x][token, head]
    s["pos_pages"].view(-1)[row] = s["pos"][token]
    if s["gate"] is not None:
        s["gate_pages"].view(-1)[row] = s["gate"][token, head]
    return _pages(s)


def _pages(s):
    out = {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "pos_pages": s["pos_pages"]}
    if s["gate"] is not None:
        out["gate_pages"] = s["gate_pages"]
    return out


# ------------------------------------------------------------------ the library's calls

def _pool(s):
    """The paged cache's handle over the state's tensors, made once as a program keeps it."""
    if "pool" not in s:
        import memory_bounded_kv_b200 as kvb
        c = s["case"]
        pool = kvb.PagedPool(c["docs"], c["Hkv"], c.get("d", 64), s["table"].shape[2], s["pages"], with_beta=c.get("beta", False))
        pool.table, pool.len, pool.free_pages, pool.free_count = s["table"], s["len"], s["free_pages"], s["free_count"]
        if c["op"] == "write":
            pool.k_pages, pool.v_pages, pool.pos_pages, pool.log_beta_pages = s["k_pages"], s["v_pages"], s["pos_pages"], s["gate_pages"]
        else:
            s["workspace"] = torch.empty(kvb.kvb_paged_plan_workspace_bytes(c["docs"], c["Hkv"]), dtype=torch.uint8, device="cuda")
        s["pool"] = pool
    return s["pool"]


def _own(s):
    import memory_bounded_kv_b200 as kvb
    c = s["case"]
    if c["op"] == "plan":
        pool = _pool(s)
        # the same call again on the same state: what the last one added is taken back first
        pool.len.copy_(s["len0"])
        pool.free_count.copy_(s["free0"])
        kvb.kvb_paged_plan(pool, s["cu"], s["slot_map"], s["workspace"])
        return {"slot_map": s["slot_map"], "table": pool.table, "len": pool.len, "free_count": pool.free_count}
    if c["op"] == "write":
        kvb.kvb_paged_write(_pool(s), s["k"], s["v"], s["gate"], s["pos"], s["slot_map"])
        return _pages(s)
    kvb.kvb_prefill_attn(s["q"], s["k"], s["v"], s["gate"], s["cu"], s["o"], s["lse"], prefix_len=s["prefix"], softcap=c["softcap"])
    out = {"o": s["o"], "lse": s["lse"]}
    if c["op"] == "train":
        if "workspace" not in s:
            s["workspace"] = torch.empty(kvb.kvb_prefill_attn_bwd_workspace_bytes(s["q"].shape[0], c["Hq"]), dtype=torch.uint8, device="cuda")
        kvb.kvb_prefill_attn_bwd(s["q"], s["k"], s["v"], s["gate"], s["cu"], s["o"], s["lse"], s["d_o"], s["d_lse"], s["dq"], s["dk"],
                                 s["dv"], s["d_gate"], s["workspace"], prefix_len=s["prefix"], softcap=c["softcap"])
        out.update(dq=s["dq"], dk=s["dk"], dv=s["dv"])
        if c["beta"]:
            out["d_gate"] = s["d_gate"]
    return out


def run(state):
    if own:
        return _own(state)
    return {"prefill": _plain_prefill, "train": _plain_train, "plan": _plain_plan, "write": _plain_write}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    if case["op"] == "plan":
        return None   # whole numbers only
    s = prepare(case, seed)
    cu = _starts(case)
    if case["op"] == "write":
        out = {k: t.double().flatten(0, 1) for k, t in _pages(s).items()}
        out["pos_pages"] = None
        for h in range(case["Hkv"]):
            to = s["slot_map"][h, :cu[-1]].long()
            out["k_pages"][to] = s["k"][:cu[-1], h].double()
            out["v_pages"][to] = s["v"][:cu[-1], h].double()
            if case["beta"]:
                out["gate_pages"][to] = s["gate"][:cu[-1], h].double()
        return {k: t if t is None else t.reshape(s[k].shape) for k, t in out.items()}
    G, scale, cap = case["Hq"] // case["Hkv"], case["d"] ** -0.5, case["softcap"]
    res = {k: torch.zeros(s[k].shape, dtype=torch.float64, device="cuda") for k in ("o", "lse", "dq", "dk", "dv", "d_gate") if s.get(k) is not None}
    for b, (n, prefix) in enumerate(zip(lengths(case), _prefixes(case))):
        if n == 0:
            continue
        rows = slice(cu[b], cu[b + 1])
        i = torch.arange(n, device="cuda", dtype=torch.float64)
        age = (i[:, None] - i[None, :]).clamp(min=0)
        hidden = (i[None, :] > i[:, None]) & (i[None, :] >= prefix)
        for h in range(case["Hq"]):
            kv = h // G
            q, k, v = s["q"][rows, h].double(), s["k"][rows, kv].double(), s["v"][rows, kv].double()
            x = torch.einsum("ie,je->ij", q, k) * scale
            slope = None
            if cap:
                y = torch.tanh(x / cap)
                x, slope = cap * y, 1 - y * y
            if case["beta"]:
                x = x + age * s["gate"][rows, kv].double()[None, :]
            x[hidden] = -math.inf
            lse = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[:, None])
            o = p @ v
            res["o"][rows, h], res["lse"][rows, h] = o, lse
            if case["op"] != "train":
                continue
            g = s["d_o"][rows, h].double()
            pull = g @ v.T - (g * o).sum(1, keepdim=True)
            if s["d_lse"] is not None:
                pull = pull + s["d_lse"][rows, h].double()[:, None]
            dx = p * pull
            res["dv"][rows, kv] += p.T @ g
            if case["beta"]:
                res["d_gate"][rows, kv] += (dx * age).sum(0)
            if slope is not None:
                dx = dx * slope
            res["dq"][rows, h] = scale * (dx @ k)
            res["dk"][rows, kv] += scale * (dx.T @ q)
    return res
