"""Prompts into a paged cache whose sequences may hold no more than the budget."""
import numpy as np
import pytest
import torch

import memory_bounded_kv_b200 as kvb
from memory_bounded_kv_b200 import _lib
from memory_bounded_kv_b200.cache import PagedKVCache
from gpu_util import host
import prefill_bounds as bounds
import prefill_ref as ref
from test_gpu_prefill import PAGE, f64, filled_pool, make

pytestmark = pytest.mark.gpu


def test_a_prompt_longer_than_the_budget_does_not_enter():
    """KVB_DERR_LEN, no slots and no pages for it; the prompts beside it enter, M tokens exactly among them."""
    B, Hq, Hkv, d, M = 4, 4, 2, 64, 100
    cache = PagedKVCache(B, Hq, Hkv, d, max_pages=6, num_pages=30, M=M)
    lens = [M + 1, M, 30, 350]
    cu = np.r_[0, np.cumsum(lens)].tolist()
    c = make(90, cu, cu[-1], Hq, Hkv, d)
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
    o = torch.full((cu[-1], Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    cache.prefill(c["q"], c["k"], c["v"], c["lb"], c["cu"], pos, o)
    assert kvb.kvb_get_error() == _lib.DERR_LEN
    assert cache.len.tolist() == [[0] * 2, [M] * 2, [30] * 2, [0] * 2]
    assert cache.pages_in_use() == 2 * (2 + 1)
    want, bound = bounds.forward(*[f64(c[n]) for n in ("q", "k", "v", "lb")], cu)
    bounds.within(f64(o), want, bound, "o")
    # decode steps keep a full sequence at M and fill one that is not
    t = torch.tensor([-1, M, 30, -1], dtype=torch.int32).cuda()
    for step in range(3):
        new = make(91 + step, [0, B], B, Hq, Hkv, d)
        od = torch.zeros(B, Hq, d, device="cuda")
        cache.step(new["q"], new["k"], new["v"], new["lb"], torch.where(t < 0, t, t + step), od)
        assert cache.len.tolist() == [[0] * 2, [M] * 2, [31 + step] * 2, [0] * 2]
    assert kvb.kvb_get_error() == 0


@pytest.mark.parametrize("held,new,max_len,empty_only", [
    ([0, 10, 64, 0], [100, 90, 37, 101], 100, False),   # just within, just within, one past, one past
    ([120, 0], [0, 5], 100, False),                     # more than that already, without new tokens
    ([120, 3, 0], [1, 1, 100], 100, True),
    ([0, 0], [500, 600], 10**6, False),                 # the table's width (8 pages) stays a limit
])
def test_plan_within(held, new, max_len, empty_only):
    """As kvb_paged_plan on the sequences that fit; the others keep what they hold and take no pages."""
    B, H, pages = len(held), 2, 60
    pool = filled_pool(92, B, H, 8, pages, held)
    cu = np.r_[1, 1 + np.cumsum(new)].astype(np.int32)
    slot_map = torch.full((H, int(cu[-1]) + 2), -7, dtype=torch.int32, device="cuda")
    # the reference plans without a limit, the sequences past it without their tokens
    past = [n > 0 and h + n > max_len for h, n in zip(held, new)]
    gone = np.r_[0, np.cumsum([0 if x else n for x, n in zip(past, new)])].astype(np.int32) + 1
    kept = np.full((H, int(gone[-1]) + 2), -7, np.int32)
    want = ref.plan(gone, host(pool.len), host(pool.table), host(pool.free_pages), int(pool.free_count), kept, pages, PAGE,
                    empty_only)
    smap = np.full(slot_map.shape, -7, np.int32)
    for b in range(B):
        smap[:, cu[b]:cu[b + 1]] = -1 if past[b] else want[0][:, gone[b]:gone[b + 1]]
    ws = torch.empty(kvb.kvb_paged_plan_workspace_bytes(B, H), dtype=torch.uint8, device="cuda")
    kvb.kvb_paged_plan(pool, torch.from_numpy(cu).cuda(), slot_map, ws, empty_only=empty_only, max_len=max_len)
    bits = kvb.kvb_get_error()
    for got, w in ((slot_map, smap), (pool.table, want[1]), (pool.len, want[2])):
        np.testing.assert_array_equal(host(got), w)
    assert int(pool.free_count) == want[3]
    assert bool(bits & _lib.DERR_LEN) == (any(past) or "len" in want[4]) and not bits & ~_lib.DERR_LEN


def test_plan_of_few_tokens_among_many_sequences():
    """The one-launch form with more sequences than its block has threads."""
    B, H, width, pages = 2100, 2, 2, 9000
    g = np.random.default_rng(93)
    held = g.integers(0, 65, B).tolist()
    new = np.where(g.random(B) < 0.3, g.integers(1, 4, B), 0)
    pool = filled_pool(93, B, H, width, pages, held)
    cu = np.r_[3, 3 + np.cumsum(new)].astype(np.int32)
    slot_map = torch.full((H, int(cu[-1]) + 1), -7, dtype=torch.int32, device="cuda")
    assert slot_map.numel() <= 4096
    want = ref.plan(cu, host(pool.len), host(pool.table), host(pool.free_pages), int(pool.free_count), host(slot_map), pages, PAGE)
    ws = torch.empty(kvb.kvb_paged_plan_workspace_bytes(B, H), dtype=torch.uint8, device="cuda")
    kvb.kvb_paged_plan(pool, torch.from_numpy(cu).cuda(), slot_map, ws)
    for got, w in ((slot_map, want[0]), (pool.table, want[1]), (pool.len, want[2])):
        np.testing.assert_array_equal(host(got), w)
    assert int(pool.free_count) == want[3] and kvb.kvb_get_error() == 0
