"""Refusals of the prompt path that reach no device, beside those of test_prefill_host.py."""
import ctypes

import pytest
import torch

import memory_bounded_kv_b200 as kvb
from memory_bounded_kv_b200 import _lib
from memory_bounded_kv_b200.cache import PagedKVCache
from test_prefill_host import Hkv, Hq, N, T, args, d


@pytest.fixture
def cache(monkeypatch):
    """A paged cache on the CPU whose kernels note that they were called, and arguments that it takes."""
    monkeypatch.setattr(kvb, "kvb_paged_reset", lambda pool, stream=None: None)
    c = PagedKVCache(N, Hq, Hkv, d, max_pages=2, num_pages=8, M=64, device="cpu")
    c.called = []
    for f in ("kvb_prefill_attn", "kvb_paged_plan", "kvb_paged_write"):
        monkeypatch.setattr(kvb, f, lambda *a, _f=f, **k: c.called.append(_f))
    a = args()
    c.good = dict(q=a["q"], k=a["k"], v=a["v"], log_beta=a["log_beta"], cu=a["cu"], pos=torch.zeros(T, dtype=torch.int32), o=a["o"])
    return c


def test_cache_prefill_has_no_cap(cache):
    """The decode steps that go on from a prompt have none, so a capped prompt would be another attention."""
    with pytest.raises(TypeError):
        cache.prefill(**cache.good, softcap=30.0)
    assert cache.called == []


def test_cache_prefill_refuses_positions_on_another_device(cache):
    """Only the write reads them, and it comes after the plan has taken pages."""
    with pytest.raises(ValueError, match="pos is on meta"):
        cache.prefill(**dict(cache.good, pos=cache.good["pos"].to("meta")))
    assert cache.called == []


def test_plan_within_refuses():
    F = 1 << 20   # a 16-byte aligned non-null value; the host checks never dereference it
    c = ctypes.byref(_lib.PagedCacheArgs(k_pages=F, v_pages=F, log_beta_pages=None, pos_pages=F, table=F, len=F, free_pages=F,
                                         free_count=F, B=2, Hkv=2, d=64, max_pages=4, num_pages=16))
    L = _lib.lib()
    ws = L.kvb_paged_plan_workspace_bytes(2, 2)
    for max_len in (0, -1):
        assert L.kvb_paged_plan_within(c, F, 8, F, 0, max_len, F, ws, None) == _lib.KVB_EINVAL
    assert L.kvb_paged_plan_within(c, F, 8, F, 0, 5, F, ws - 1, None) == _lib.KVB_EINVAL


@pytest.mark.parametrize("kernel,cta,limit", [(-1, 0, 10**6), (3, 0, 10**6), (0, -1, 10**6), (0, 65536, 10**6), (0, 0, 999),
                                              (0, 0, 10**9 + 1)])
def test_withholding_refuses(kernel, cta, limit):
    with pytest.raises(kvb.KvbError):
        kvb.kvb_test_withhold_next_prefill(kernel, cta, limit)
    assert _lib.lib().kvb_test_withhold_next_prefill(kernel, cta, limit) == _lib.KVB_EINVAL
