"""Refusals of the prompt path that reach no device, beside those of test_prefill_host.py."""
import pytest

import memory_bounded_kv_b200 as kvb
from memory_bounded_kv_b200 import _lib


@pytest.mark.parametrize("kernel,cta,limit", [(-1, 0, 10**6), (3, 0, 10**6), (0, -1, 10**6), (0, 65536, 10**6), (0, 0, 999),
                                              (0, 0, 10**9 + 1)])
def test_withholding_refuses(kernel, cta, limit):
    with pytest.raises(kvb.KvbError):
        kvb.kvb_test_withhold_next_prefill(kernel, cta, limit)
    assert _lib.lib().kvb_test_withhold_next_prefill(kernel, cta, limit) == _lib.KVB_EINVAL
