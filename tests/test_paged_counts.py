"""Windows, sinks and chunks past 32 bits are refused by the binding, on the CPU: cut to 32 bits,
2^32 + 5 would be a window of 5 and 2^32 none at all."""
import pytest

import kv_cache_csa2_b200 as K


@pytest.mark.parametrize("x", [1 << 31, 1 << 32, (1 << 32) + 5, -(1 << 32), -(1 << 31) - 1])
def test_counts_past_32_bits(x):
    for kw in (dict(window=x), dict(sinks=x), dict(chunk=x)):
        with pytest.raises(ValueError, match="32 bits"):
            K.csa2_paged_decode_attn(None, None, 1.0, **kw)
    for kw in (dict(window=x), dict(sinks=x)):
        with pytest.raises(ValueError, match="32 bits"):
            K.csa2_paged_window_attn(None, None, None, 1.0, **kw)
