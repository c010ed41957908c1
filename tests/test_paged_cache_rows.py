"""A cache that is written has rows of its own, on the CPU: layouts that nest are taken, strides
under which two rows share channels are refused before anything is enqueued."""
import pytest

import kv_cache_csa2_b200 as K
from tests.test_paged_refusals import append, heads

# pages of 16 tokens, 2 heads of 128 channels, 10 pages
OVERLAP = [dict(page_stride=4096, token_stride=128, head_stride=128), dict(page_stride=2048, token_stride=256, head_stride=128),
           dict(page_stride=4096, token_stride=256, head_stride=2048), dict(page_stride=128, token_stride=1280, head_stride=128),
           dict(page_stride=4096, token_stride=136, head_stride=128)]
NEST = [dict(), dict(page_stride=4096, token_stride=128, head_stride=2048), dict(page_stride=8192, token_stride=256, head_stride=128),
        dict(page_stride=128, token_stride=2560, head_stride=1280), dict(page_stride=256, token_stride=2560, head_stride=128),
        dict(page_stride=128, token_stride=128, head_stride=128, heads=1, page_size=1)]


@pytest.mark.parametrize("strides", OVERLAP)
def test_append_refuses_overlapping_rows(strides):
    assert append(**strides) == 1
    assert b"overlap" in K.lib().csa2_last_error()


@pytest.mark.parametrize("strides", NEST)
def test_append_takes_layouts_that_nest(strides):
    n = strides.get("heads", 2)
    assert append(T=0, k=heads(n), v=heads(n), **strides) == 0
