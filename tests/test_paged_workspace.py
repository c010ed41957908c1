"""The scratch a decode call asks for shows its chunk length, on the CPU: the stated multiple for
every format, width and page size."""
import pytest

import kv_cache_csa2_b200 as K
from tests.test_paged_refusals import paged


@pytest.mark.parametrize("fmt,dim,page,unit", [(K.KV_BF16, 512, 64, 128), (K.KV_F16, 512, 8, 128), (K.KV_BF16, 512, 4, 64),
                                               (K.KV_FP4, 512, 64, 64), (K.KV_FP4, 512, 4, 64), (K.KV_BF16, 256, 64, 64),
                                               (K.KV_F16, 128, 16, 64), (K.KV_FP4, 64, 16, 64)])
@pytest.mark.parametrize("chunk", [64, 128, 192, 320])
def test_chunk_lengths(fmt, dim, page, unit, chunk):
    scales = dict(k_scales=4096, v_scales=8192) if fmt == K.KV_FP4 else {}
    tokens, B, Hq = 3840, 3, 8
    need = K.lib().csa2_paged_decode_attn_workspace(paged(fmt=fmt, dim=dim, page_size=page, max_pages=tokens // page, **scales),
                                                    Hq, 0, 0, chunk)
    length = -(-chunk // unit) * unit
    assert need == B * Hq * -(-tokens // length) * (dim * 4 + 8)
