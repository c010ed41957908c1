"""Paged-cache calls in forms that the operator-by-operator tests leave out: tables wider than
the sequences."""
import numpy as np
import pytest
import torch

import kv_cache_csa2_b200 as K
import oracle as O
from tests import paged_util as P

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device_clean():
    yield
    K.csa2_device_error()


def _ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ bits

@pytest.mark.parametrize("kind,D,G,page,window,sinks", [("bf16", 512, 64, 16, 0, 0), ("f16", 512, 33, 64, 0, 0),
                                                        ("bf16", 256, 32, 32, 300, 300), ("f16", 256, 64, 8, 0, 0),
                                                        ("bf16", 512, 4, 16, 0, 0), ("bf16", 128, 8, 16, 0, 0)])
def test_window_bits_do_not_depend_on_the_tables_width(kind, D, G, page, window, sinks):
    """One prompt of 300 tokens through a table of 320 tokens and one of 4096."""
    cache, host = P.make_cache(kind, [300], page, 1, D, shared=True, seed=7)
    q = P.rng_normal(8, 300, G, D, dt=cache.dtype)
    got = []
    for width in (320 // page, 4096 // page):
        table = torch.full((1, width), 2 ** 30, dtype=torch.int32, device="cuda")
        n = min(width, cache.table.shape[1])
        table[:, :n] = cache.table[:, :n]
        wide = K.PagedKv(cache.k, table, cache.lens)
        got.append(K.csa2_paged_window_attn(q, _ints(0, 300), wide, D ** -0.5, window=window, sinks=sinks))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    want = O.causal_attn(P.f64(q), np.arange(300), *host[0], D ** -0.5, window, sinks)
    P.check_attn(*got[0], want, P.f64(q), host[0][0], D ** -0.5, cache.dtype, 300)
