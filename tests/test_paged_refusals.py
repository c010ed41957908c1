"""Refusals of the head and paged-cache calls, on the CPU: every bad argument is
reported by status before anything is enqueued."""
import ctypes

import pytest
import torch

import kv_cache_csa2_b200 as K

P = ctypes.c_void_p(4096)


def heads(n=8, ts=0, hs=0, data=4096):
    return ctypes.byref(K.CSA2Heads(data, n, ts, hs))


def rope(half=32, offset=0, freq=4096):
    return ctypes.byref(K.CSA2Rope(freq, half, offset, 0, 0))


def paged(**kw):
    d = dict(fmt=K.KV_BF16, k=4096, v=8192, k_scales=None, v_scales=None, n_pages=10, page_stride=0, token_stride=0,
             head_stride=0, page_size=16, heads=2, dim=128, B=3, max_pages=4, table_stride=0, table=4096, lens=4096,
             max_len=0)
    d.update(kw)
    return ctypes.byref(K.CSA2PagedKv(*(d[n] for n, _ in K.CSA2PagedKv._fields_)))


def norm(dtype=0, q=None, q_out=None, k=None, T=4, D=128, positions=P, r=None, weight=None):
    q = heads() if q is None else q
    return K.lib().csa2_qk_norm_rope(dtype, q, weight, heads() if q_out is None else q_out, k, None, None, T, D, 1e-6,
                                     positions, r, None)


def test_norm_rope_refusals():
    bad = [dict(dtype=2), dict(D=132), dict(D=520), dict(D=0), dict(T=-1), dict(q=heads(0)), dict(q=heads(data=0)),
           dict(q=heads(data=4098)), dict(q=heads(ts=1028)), dict(q_out=heads(7)), dict(q_out=heads(ts=8, hs=8)),
           dict(r=rope(half=12)), dict(r=rope(offset=4)), dict(r=rope(half=64, offset=8)), dict(r=rope(freq=0)),
           dict(r=rope(), positions=None), dict(weight=ctypes.c_void_p(4100)), dict(q_out=heads(ts=2048))]
    for kw in bad:
        assert norm(**kw) == 1, kw
    assert K.lib().csa2_qk_norm_rope(0, None, None, None, None, None, None, 4, 128, 1e-6, P, None, None) == 1
    assert norm(T=0, q=heads(data=0), q_out=heads(data=0)) == 0      # no rows: nothing to do


def test_rotation_far_outside_the_row():
    """offset + 2 * half past 32 bits is still outside the row."""
    far = 0x7fffffc0
    assert norm(r=rope(half=32, offset=far)) == 1
    assert append(r=rope(half=32, offset=far)) == 1


def append(dtype=0, k=None, v=None, seq=P, pos=P, T=4, r=None, shared=False, **cache):
    if shared:
        cache["v"] = None
    v = None if shared else heads(2) if v is None else v
    return K.lib().csa2_paged_append(dtype, heads(2) if k is None else k, v, seq, pos, T, r, paged(**cache), None)


def test_append_refusals():
    bad = [dict(dtype=1), dict(fmt=K.KV_F16), dict(fmt=7), dict(T=-1), dict(seq=None), dict(pos=None), dict(k=heads(3)),
           dict(v=heads(1)), dict(page_size=24), dict(page_size=0), dict(page_size=1 << 17), dict(dim=130), dict(dim=520),
           dict(heads=0), dict(n_pages=-1), dict(table=None), dict(k=heads(2, data=0)), dict(table_stride=3),
           dict(page_stride=4096, token_stride=256, head_stride=4), dict(page_stride=4096, token_stride=64, head_stride=128),
           dict(fmt=K.KV_FP4), dict(fmt=K.KV_FP4, k_scales=4096, v_scales=4097), dict(fmt=K.KV_FP4, dim=80, k_scales=4096,
                                                                                      v_scales=4096),
           dict(fmt=K.KV_FP4, k_scales=4096, v_scales=4096, r=rope(half=8)),
           dict(fmt=K.KV_FP4, k_scales=4096, v_scales=4096, r=rope(half=16, offset=8)), dict(v=heads(2, ts=12))]
    for kw in bad:
        assert append(**kw) == 1, kw
    lib = K.lib()
    assert lib.csa2_paged_append(0, heads(2), None, P, P, 4, None, paged(), None) == 1          # separate cache, no v
    assert lib.csa2_paged_append(0, heads(2), heads(2), P, P, 4, None, paged(v=None), None) == 1   # shared cache, v given
    assert lib.csa2_paged_append(0, heads(2), None, P, P, 4, None, None, None) == 1
    assert append(T=0, seq=None, pos=None) == 0


def decode(q=None, Hq=8, window=0, sinks=0, chunk=0, out=P, ws=P, nb=1 << 30, **cache):
    return K.lib().csa2_paged_decode_attn(heads(Hq) if q is None else q, paged(**cache), 0.1, window, sinks, chunk, out,
                                          None, ws, nb, None)


def test_decode_refusals():
    bad = [dict(dim=96), dict(Hq=9), dict(window=-1), dict(sinks=-1), dict(chunk=-64), dict(chunk=100), dict(out=None),
           dict(out=ctypes.c_void_p(4100)), dict(lens=None), dict(table=None), dict(q=heads(8, data=0)),
           dict(page_size=3), dict(fmt=9), dict(B=70000), dict(k=None), dict(k=4100), dict(max_len=-1)]
    for kw in bad:
        assert decode(**kw) == 1, kw
    assert decode(B=0) == 0
    # scratch: long sequences are split, their partials need room
    need = K.lib().csa2_paged_decode_attn_workspace(paged(max_pages=4096), 8, 0, 0, 256)
    chunks = 4096 * 16 // 256
    assert need == 3 * 8 * chunks * (128 * 4 + 8)
    assert decode(max_pages=4096, chunk=256, nb=need - 1) == 6
    assert decode(max_pages=4096, chunk=256, ws=None) == 6
    assert K.lib().csa2_paged_decode_attn_workspace(paged(max_pages=4096, max_len=256), 8, 0, 0, 256) == 0
    assert K.lib().csa2_paged_decode_attn_workspace(paged(max_pages=4096), 8, 100, 20, 128) == 0
    assert K.lib().csa2_paged_decode_attn_workspace(paged(), 9, 0, 0, 0) == 0


def window(q=None, cu=P, T=10, win=0, sinks=0, out=P, **cache):
    return K.lib().csa2_paged_window_attn(heads(8) if q is None else q, cu, T, paged(**cache), 0.1, win, sinks, out, None,
                                          None)


def test_window_refusals():
    bad = [dict(dim=96), dict(q=heads(7)), dict(win=-1), dict(sinks=-2), dict(out=None), dict(cu=None), dict(T=-1),
           dict(T=1 << 31), dict(lens=None), dict(q=heads(8, data=0))]
    for kw in bad:
        assert window(**kw) == 1, kw
    assert window(T=0) == 0 and window(B=0) == 0


def test_fault_injection_covers_the_calls():
    try:
        K.set_fault("launch")
        assert [norm(), append(), decode(), window()] == [4] * 4
    finally:
        K.set_fault("")


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        K.csa2_qk_norm_rope(x, None)                                 # not on a GPU
    with pytest.raises(ValueError):
        K.PagedKv(torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16), torch.zeros(1, 2, dtype=torch.int32),
                  torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        K._rows(torch.zeros(4, 2, 64).to(torch.bfloat16).expand(4, 2, 64)[:, :, ::2], "x")
    with pytest.raises(ValueError):
        K._rows(torch.zeros(1, 2, 64, dtype=torch.bfloat16).expand(4, 2, 64), "x")
    with pytest.raises(ValueError):
        K._rows(torch.zeros(4, 2, 64), "x")
    with pytest.raises(ValueError):
        K._ints(torch.zeros(4, dtype=torch.int64), "x", 4)
