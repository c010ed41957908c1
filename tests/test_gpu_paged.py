"""GPU parity of the head and paged-cache calls (include/csa2.h, part p) through the
public binding, against the float64 oracle; bounds in paged_util."""
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


def _freq(half, base=10000.0):
    return (base ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()


# ------------------------------------------------------------------ head norm and rotation

def _check_rows(got, exact, before, rope, dt):
    """before: the normed rows; a rotated channel's error scales with its pair."""
    pair = np.abs(before).copy()
    if rope is not None:
        half, off, inter = rope
        a = off + (2 * np.arange(half) if inter else np.arange(half))
        b = a + 1 if inter else a + half
        pair[..., a] = pair[..., b] = np.abs(before[..., a]) + np.abs(before[..., b])
    slack = 2.0 ** -19 * pair
    tol = P.half_step(dt) * (np.abs(exact) + slack) + slack + (2.0 ** -25 if dt == torch.float16 else 0.0)
    assert np.all(np.abs(P.f64(got) - exact) <= tol), np.abs(P.f64(got) - exact).max()


@pytest.mark.parametrize("T,Hq,Hk,D,half,off,inter,inverse,dt", [
    (1, 16, 1, 128, 64, 0, False, False, "bf16"), (3, 5, 2, 64, 32, 0, False, True, "f16"),
    (129, 8, 8, 128, 32, 64, True, False, "bf16"), (7, 64, 1, 512, 32, 448, True, False, "f16"),
    (65, 3, 1, 96, 16, 24, False, False, "bf16"), (2, 1, 1, 8, 0, 0, False, False, "f16"),
    (33, 7, 2, 80, 40, 0, False, False, "bf16"), (1200, 9, 3, 256, 128, 0, True, True, "f16"),
    (4000, 8, 1, 512, 256, 0, False, False, "bf16"), (5, 2, 1, 40, 8, 16, True, False, "bf16")])
@pytest.mark.parametrize("norm", [True, False])
def test_norm_rope(T, Hq, Hk, D, half, off, inter, inverse, dt, norm):
    dt = P.DT[dt]
    qkv = P.rng_normal(1, T, Hq + 2 * Hk, D, dt=dt, std=3.0)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    r = np.random.default_rng(2)
    pos = torch.from_numpy(r.integers(-5, 1 << 20, T).astype(np.int32)).cuda()
    wq = torch.from_numpy(r.standard_normal(D).astype(np.float32)).cuda() if norm else None
    wk = torch.from_numpy(r.standard_normal(D).astype(np.float32)).cuda() if norm else None
    freq = _freq(half) if half else None
    rope = K.Rope(freq, offset=off, interleaved=inter, inverse=inverse) if half else None
    qo, ko = K.csa2_qk_norm_rope(q, k, pos if half else None, q_weight=wq, k_weight=wk, eps=1e-5, rope=rope)
    for x, w, o in ((q, wq, qo), (k, wk, ko)):
        n = O.head_norm(P.f64(x), None if w is None else P.f64(w), 1e-5)
        exact = O.rotate(n, pos.cpu().numpy(), P.f64(freq), off, inter, inverse) if half else n
        _check_rows(o, exact, n, (half, off, inter) if half else None, dt)
    # one side alone, in place, gives the same bits; the rows beside it stay
    before = qkv.clone()
    K.csa2_qk_norm_rope(None, k, pos if half else None, k_weight=wk, eps=1e-5, rope=rope, k_out=k)
    assert torch.equal(k, ko) and torch.equal(qkv[:, :Hq], before[:, :Hq])
    assert torch.equal(qkv[:, Hq + Hk:], before[:, Hq + Hk:])


def test_norm_rope_head_major_and_inverse_undoes():
    T, H, D = 37, 6, 128
    x = P.rng_normal(3, H, T, D).transpose(0, 1)                     # head-major rows
    out = torch.empty(H, T, D, dtype=x.dtype, device="cuda").transpose(0, 1)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 7919
    f = _freq(64)
    K.csa2_qk_norm_rope(x, None, pos, rope=K.Rope(f), q_out=out)
    assert torch.equal(out, K.csa2_qk_norm_rope(x.contiguous(), None, pos, rope=K.Rope(f))[0])
    back = K.csa2_qk_norm_rope(out, None, pos, rope=K.Rope(f, inverse=True))[0]
    # two roundings to bf16 of a pair of norm |x|: each channel off by at most 2 u (|a| + |b|) + one rounding
    pair = x.float().abs()
    pair = pair[..., :64] + pair[..., 64:]
    assert torch.all((back.float() - x.float()).abs() <= 4 * P.half_step(x.dtype) * torch.cat((pair, pair), -1))


def test_norm_rope_special_rows():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    x[1] = float("nan")
    x[2] = 3e38
    x[3, 0, 5] = float("inf")
    w = torch.ones(64, device="cuda")
    y = K.csa2_qk_norm_rope(x, None, q_weight=w)[0]
    assert torch.all(y[0] == 0)                                      # eps keeps a zero row finite
    assert torch.isnan(y[1]).all() and torch.all(y[3, 1] == 0)
    assert torch.all(y[2] == 0)                                      # the sum of squares overflows: x / inf


# ------------------------------------------------------------------ append

def _append_case(kind, B, page, heads, D, shared, layout, T, pad, seed, rope):
    cache, _ = P.make_cache(kind, [600 + 17 * b for b in range(B)], page, heads, D, shared=shared, seed=seed,
                            layout=layout)
    r = np.random.default_rng(seed)
    spots = r.permutation([(b, j) for b in range(B) for j in range(600)])[:T]
    seq = np.concatenate([spots[:, 0], np.full(pad, -1)]).astype(np.int32)
    pos = np.concatenate([spots[:, 1], r.integers(-9, 9, pad)]).astype(np.int32)
    mix = r.permutation(T + pad)                                     # padded rows anywhere
    seq, pos = seq[mix], pos[mix]
    k = P.rng_normal(seed + 1, T + pad, heads, D, dt=cache.dtype, std=2.0)
    v = None if shared else P.rng_normal(seed + 2, T + pad, heads, D, dt=cache.dtype, std=2.0)
    return cache, seq, pos, k, v


@pytest.mark.parametrize("kind,B,page,heads,D,shared,layout,T,pad,half,off,inter", [
    ("bf16", 1, 64, 1, 128, True, "dense", 1, 0, 64, 0, False), ("bf16", 3, 16, 8, 128, False, "dense", 61, 3, 64, 0, False),
    ("f16", 2, 1, 2, 64, False, "heads", 130, 0, 16, 32, True), ("f16", 4, 32, 3, 96, False, "pair", 7, 30, 0, 0, False),
    ("bf16", 2, 128, 1, 512, True, "dense", 700, 5, 32, 448, True), ("fp4", 3, 64, 4, 128, False, "pair", 200, 9, 32, 32, False),
    ("fp4", 1, 16, 1, 512, True, "dense", 64, 0, 32, 448, True), ("fp4", 2, 64, 2, 64, False, "heads", 33, 1, 16, 0, False),
    ("fp4", 2, 32, 5, 256, False, "dense", 300, 0, 0, 0, False)])
def test_append(kind, B, page, heads, D, shared, layout, T, pad, half, off, inter):
    cache, seq, pos, k, v = _append_case(kind, B, page, heads, D, shared, layout, T, pad, 11, half)
    freq = _freq(half) if half else None
    rope = K.Rope(freq, offset=off, interleaved=inter) if half else None
    before = [None if t is None else t.clone() for t in cache.tensors]
    K.csa2_paged_append(cache, k, v, torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda(), rope=rope)
    live = np.flatnonzero(seq >= 0)
    table = cache.table.cpu().numpy()
    page_of = table[seq[live], pos[live] // page].astype(np.int64)
    slot = pos[live] % page
    rows = torch.from_numpy(live).cuda()
    turned = k if rope is None else K.csa2_qk_norm_rope(k, None, torch.from_numpy(pos).cuda(), rope=rope)[0]
    exact = P.f64(k) if rope is None else O.rotate(P.f64(k), pos, P.f64(freq), off, inter)
    _check_rows(turned, exact, P.f64(k), (half, off, inter) if half else None, cache.dtype)
    for data, scales, old, old_s, new in ((cache.k, cache.k_scales, before[0], before[2], turned),
                                          (cache.v, cache.v_scales, before[1], before[3], v)):
        if data is None:
            continue
        idx = (torch.from_numpy(page_of).cuda(), torch.from_numpy(slot.astype(np.int64)).cuda())
        want, want_s = old.clone(), None if old_s is None else old_s.clone()
        if kind == "fp4":                                            # exactly csa2_fp4_pack of the rounded row
            codes, sc = K.csa2_fp4_pack(new[rows].contiguous())
            want[idx], want_s[idx] = codes, sc
            assert torch.equal(scales, want_s)
        else:
            want[idx] = new[rows]
        assert torch.equal(data.view(torch.uint8) if kind == "fp4" else data.view(torch.int16),
                           want.view(torch.uint8) if kind == "fp4" else want.view(torch.int16))


def test_append_records_bad_places_and_skips_them():
    cache, _ = P.make_cache("bf16", [100, 100], 16, 2, 64, seed=5)
    cache.table[1, 2] = -7
    cache.table[1, 3] = cache.k.shape[0]
    before = (cache.k.clone(), cache.v.clone())
    k, v = P.rng_normal(1, 6, 2, 64), P.rng_normal(2, 6, 2, 64)
    cap = cache.table.shape[1] * 16
    seq = torch.tensor([2, 0, 0, 1, 1, -2], dtype=torch.int32, device="cuda")
    pos = torch.tensor([3, -1, cap, 32, 48, 0], dtype=torch.int32, device="cuda")
    K.csa2_paged_append(cache, k, v, seq, pos)
    with pytest.raises(K.CSA2Error) as e:
        K.csa2_device_error()
    assert e.value.status == 7
    assert torch.equal(cache.k.view(torch.int16), before[0].view(torch.int16))
    assert torch.equal(cache.v.view(torch.int16), before[1].view(torch.int16))


# ------------------------------------------------------------------ decode attention

def _decode_check(kind, lens, page, heads, G, D, shared, layout, window, sinks, chunk, seed, max_len=0):
    cache, host = P.make_cache(kind, lens, page, heads, D, shared=shared, seed=seed, layout=layout, max_len=max_len)
    B, Hq = len(lens), heads * G
    wide = P.rng_normal(seed + 9, B, Hq + 3, D, dt=cache.dtype)
    q = wide[:, 1:1 + Hq]                                            # a strided slice
    scale = 1.3 * D ** -0.5
    out, lse = K.csa2_paged_decode_attn(q, cache, scale, window=window, sinks=sinks, chunk=chunk)
    qh = P.f64(q)
    for b, n in enumerate(lens):
        want = O.causal_attn(qh[b:b + 1], [n - 1], *host[b], scale, window, sinks)
        P.check_attn(out[b:b + 1], lse[b:b + 1], want, qh[b:b + 1], host[b][0], scale, cache.dtype, n, f"seq {b} of {n}")
    return cache, q, scale, out, lse


@pytest.mark.parametrize("kind", ["bf16", "f16", "fp4"])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("page,heads,G,shared,layout,window,sinks,chunk", [
    (16, 2, 4, False, "dense", 0, 0, 0), (64, 1, 16, True, "dense", 0, 0, 64), (1, 2, 3, False, "heads", 100, 3, 0),
    (32, 1, 64, True, "dense", 129, 70, 128), (128, 3, 1, False, "pair", 1, 0, 0), (8, 1, 33, False, "heads", 0, 0, 192)])
def test_decode(kind, D, page, heads, G, shared, layout, window, sinks, chunk):
    _decode_check(kind, [0, 1, 2, 63, 64, 65, 131, 517], page, heads, G, D, shared, layout, window, sinks, chunk, 21)


@pytest.mark.parametrize("kind,D,heads,G,shared", [("bf16", 128, 1, 16, True), ("fp4", 128, 2, 8, False),
                                                   ("f16", 64, 2, 7, False), ("bf16", 512, 1, 64, True)])
def test_decode_long_and_split(kind, D, heads, G, shared):
    cache, q, scale, out, lse = _decode_check(kind, [5000, 3, 2049, 0], 64, heads, G, D, shared, "dense", 0, 0, 0, 31)
    # a bound of the lengths changes the split, not the answer; a sequence past it is still attended whole
    for max_len in (5000, 2048, 1):
        again = K.PagedKv(cache.k, cache.table, cache.lens, v=cache.v, k_scales=cache.k_scales, v_scales=cache.v_scales,
                          max_len=max_len)
        o2, l2 = K.csa2_paged_decode_attn(q, again, scale)
        assert torch.allclose(l2, lse, rtol=1e-5, atol=1e-5)
        assert (o2.float() - out.float()).abs().max() <= 4 * P.half_step(out.dtype) * 8
    # with a fixed chunk a query's bits do not depend on its batch
    o3, l3 = K.csa2_paged_decode_attn(q, cache, scale, chunk=256)
    one = K.PagedKv(cache.k, cache.table[2:3], cache.lens[2:3], v=cache.v, k_scales=cache.k_scales, v_scales=cache.v_scales)
    o4, l4 = K.csa2_paged_decode_attn(q[2:3], one, scale, chunk=256)
    assert torch.equal(o3[2:3], o4) and torch.equal(l3[2:3], l4)


def test_decode_huge_scores_and_identical_keys():
    """Scores of +-thousands (the weights of all but one key vanish) and equal keys (uniform weights)."""
    cache, host = P.make_cache("bf16", [300, 300], 16, 1, 128, seed=41, std=30.0)
    q = P.rng_normal(42, 2, 8, 128, std=30.0)
    out, lse = K.csa2_paged_decode_attn(q, cache, 1.0)
    for b in range(2):
        want = O.causal_attn(P.f64(q[b:b + 1]), [299], *host[b], 1.0)
        score = np.sort(P.f64(q[b]) @ host[b][0][:, 0].T, -1)
        top = np.argmax(P.f64(q[b]) @ host[b][0][:, 0].T, -1)
        alone = score[:, -1] - score[:, -2] > 40                     # the other weights are below e^-40: the value itself
        assert alone.any()
        np.testing.assert_array_equal(P.f64(out[b])[alone], host[b][1][top, 0][alone])
        np.testing.assert_allclose(P.f64(lse[b])[alone], want[1][0][alone], rtol=2.0 ** -20)
    cache.k[...] = torch.where(torch.isnan(cache.k), cache.k, torch.ones_like(cache.k))
    out, lse = K.csa2_paged_decode_attn(q, cache, 0.01)
    for b in range(2):
        mean = host[b][1][:, 0].mean(0)
        mag = np.abs(host[b][1][:, 0]).mean(0)
        assert np.all(np.abs(P.f64(out[b]) - mean) <= P.half_step(torch.bfloat16) * (np.abs(mean) + 1.02 * mag) + 2e-5 * mag)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("G", [1, 5, 8, 9, 16, 17])
@pytest.mark.parametrize("shared,window,sinks,sign", [(False, 0, 0, 1.0), (True, 150, 5, -1.0)])
def test_decode_fp4_groups_and_magnitudes(D, G, shared, window, sinks, sign):
    """Query heads that fill the products' columns or not, each of its own magnitude (0 among
    them), a page that is not in the pool, and a length inside a slice."""
    lens, page = [700, 33, 18], 16
    cache, host = P.make_cache("fp4", lens, page, 2, D, shared=shared, seed=151)
    q = P.rng_normal(152, 3, 2 * G, D)
    q *= torch.tensor([1.0, 2.0 ** -20, 0.0, 8.0, 2.0 ** -3], device="cuda").repeat(2 * G)[:2 * G, None].to(q.dtype)
    gone = 2 if window == 0 else 40                                  # a page that is seen
    cache.table[0, gone] = -3
    scale = sign * D ** -0.5
    out, lse = K.csa2_paged_decode_attn(q, cache, scale, window=window, sinks=sinks, chunk=128)
    with pytest.raises(K.CSA2Error):
        K.csa2_device_error()
    qh = P.f64(q)
    for b, n in enumerate(lens):
        at = np.arange(n)
        seen = (n - 1 - at < window) | (at < sinks) if window else at >= 0
        if b == 0:
            seen &= at // page != gone
        k, v = host[b][0][seen], host[b][1][seen]
        want = O.causal_attn(qh[b:b + 1], [len(k) - 1], k, v, scale)
        P.check_attn(out[b:b + 1], lse[b:b + 1], want, qh[b:b + 1], k, abs(scale), torch.bfloat16, n, f"seq {b}")


def test_decode_bad_table_and_length():
    cache, host = P.make_cache("bf16", [200, 40, 10], 16, 1, 128, seed=51)
    q = P.rng_normal(52, 3, 4, 128)
    cache.table[0, 3] = cache.k.shape[0] + 5                         # tokens 48..63 of sequence 0 are lost
    out, lse = K.csa2_paged_decode_attn(q, cache, 0.1)
    with pytest.raises(K.CSA2Error) as e:
        K.csa2_device_error()
    assert e.value.status == 7
    keep = np.r_[0:48, 64:200]
    want = O.causal_attn(P.f64(q[:1]), [len(keep) - 1], host[0][0][keep], host[0][1][keep], 0.1)
    P.check_attn(out[:1], lse[:1], want, P.f64(q[:1]), host[0][0], 0.1, torch.bfloat16, 200)
    cache.table[0, 3] = 0
    cache.lens[1] = -4
    out, lse = K.csa2_paged_decode_attn(q, cache, 0.1)
    with pytest.raises(K.CSA2Error):
        K.csa2_device_error()
    assert torch.all(out[1] == 0) and torch.all(torch.isneginf(lse[1]))


# ------------------------------------------------------------------ prompt attention

def _window_check(kind, news, lens, page, heads, G, D, shared, layout, window, sinks, seed, tail=0):
    cache, host = P.make_cache(kind, lens, page, heads, D, shared=shared, seed=seed, layout=layout)
    T, Hq = sum(news) + tail, heads * G
    q = P.rng_normal(seed + 9, T, Hq + 2, D, dt=cache.dtype)[:, 2:]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device="cuda")
    out = torch.full((T, Hq, D), 7.0, dtype=cache.dtype, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    scale = D ** -0.5
    K.csa2_paged_window_attn(q, cu, cache, scale, window=window, sinks=sinks, out=out, lse=lse)
    qh, at = P.f64(q), 0
    for b, (n, total) in enumerate(zip(news, lens)):
        sl = slice(at, at + n)
        want = O.causal_attn(qh[sl], np.arange(total - n, total), *host[b], scale, window, sinks)
        P.check_attn(out[sl], lse[sl], want, qh[sl], host[b][0], scale, cache.dtype, total, f"seq {b}: {n} of {total}")
        at += n
    assert torch.all(out[at:] == 7) and torch.all(lse[at:] == 7)     # rows behind the last sequence
    return cache, q, cu, scale, out, lse


@pytest.mark.parametrize("kind", ["bf16", "f16", "fp4"])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("page,heads,G,shared,layout,window,sinks", [
    (16, 2, 4, False, "dense", 0, 0), (64, 1, 16, True, "dense", 40, 4), (1, 2, 3, False, "heads", 100, 0),
    (32, 1, 33, True, "dense", 1, 0), (128, 3, 1, False, "pair", 64, 70)])
def test_window(kind, D, page, heads, G, shared, layout, window, sinks):
    _window_check(kind, [1, 0, 130, 33, 5, 64], [1, 9, 130, 200, 5, 257], page, heads, G, D, shared, layout, window,
                  sinks, 61, tail=3)


@pytest.mark.parametrize("kind,D,heads,G,window,sinks", [("bf16", 512, 1, 64, 0, 0), ("f16", 256, 2, 40, 600, 9),
                                                         ("bf16", 128, 2, 8, 128, 4), ("f16", 64, 1, 4, 0, 0),
                                                         ("bf16", 128, 1, 1, 300, 130)])
def test_window_longer(kind, D, heads, G, window, sinks):
    _window_check(kind, [700, 3, 411], [700, 900, 1000], 64, heads, G, D, False, "dense", window, sinks, 71)


def test_window_rows_before_the_start_see_nothing():
    """More new rows than cached tokens: the first positions would be negative."""
    cache, host = P.make_cache("bf16", [5], 16, 1, 64, seed=75)
    q = P.rng_normal(76, 9, 4, 64)
    cu = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    out, lse = K.csa2_paged_window_attn(q, cu, cache, 0.125)
    assert torch.all(out[:4] == 0) and torch.all(torch.isneginf(lse[:4]))
    want = O.causal_attn(P.f64(q[4:]), np.arange(5), *host[0], 0.125)
    P.check_attn(out[4:], lse[4:], want, P.f64(q[4:]), host[0][0], 0.125, torch.bfloat16, 5)


@pytest.mark.parametrize("kind,D,G,window", [("bf16", 512, 64, 0), ("bf16", 128, 8, 0), ("f16", 64, 3, 90), ("bf16", 512, 16, 50)])
def test_window_bits_do_not_depend_on_batch_or_cut(kind, D, G, window):
    cache, q, cu, scale, out, lse = _window_check(kind, [203, 340], [203, 400], 16, 1, G, D, True, "dense", window, 3, 81)
    # the second sequence alone, its last 77 tokens as a chunk of their own
    one = K.PagedKv(cache.k, cache.table[1:], cache.lens[1:], k_scales=cache.k_scales)
    o, l = K.csa2_paged_window_attn(q[-77:], torch.tensor([0, 77], dtype=torch.int32, device="cuda"), one, scale,
                                    window=window, sinks=3)
    assert torch.equal(o, out[-77:]) and torch.equal(l, lse[-77:])


@pytest.mark.parametrize("D,page,shared", [(64, 8, False), (128, 16, False), (128, 32, True), (128, 2, False)])
def test_window_ignores_what_ran_before(D, page, shared):
    """A launch over NaN values leaves them in shared memory; the next one, whose window starts
    inside a block of tokens and whose pages end inside it, must not see them."""
    cache, host = P.make_cache("bf16", [300], page, 1, D, shared=shared, seed=87)
    q = P.rng_normal(88, 40, 8, D)
    cu = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    bad = K.PagedKv(torch.full_like(cache.k, float("nan")), cache.table, cache.lens,
                    v=None if shared else torch.full_like(cache.k, float("nan")))
    wide = P.rng_normal(89, 40 * 32, 8, D)                           # every SM
    many = K.PagedKv(bad.k, cache.table.expand(32, -1).contiguous(), cache.lens.expand(32).contiguous(), v=bad.v)
    for window, sinks in ((53, 0), (70, 3), (0, 0), (17, 9)):
        K.csa2_paged_window_attn(wide, torch.arange(33, dtype=torch.int32, device="cuda") * 40, many, 0.1)
        out, lse = K.csa2_paged_window_attn(q, cu, cache, 0.1, window=window, sinks=sinks)
        want = O.causal_attn(P.f64(q), np.arange(260, 300), *host[0], 0.1, window, sinks)
        P.check_attn(out, lse, want, P.f64(q), host[0][0], 0.1, torch.bfloat16, 300)


@pytest.mark.parametrize("kind,D,G,page,shared,window,sinks,scale", [
    ("bf16", 128, 8, 16, False, 0, 0, 0.1), ("f16", 64, 3, 64, False, 50, 4, 0.1), ("bf16", 64, 1, 4, False, 33, 0, -0.1),
    ("bf16", 128, 16, 32, True, 40, 0, 0.1), ("f16", 256, 2, 16, False, 50, 4, 0.1), ("bf16", 512, 4, 16, True, 0, 0, -0.1)])
def test_window_masked_values_that_are_not_finite(kind, D, G, page, shared, window, sinks, scale):
    """A NaN or infinite row reaches only the queries that see its token."""
    n, L = 150, 260
    cache, host = P.make_cache(kind, [L], page, 1, D, shared=shared, seed=93)
    dt = cache.dtype
    table = cache.table.cpu().numpy()
    odd = {141: float("nan"), 200: float("inf"), 201: float("-inf"), 259: float("nan")}
    for j, x in odd.items():
        rows = cache.k if shared else cache.v
        rows[table[0, j // page], j % page, 0, 3 * j % D] = x
    q = P.rng_normal(94, n, G, D, dt=dt)
    out, lse = K.csa2_paged_window_attn(q, torch.tensor([0, n], dtype=torch.int32, device="cuda"), cache, scale,
                                        window=window, sinks=sinks)
    pos = np.arange(L - n, L)
    sees = lambda j: (j <= pos) & ((window == 0) | (pos - j < window) | (j < sinks))
    clean = ~np.any([sees(j) for j in odd], 0)
    assert 20 < clean.sum() < n
    rows = torch.from_numpy(np.flatnonzero(clean)).cuda()
    want = O.causal_attn(P.f64(q[rows]), pos[clean], *host[0], scale, window, sinks)
    P.check_attn(out[rows], lse[rows], want, P.f64(q[rows]), host[0][0], abs(scale), dt, L)
    if not shared:
        got = P.f64(out)
        for j in odd:
            assert not np.isfinite(got[sees(j)][:, :, 3 * j % D]).any()


def test_window_scores_far_below_the_maximum():
    """Scores thousands below the row's largest weigh nothing; equal scores weigh the same."""
    cache, host = P.make_cache("bf16", [200], 16, 1, 64, seed=97, std=20.0)
    q = P.rng_normal(98, 70, 4, 64, std=20.0)
    cu = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    out, lse = K.csa2_paged_window_attn(q, cu, cache, 1.0)
    qh, pos = P.f64(q), np.arange(130, 200)
    want = O.causal_attn(qh, pos, *host[0], 1.0)
    s = np.einsum("qhd,kd->qhk", qh, host[0][0][:, 0])
    s = np.where(np.arange(200) > pos[:, None, None], -np.inf, s)
    order = np.sort(s, -1)
    alone = order[..., -1] - order[..., -2] > 40                     # the other weights are below e^-40
    assert alone.mean() > 0.5
    np.testing.assert_array_equal(P.f64(out)[alone], host[0][1][np.argmax(s, -1), 0][alone])
    np.testing.assert_allclose(P.f64(lse)[alone], want[1][alone], rtol=2.0 ** -20)
    out, lse = K.csa2_paged_window_attn(torch.zeros_like(q), cu, cache, 1.0)
    for i in (0, 69):
        mean, mag = host[0][1][:pos[i] + 1, 0].mean(0), np.abs(host[0][1][:pos[i] + 1, 0]).mean(0)
        assert np.all(np.abs(P.f64(out[i]) - mean) <= P.half_step(torch.bfloat16) * (np.abs(mean) + 1.02 * mag) + 2e-5 * mag)
    np.testing.assert_allclose(P.f64(lse), np.log(pos + 1.0)[:, None].repeat(4, 1), rtol=2.0 ** -20)


def test_window_bad_cu_q():
    cache, _ = P.make_cache("bf16", [50, 50, 50], 16, 1, 64, seed=85)
    q = P.rng_normal(86, 40, 2, 64)
    good = K.csa2_paged_window_attn(q, torch.tensor([0, 10, 20, 40], dtype=torch.int32, device="cuda"), cache, 0.1)
    out = torch.full_like(q, 7.0)
    # sequence 0 descends, sequence 1 leaves [0, T]: both skipped
    K.csa2_paged_window_attn(q, torch.tensor([12, 10, 50, 40], dtype=torch.int32, device="cuda"), cache, 0.1, out=out)
    with pytest.raises(K.CSA2Error) as e:
        K.csa2_device_error()
    assert e.value.status == 7
    assert torch.all(out == 7)
    K.csa2_paged_window_attn(q, torch.tensor([12, 10, 20, 40], dtype=torch.int32, device="cuda"), cache, 0.1, out=out)
    with pytest.raises(K.CSA2Error):
        K.csa2_device_error()
    assert torch.equal(out[10:], good[0][10:])


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_layer_prompt_then_tokens(kind):
    """A layer as a server runs it: norm and rotate the prompt's heads, append, attend with
    a window and sinks; then tokens one by one (captured once, replayed per token with the
    lengths advanced on the device), padded to the graph's batch."""
    B, Hq, Hk, D, page, W, S = 3, 8, 2, 128, 16, 40, 2
    news = [50, 1, 77]
    steps = 5
    cap = 96
    n_pages = B * (cap // page)
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(3)).view(B, -1).int().cuda()
    if kind == "fp4":
        mk = lambda w: torch.zeros(n_pages, page, Hk, w, dtype=torch.uint8, device="cuda")
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        cache = K.PagedKv(mk(D // 2), perm, lens, v=mk(D // 2), k_scales=mk(D // 16), v_scales=mk(D // 16))
    else:
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        mk = lambda: torch.full((n_pages, page, Hk, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        cache = K.PagedKv(mk(), perm, lens, v=mk())
    f = _freq(D // 2)
    rope, wq, wk = K.Rope(f), torch.rand(D, device="cuda") + 0.5, torch.rand(D, device="cuda") + 0.5
    total = [n + steps for n in news]
    x = [P.rng_normal(100 + b, total[b], Hq + 2 * Hk, D) for b in range(B)]

    # the float64 side, with the rounding of stored rows
    keys, vals, qs = [], [], []
    for b in range(B):
        pos = torch.arange(total[b], dtype=torch.int32, device="cuda")
        qr, kr = K.csa2_qk_norm_rope(x[b][:, :Hq], x[b][:, Hq:Hq + Hk], pos, q_weight=wq, k_weight=wk, rope=rope)
        exact = O.rotate(O.head_norm(P.f64(x[b][:, Hq:Hq + Hk]), P.f64(wk), 1e-6), np.arange(total[b]), P.f64(f))
        _check_rows(kr, exact, O.head_norm(P.f64(x[b][:, Hq:Hq + Hk]), P.f64(wk), 1e-6), (D // 2, 0, False), kr.dtype)
        v = x[b][:, Hq + Hk:].contiguous()
        if kind == "fp4":
            kr, v = K.csa2_fp4_unpack(*K.csa2_fp4_pack(kr)), K.csa2_fp4_unpack(*K.csa2_fp4_pack(v))
        keys.append(P.f64(kr)), vals.append(P.f64(v)), qs.append(P.f64(qr))
    scale = D ** -0.5

    def check(out, lse, b, at, what):
        n = out.shape[0]
        want = O.causal_attn(qs[b][at:at + n], np.arange(at, at + n), keys[b], vals[b], scale, W, S)
        P.check_attn(out, lse, want, qs[b][at:at + n], keys[b], scale, torch.bfloat16, total[b], what)

    # prompt
    xp = torch.cat([x[b][:news[b]] for b in range(B)])
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(news)]).int().cuda()
    pos = torch.cat([torch.arange(n) for n in news]).int().cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device="cuda")
    lens.copy_(torch.tensor(news, dtype=torch.int32))
    q, k = K.csa2_qk_norm_rope(xp[:, :Hq], xp[:, Hq:Hq + Hk], pos, q_weight=wq, k_weight=wk, rope=rope)
    K.csa2_paged_append(cache, k, xp[:, Hq + Hk:], seq, pos)
    out, lse = K.csa2_paged_window_attn(q, cu, cache, scale, window=W, sinks=S)
    for b, n in enumerate(news):
        check(out[cu[b]:cu[b] + n], lse[cu[b]:cu[b] + n], b, 0, f"prompt {b}")

    # one token per step: static inputs, one graph
    xin = torch.zeros(B + 2, Hq + 2 * Hk, D, dtype=torch.bfloat16, device="cuda")
    seq1 = torch.tensor([0, 1, 2, -1, -1], dtype=torch.int32, device="cuda")
    pos1 = torch.zeros(B + 2, dtype=torch.int32, device="cuda")

    def step():
        pos1[:B] = lens
        lens.add_(1)
        q, k = K.csa2_qk_norm_rope(xin[:, :Hq], xin[:, Hq:Hq + Hk], pos1, q_weight=wq, k_weight=wk, rope=rope)
        K.csa2_paged_append(cache, k, xin[:, Hq + Hk:], seq1, pos1)
        return K.csa2_paged_decode_attn(q[:B], cache, scale, window=W, sinks=S)

    graph = torch.cuda.CUDAGraph()
    keep = lens.clone()
    with torch.cuda.graph(graph):
        out, lse = step()
    assert torch.equal(lens, keep)
    for s in range(steps):
        for b in range(B):
            xin[b] = x[b][news[b] + s]
        graph.replay()
        for b in range(B):
            check(out[b:b + 1], lse[b:b + 1], b, news[b] + s, f"step {s} of {b}")
    assert lens.tolist() == total


def test_calls_on_a_side_stream():
    """With `stream` every call runs there, its results and scratch allocated for it."""
    cache, host = P.make_cache("bf16", [3000, 700], 64, 1, 128, shared=True, seed=91)
    q = P.rng_normal(92, 2, 16, 128)
    want = K.csa2_paged_decode_attn(q, cache, 0.1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = []
    for _ in range(4):
        got.append(K.csa2_paged_decode_attn(q, cache, 0.1, stream=s))
        junk = torch.full((1 << 20,), float("nan"), device="cuda")   # the default stream reuses what it owns
        del junk
    s.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_rounds_every_step(inter):
    """The rotation's f32 steps one by one (products, then their sum, then the 16-bit type), as
    the header states them: the same bits as separate torch operations."""
    T, H, D, half = 500, 8, 128, 64
    x = P.rng_normal(121, T, H, D, dt=torch.float16)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 1931
    f = _freq(half)
    got = K.csa2_qk_norm_rope(x, None, pos, rope=K.Rope(f, interleaved=inter))[0]
    angle = pos.double()[:, None, None] * f.double()
    cos, sin = angle.cos().float(), angle.sin().float()
    y = x.float()
    a, b = (y[..., 0::2], y[..., 1::2]) if inter else (y[..., :half], y[..., half:])
    a, b = a * cos - b * sin, b * cos + a * sin
    want = (torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)).half()
    # the angle's sine may round to its neighbour (64-bit sines differ in their last bit)
    assert (got != want).sum().item() <= 2


def test_two_graphs_interleaved_and_two_streams():
    """Split decode calls captured in two graphs, replayed in turn and on two streams at once:
    each call has scratch of its own."""
    caches = [P.make_cache("bf16", [4000, 900], 64, 1, 128, shared=True, seed=130 + i)[0] for i in range(2)]
    qs = [P.rng_normal(135 + i, 2, 16, 128) for i in range(2)]
    want = [K.csa2_paged_decode_attn(q, c, 0.1) for q, c in zip(qs, caches)]
    graphs, outs = [], []
    for q, c in zip(qs, caches):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(K.csa2_paged_decode_attn(q, c, 0.1))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for o, l in outs:
            o.zero_(), l.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(outs, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


@pytest.mark.parametrize("G,D", [(4, 64), (8, 128), (3, 128)])
def test_window_rows_that_see_nothing(G, D):
    """Many row tiles without a key: zeros, whatever q holds (it lands late in shared memory)."""
    B, n = 64, 96
    k = torch.zeros(4, 16, 2, D, dtype=torch.bfloat16, device="cuda")
    cache = K.PagedKv(k, torch.zeros(B, 2, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda"),
                      v=torch.ones_like(k))
    cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    q = torch.ones(B * n, 2 * G, D, dtype=torch.bfloat16, device="cuda")
    for _ in range(5):
        out, lse = K.csa2_paged_window_attn(q, cu, cache, 1.0)
        assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


def test_empty_batches_do_nothing():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    cache = K.PagedKv(k, torch.zeros(0, 3, dtype=torch.int32, device="cuda"), none, v=torch.zeros_like(k))
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert K.csa2_paged_decode_attn(q, cache, 1.0)[0].shape == (0, 4, 64)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert K.csa2_paged_window_attn(q, one, cache, 1.0)[1].shape == (0, 4)
    K.csa2_paged_append(cache, q[:, :2], q[:, :2], none, none)
    assert K.csa2_qk_norm_rope(q, q[:, :2])[1].shape == (0, 2, 64)
    # no pages at all: every sequence is empty
    bare = K.PagedKv(k[:0], torch.zeros(3, 0, dtype=torch.int32, device="cuda"),
                     torch.zeros(3, dtype=torch.int32, device="cuda"), v=k[:0])
    out, lse = K.csa2_paged_decode_attn(torch.ones(3, 4, 64, dtype=torch.bfloat16, device="cuda"), bare, 1.0)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
    out, lse = K.csa2_paged_window_attn(torch.ones(3, 4, 64, dtype=torch.bfloat16, device="cuda"),
                                        torch.arange(4, dtype=torch.int32, device="cuda"), bare, 1.0)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
