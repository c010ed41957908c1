"""Paged-cache calls in forms that the operator-by-operator tests leave out: tables wider than
the sequences, f16 weights far below a row's largest, scores of any size, pages longer than a
tile of tokens, offsets past 32 bits, and a side stream for every call.  Bounds follow
paged_util; _check_relative leaves out its allowance for the fixed step of small f16 weights."""
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


def _check_relative(out, lse, want, q, keys, scale, dt, tokens, what=""):
    """paged_util's bound with every weight rounded by half a step relative to itself; 2^-25 is the
    half step of an f16 output below 2^-14."""
    o, s, mag = want
    u = P.half_step(dt)
    ka = np.abs(keys).max(0).repeat(q.shape[1] // keys.shape[1], 0)
    ds = (q.shape[2] + 8) * 2.0 ** -24 * scale * (np.abs(q) * ka[None]).sum(-1)
    rel = 2 * ds + 2.0 ** -20 + (tokens / 8 + 64) * 2.0 ** -23 + u * 1.01
    tol = rel[..., None] * mag + u * np.abs(o) + (2.0 ** -25 if dt == torch.float16 else 0.0)
    err = np.abs(P.f64(out) - o)
    assert np.all(err <= tol), f"{what}: out off by {(err / tol).max():.3g} times its bound"
    ltol = ds + (tokens / 8 + 64) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * np.abs(s)
    assert np.all(np.abs(P.f64(lse) - s) <= ltol), f"{what}: lse"


def _paged(rows, page, seed=0):
    """Rows [n, heads, D] of one sequence as pages in random order, and the table's row."""
    n, heads, D = rows.shape
    need = -(-n // page)
    perm = torch.randperm(need, generator=torch.Generator().manual_seed(seed))
    pages = torch.full((need, page, heads, D), float("nan"), dtype=rows.dtype, device="cuda")
    full = torch.cat([rows, torch.full((need * page - n, heads, D), float("nan"), dtype=rows.dtype, device="cuda")])
    pages[perm.cuda()] = full.view(need, page, heads, D)
    return pages, perm.int().cuda()


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


# ------------------------------------------------------------------ f16 weights

def _dominated(D, heads, G, page, L, T, seed):
    """A cache whose first token outweighs each other one by 2^16 to 2^20, by query head, and has a
    zero value row; every other token of a head weighs the same, so that a rounding of the weights
    does not average out."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    Hq, scale, c = heads * G, D ** -0.5, 16.0
    w = (torch.randn(1, heads, D, generator=g, device="cuda") * 0.3).half()
    w[..., 0] = 0
    k = w.repeat(L, 1, 1)
    k[0, :, 0] = c
    v = (torch.rand(L, heads, D, generator=g, device="cuda") + 0.5).half()
    v[0] = 0
    q = (torch.randn(T, Hq, D, generator=g, device="cuda") * 0.5).half()
    order = torch.linspace(16.2, 19.9, Hq, device="cuda") + torch.rand(T, Hq, generator=g, device="cuda") * 0.1
    q[..., 0] = (order / (scale * c * np.log2(np.e))).half()
    kp, table = _paged(k, page, seed)
    vp, _ = _paged(v, page, seed)
    cache = K.PagedKv(kp, table[None], _ints(L), v=vp)
    return cache, q, P.f64(k), P.f64(v), scale


@pytest.mark.parametrize("D,G,page", [(64, 8, 16), (128, 16, 16), (256, 3, 32), (512, 64, 64), (512, 16, 16), (512, 5, 4)])
@pytest.mark.parametrize("chunk", [0, 256])
def test_decode_f16_weights_far_below_the_largest(D, G, page, chunk):
    cache, q, k, v, scale = _dominated(D, 2, G, page, 1000, 1, 17)
    out, lse = K.csa2_paged_decode_attn(q, cache, scale, chunk=chunk)
    want = O.causal_attn(P.f64(q), [999], k, v, scale)
    _check_relative(out, lse, want, P.f64(q), k, scale, torch.float16, 1000)


@pytest.mark.parametrize("D,G,page", [(64, 8, 16), (128, 4, 64), (128, 3, 4), (256, 2, 16), (256, 40, 16), (512, 4, 16),
                                      (512, 64, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (600, 1)])
def test_window_f16_weights_far_below_the_largest(D, G, page, window, sinks):
    cache, q, k, v, scale = _dominated(D, 2, G, page, 1000, 20, 18)
    out, lse = K.csa2_paged_window_attn(q, _ints(0, 20), cache, scale, window=window, sinks=sinks)
    want = O.causal_attn(P.f64(q), np.arange(980, 1000), k, v, scale, window, sinks)
    _check_relative(out, lse, want, P.f64(q), k, scale, torch.float16, 1000)


# ------------------------------------------------------------------ scores of any size

@pytest.mark.parametrize("low,offset", [(float("-inf"), 300.0), (-65504.0, 0.0)])
@pytest.mark.parametrize("D,G,page", [(64, 8, 16), (128, 4, 64), (256, 2, 16), (256, 40, 16), (512, 4, 16), (512, 16, 64),
                                      (512, 64, 64), (512, 3, 4)])
@pytest.mark.parametrize("prompt,chunk", [(True, 0), (False, 0), (False, 768)])
def test_first_tokens_that_weigh_nothing(D, G, page, low, offset, prompt, chunk):
    """The first 140 tokens score -inf (the rest about -300) or 10^8 below the rest: the answer is the
    softmax over the rest, to the precision of the rest's scores."""
    L, T, scale, dt = 700, 12 if prompt else 1, D ** -0.5, torch.float16
    g = torch.Generator(device="cuda").manual_seed(23)
    k = torch.randn(L, 1, D, generator=g, device="cuda")
    k[..., 0] = 0
    k[..., 1] = -8.0
    k[:140, :, 0] = low
    k = k.half()
    v = torch.randn(L, 1, D, generator=g, device="cuda").half()
    q = torch.randn(T, G, D, generator=g, device="cuda") * 0.5
    q[..., 0] = 30000.0
    q[..., 1] = offset / (8.0 * scale)
    q = q.half()
    kp, table = _paged(k, page)
    vp, _ = _paged(v, page)
    cache = K.PagedKv(kp, table[None], _ints(L), v=vp)
    if prompt:
        out, lse = K.csa2_paged_window_attn(q, _ints(0, T), cache, scale)
    else:
        out, lse = K.csa2_paged_decode_attn(q, cache, scale, chunk=chunk)
    qh, kh = P.f64(q), P.f64(k[140:])
    want = O.causal_attn(qh, np.arange(L - 140 - T, L - 140), kh, P.f64(v[140:]), scale)
    _check_relative(out, lse, want, qh, kh, scale, dt, L)


@pytest.mark.parametrize("size", [0, 20, 22, 23, 24, 26])
@pytest.mark.parametrize("kind", ["bf16", "f16", "fp4"])
@pytest.mark.parametrize("D,G,page", [(64, 8, 16), (128, 3, 64), (256, 2, 16), (256, 40, 16), (512, 4, 16), (512, 64, 64),
                                      (512, 2, 4)])
def test_equal_scores_of_any_size(kind, D, G, page, size):
    """Tokens with the same key weigh the same, however large its score (1.37 * 2^size in base 2, both
    signs): the answer is the mean of the values.  Every token's score is one and the same number, so
    its error leaves the weights alone and shows in lse only."""
    n, T, scale = 700, 9, D ** -0.5
    top = 2688.0 if kind == "fp4" else 32768.0
    dt = P.DT[kind]
    k = torch.zeros(n, 1, D, device="cuda")
    k[..., 0] = top
    v = P.rng_normal(27, n, 1, D, dt=dt) + 1
    kp, table = _paged(k.to(dt), page)
    vp, _ = _paged(v, page)
    sc = [None, None]
    if kind == "fp4":
        kp, vp = torch.nan_to_num(kp), torch.nan_to_num(vp)
        (kp, sc[0]), (vp, sc[1]) = K.csa2_fp4_pack(kp), K.csa2_fp4_pack(vp)
        v = K.csa2_fp4_unpack(vp, sc[1])[table.long()].flatten(0, 1)[:n]
    cache = K.PagedKv(kp, table[None], _ints(n), v=vp, k_scales=sc[0], v_scales=sc[1])
    q = torch.zeros(T, G, D, device="cuda")
    q[..., 0] = 1.37 * 2.0 ** size / (scale * top * np.log2(np.e))
    q[:, ::2] *= -1
    q = q.to(dt)
    u, vh = P.half_step(dt), P.f64(v)[:, 0]
    score = P.f64(q)[..., 0] * top * scale
    def check(out, lse, at, seen):
        mean, mag = vh[:seen].mean(0), np.abs(vh[:seen]).mean(0)
        tol = (2.0 ** -20 + (n / 8 + 64) * 2.0 ** -23 + u * 1.01) * mag + u * np.abs(mean) + 2.0 ** -25
        assert np.all(np.abs(P.f64(out) - mean) <= tol), f"token {at}"
        want = score[at] + np.log(seen)
        assert np.all(np.abs(P.f64(lse) - want) <= 2.0 ** -15 + 2.0 ** -21 * np.abs(want)), f"token {at}: lse"

    for chunk in (0, 384):
        out, lse = K.csa2_paged_decode_attn(q[:1], cache, scale, chunk=chunk)
        check(out[0], lse[0], 0, n)
    out, lse = K.csa2_paged_window_attn(q, _ints(0, T), cache, scale)
    for t in range(T):
        check(out[t], lse[t], t, n - T + 1 + t)


# ------------------------------------------------------------------ long pages

def _long_pages(kind, D, heads, G, shared, page, window, sinks, lens, news):
    cache, host = P.make_cache(kind, lens, page, heads, D, shared=shared, seed=33, spare=0)
    q = P.rng_normal(34, len(lens), heads * G, D, dt=cache.dtype)
    out, lse = K.csa2_paged_decode_attn(q, cache, D ** -0.5, window=window, sinks=sinks)
    qh = P.f64(q)
    for b, n in enumerate(lens):
        want = O.causal_attn(qh[b:b + 1], [n - 1], *host[b], D ** -0.5, window, sinks)
        P.check_attn(out[b:b + 1], lse[b:b + 1], want, qh[b:b + 1], host[b][0], D ** -0.5, cache.dtype, n, f"decode {b}")
    q = P.rng_normal(35, sum(news), heads * G, D, dt=cache.dtype)
    cu = np.concatenate([[0], np.cumsum(news)])
    out, lse = K.csa2_paged_window_attn(q, _ints(*cu), cache, D ** -0.5, window=window, sinks=sinks)
    qh = P.f64(q)
    for b, n in enumerate(lens):
        sl = slice(cu[b], cu[b + 1])
        want = O.causal_attn(qh[sl], np.arange(n - news[b], n), *host[b], D ** -0.5, window, sinks)
        P.check_attn(out[sl], lse[sl], want, qh[sl], host[b][0], D ** -0.5, cache.dtype, n, f"prompt {b}")


@pytest.mark.parametrize("kind", ["bf16", "f16", "fp4"])
@pytest.mark.parametrize("D,heads,G,shared", [(64, 2, 4, False), (128, 1, 8, True), (256, 1, 33, False), (512, 1, 64, True),
                                              (512, 2, 3, False)])
@pytest.mark.parametrize("page,window,sinks", [(256, 0, 0), (1024, 300, 140)])
def test_pages_longer_than_a_tile(kind, D, heads, G, shared, page, window, sinks):
    _long_pages(kind, D, heads, G, shared, page, window, sinks, [1, 300, 1290], [1, 40, 9])


@pytest.mark.parametrize("D,G", [(64, 4), (512, 64)])
def test_the_longest_pages(D, G):
    _long_pages("bf16", D, 1, G, True, 65536, 0, 0, [700], [50])


@pytest.mark.parametrize("kind", ["bf16", "fp4"])
def test_append_to_pages_longer_than_a_tile(kind):
    page, D, T = 1024, 64, 70
    rows = P.rng_normal(36, T, 2, D)
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    table = _ints(2, 0, 1, 3).view(2, 2)
    w = D // 2 if kind == "fp4" else D
    k = torch.zeros(4, page, 2, w, dtype=torch.uint8 if kind == "fp4" else torch.bfloat16, device="cuda")
    s = torch.zeros(4, page, 2, D // 16, dtype=torch.uint8, device="cuda") if kind == "fp4" else None
    cache = K.PagedKv(k, table, lens, k_scales=s)
    seq = (torch.arange(T, device="cuda") % 2).int()
    pos = (torch.arange(T, device="cuda") // 2 * 37 + 500).int()     # over the page border
    K.csa2_paged_append(cache, rows, None, seq, pos)
    at = table[seq.long(), pos.long() // page].long(), pos.long() % page
    if kind == "fp4":
        codes, scales = K.csa2_fp4_pack(rows)
        assert torch.equal(k[at], codes) and torch.equal(s[at], scales)
        assert int((s != 0).sum()) == int((scales != 0).sum())
    else:
        assert torch.equal(k[at], rows) and int((k != 0).sum()) == int((rows != 0).sum())


# ------------------------------------------------------------------ values that are not finite

@pytest.mark.parametrize("D,heads", [(64, 2), (512, 1)])
def test_append_fp4_of_rows_that_are_not_finite(D, heads):
    """A NaN takes no part in its block's scale, an infinity saturates it: csa2_fp4_pack of the row."""
    T, page = 40, 16
    rows = P.rng_normal(61, T, heads, D)
    g = torch.Generator(device="cuda").manual_seed(62)
    for i, x in enumerate((float("nan"), float("inf"), float("-inf"))):
        at = torch.rand(rows.shape, generator=g, device="cuda") < 0.02
        rows[at] = x
    rows[7] = float("nan")
    rows.view(torch.int16)[8, 0, :16] = -1                           # NaN with the sign and every payload bit
    codes, scales = K.csa2_fp4_pack(rows)
    k = torch.zeros(3, page, heads, D // 2, dtype=torch.uint8, device="cuda")
    s = torch.zeros(3, page, heads, D // 16, dtype=torch.uint8, device="cuda")
    cache = K.PagedKv(k, _ints(2, 0, 1)[None], _ints(0), k_scales=s)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    K.csa2_paged_append(cache, rows, None, torch.zeros_like(pos), pos)
    at = cache.table[0][pos.long() // page].long(), pos.long() % page
    assert torch.equal(s[at], scales) and torch.equal(k[at], codes)


# ------------------------------------------------------------------ offsets past 32 bits

@pytest.mark.parametrize("T,H,ts,hs", [(6, 2, (1 << 29) + 64, 128), (2, 6, 128, (1 << 29) + 64)])
def test_norm_rope_offsets_past_32_bits(T, H, ts, hs):
    """Rows of one CTA that lie more than 2^31 elements apart, token by token or head by head."""
    D = 64
    span = (T - 1) * ts + (H - 1) * hs + D
    assert span > 1 << 31
    buf = torch.empty(span, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((T, H, D), (ts, hs, 1))
    rows = P.rng_normal(41, T, H, D)
    x.copy_(rows)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 5
    w = torch.rand(D, device="cuda") + 0.5
    rope = K.Rope((10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().cuda())
    want = K.csa2_qk_norm_rope(rows, rows, pos, q_weight=w, k_weight=w, rope=rope)
    q, _ = K.csa2_qk_norm_rope(x, rows, pos, q_weight=w, k_weight=w, rope=rope)
    _, k = K.csa2_qk_norm_rope(rows, x, pos, q_weight=w, k_weight=w, rope=rope)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    K.csa2_qk_norm_rope(x, None, pos, q_weight=w, rope=rope, q_out=x)             # in place
    assert torch.equal(x.contiguous(), want[0])


@pytest.mark.parametrize("kind,D,G,page", [("bf16", 512, 64, 64), ("f16", 512, 4, 16), ("bf16", 512, 3, 4), ("bf16", 256, 8, 16),
                                           ("bf16", 128, 8, 16), ("fp4", 128, 4, 64), ("fp4", 512, 20, 64)])
def test_cache_past_32_bits(kind, D, G, page):
    """A pool of more than 2^31 channels (FP4: 2^32 channels, 2^31 bytes of codes) with the sequences in
    its last pages and its first: append, single tokens and a prompt."""
    far = (1 << (32 if kind == "fp4" else 31)) // (page * D)
    n_pages, n, new = far + 40, 130, 9
    dt, need = P.DT[kind], -(-n // page)
    empty = lambda w, t: torch.empty(n_pages, page, 1, w, dtype=t, device="cuda")
    fp4 = kind == "fp4"
    table = torch.stack([torch.arange(n_pages - need, n_pages), torch.arange(need)]).int().cuda()
    cache = K.PagedKv(empty(D // 2 if fp4 else D, torch.uint8 if fp4 else dt), table, _ints(n, n),
                      k_scales=empty(D // 16, torch.uint8) if fp4 else None)
    rows = P.rng_normal(71, 2 * n, 1, D, dt=dt)
    seq = (torch.arange(2 * n, device="cuda") // n).int()
    pos = (torch.arange(2 * n, device="cuda") % n).int()
    K.csa2_paged_append(cache, rows, None, seq, pos)
    kept = K.csa2_fp4_unpack(*K.csa2_fp4_pack(rows)) if fp4 else rows
    host = P.f64(kept).reshape(2, n, 1, D)
    scale = D ** -0.5
    q = P.rng_normal(72, 2, G, D, dt=dt)
    out, lse = K.csa2_paged_decode_attn(q, cache, scale)
    qp = P.rng_normal(73, 2 * new, G, D, dt=dt)
    outp, lsep = K.csa2_paged_window_attn(qp, _ints(0, new, 2 * new), cache, scale)
    for b in range(2):
        h = host[b]
        want = O.causal_attn(P.f64(q[b:b + 1]), [n - 1], h, h, scale)
        P.check_attn(out[b:b + 1], lse[b:b + 1], want, P.f64(q[b:b + 1]), h, scale, dt, n, f"single token {b}")
        sl = slice(b * new, (b + 1) * new)
        want = O.causal_attn(P.f64(qp[sl]), np.arange(n - new, n), h, h, scale)
        P.check_attn(outp[sl], lsep[sl], want, P.f64(qp[sl]), h, scale, dt, n, f"prompt {b}")


# ------------------------------------------------------------------ streams

def test_every_call_on_a_side_stream():
    """`stream` with every other argument away from its default: the same results as without."""
    T, Hq, Hk, D = 120, 8, 2, 128
    x = P.rng_normal(51, T, Hq + 2 * Hk, D, dt=torch.float16)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    seq = (pos >= 70).int()
    at = torch.where(seq == 1, pos - 70, pos)
    w = [torch.rand(D, device="cuda") + 0.5 for _ in range(2)]
    rope = K.Rope((10000.0 ** (-torch.arange(16, dtype=torch.float64) / 16)).float().cuda(), offset=64, interleaved=True)
    side = torch.cuda.Stream()

    def layer(s):
        kv = [torch.zeros(10, 16, Hk, D, dtype=torch.float16, device="cuda") for _ in range(2)]
        cache = K.PagedKv(kv[0], torch.arange(10, dtype=torch.int32, device="cuda").flip(0).view(2, 5).contiguous(),
                          _ints(70, 50), v=kv[1])
        cu, outs = _ints(0, 70, 120), (torch.zeros(T, Hq, D, dtype=torch.float16, device="cuda"), torch.zeros(T, Hq, device="cuda"))
        qk = torch.zeros(T, Hq, D, dtype=torch.float16, device="cuda"), torch.zeros(T, Hk, D, dtype=torch.float16, device="cuda")
        torch.cuda.synchronize()
        q, k = K.csa2_qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hk], at, q_weight=w[0], k_weight=w[1], eps=0.25, rope=rope,
                                   q_out=qk[0], k_out=qk[1], stream=s)
        assert q is qk[0] and k is qk[1]
        K.csa2_paged_append(cache, k, x[:, Hq + Hk:], seq, at, rope=rope, stream=s)
        a = K.csa2_paged_window_attn(q, cu, cache, 0.07, window=30, sinks=3, out=outs[0], lse=outs[1], stream=s)
        assert a[0] is outs[0] and a[1] is outs[1]
        d = K.csa2_paged_decode_attn(q[:2], cache, 0.07, window=30, sinks=3, chunk=64, stream=s)
        torch.cuda.synchronize()
        return q, k, *kv, *a, *d

    for want, got in zip(layer(None), layer(side)):
        assert torch.equal(want, got)
