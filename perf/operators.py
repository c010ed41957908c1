"""What the paged-cache operators are measured on.

Four operators of a serving path, in the order a layer calls them: norms and
position rotation of queries and keys, appending keys and values to a paged
cache, attention of one new token per sequence over that cache, and attention
of a prompt chunk with a sliding window and sinks.  `run` computes one call in
plain torch operations in 32 bits (`own` false) or through the library.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "fp4": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of the smallest configuration (16 query heads over one shared 128-wide row): latency
        dict(name="norm_rope_one_token", op="norm_rope", type="bf16", T=1, Hq=16, Hk=1, D=128, rot=128,
             tail=False, inter=False, fused=True, far=8192),
        # a prompt chunk with grouped heads, q and k slices of one projection's output
        dict(name="norm_rope_prompt", op="norm_rope", type="bf16", T=8192, Hq=64, Hk=8, D=128, rot=128,
             tail=False, inter=False, fused=True, far=65536),
        # the 4096-token prefill chunk's latent heads, only the last 64 channels rotated, far positions
        dict(name="norm_rope_latent_tail", op="norm_rope", type="f16", T=4096, Hq=64, Hk=1, D=512, rot=64,
             tail=True, inter=True, fused=False, far=1048576),
        # one new token of 64 sequences, padded to a graph's batch of 80
        dict(name="append_decode_batch", op="append", type="bf16", T=64, pad=16, B=64, Hkv=8, D=128, rot=128,
             tail=False, inter=False, page=64, shared=False, room=960),
        # a ragged prompt batch into the cache, the rotation on the way
        dict(name="append_prompt", op="append", type="f16", T=8191, pad=0, B=5, Hkv=8, D=128, rot=64,
             tail=False, inter=False, page=16, shared=False, room=4096),
        # the prefill chunk's shared 512-wide rows, packed to FP4 on the way and read back
        dict(name="append_latent_fp4", op="append", type="fp4", T=4096, pad=0, B=1, Hkv=1, D=512, rot=64,
             tail=True, inter=True, page=64, shared=True, room=4096),
        # one sequence of 8192 tokens, 16 heads over one shared 128-wide row: latency
        dict(name="decode_one_8k", op="decode", type="bf16", B=1, L=8192, ragged=False, Hq=16, Hkv=1, D=128, page=64,
             shared=True, window=0, sinks=0),
        # grouped heads, 64 sequences of very different lengths, one of them empty
        dict(name="decode_grouped_ragged", op="decode", type="bf16", B=64, L=16384, ragged=True, Hq=64, Hkv=8, D=128,
             page=16, shared=False, window=0, sinks=0),
        # 32 sequences of 64K tokens, 64 heads over a shared 512-wide row
        dict(name="decode_latent_64k", op="decode", type="bf16", B=32, L=65536, ragged=False, Hq=64, Hkv=1, D=512,
             page=64, shared=True, window=0, sinks=0),
        # 64 sequences in FP4, a window with sinks over a long cache
        dict(name="decode_fp4_window", op="decode", type="fp4", B=64, L=32767, ragged=True, Hq=32, Hkv=4, D=128,
             page=64, shared=False, window=8192, sinks=4),
        # short chunks of seven sequences behind cached tokens, narrow heads
        dict(name="window_chunks", op="window", type="f16", B=7, T=331, past=900, Hq=16, Hkv=2, D=64, page=16,
             shared=False, window=256, sinks=4),
        # a whole prompt, window of 2048 with sinks, grouped heads
        dict(name="window_prompt", op="window", type="bf16", B=2, T=8192, past=0, Hq=32, Hkv=4, D=128, page=64,
             shared=False, window=2048, sinks=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "decode", "window"])
    D = rng.choice([64, 128, 128, 256, 512])
    kind = rng.choice(["bf16", "bf16", "f16", "fp4"])
    page = rng.choice([1, 16, 32, 64, 128])
    shared = rng.random() < 0.4
    if op == "norm_rope":
        D = rng.choice([64, 80, 96, 128, 256, 512])
        Hk = rng.choice([1, 2, 5, 8])
        Hq = Hk * rng.choice([1, 4, 7, 8])
        T = _log(rng, 1, max(2, (8192 * 72 * 128) // ((Hq + Hk) * D)))
        return dict(op=op, type=rng.choice(["bf16", "f16"]), T=T, Hq=Hq, Hk=Hk, D=D, rot=rng.choice([16, 32, D // 16 * 16]),
                    tail=rng.random() < 0.5, inter=rng.random() < 0.5, fused=rng.random() < 0.5, far=_log(rng, 100, 1 << 20))
    if op == "append":
        Hkv = rng.choice([1, 2, 3, 8])
        T = _log(rng, 1, min(16384, 8192 * 1024 // (Hkv * D)))
        return dict(op=op, type=kind, T=T, pad=rng.choice([0, 0, 5, 33]), B=rng.randint(1, min(T, 64)), Hkv=Hkv, D=D,
                    rot=rng.choice([32, 64]), tail=rng.random() < 0.5, inter=rng.random() < 0.5, page=page, shared=shared,
                    room=_log(rng, 1, 2000))
    window, sinks = rng.choice([(0, 0), (0, 0), (128, 0), (1000, 4), (4096, 64), (_log(rng, 1, 9000), 5)])
    Hkv = rng.choice([1, 1, 2, 8])
    G = rng.choice([1, 3, 8, 16, 64 // Hkv])
    if op == "decode":
        B = _log(rng, 1, 128)
        most = 32 * 65536 * 512 // (B * Hkv * D * (1 if shared else 2))
        return dict(op=op, type=kind, B=B, L=_log(rng, 1, min(most, 131072)), ragged=rng.random() < 0.6, Hq=Hkv * G,
                    Hkv=Hkv, D=D, page=page, shared=shared, window=window, sinks=sinks)
    B = rng.randint(1, 9)
    past = rng.choice([0, 0, _log(rng, 1, 2000)])
    most = int(math.sqrt(2.0e8 / (Hkv * G)))          # the plain form holds every head's whole score matrix
    return dict(op=op, type=kind, B=B, T=max(B, _log(rng, B, max(B, min(4096, most)))), past=min(past, most), Hq=Hkv * G,
                Hkv=Hkv, D=D, page=page, shared=shared, window=window, sinks=sinks)


def _lens(case):
    """Decode: cached tokens of each sequence (the last one empty when ragged)."""
    B, L = case["B"], case["L"]
    if not case["ragged"]:
        return [L] * B
    r = random.Random(B * 1000003 + L)
    got = [max(1, int(L * r.random() ** 2)) for _ in range(B)]
    got[0] = L
    if B > 2:
        got[-1] = 0
    return got


def _chunks(case):
    """Ragged split of the T new tokens over the B sequences."""
    B, T = case["B"], case["T"]
    r = random.Random(T * 1000003 + B)
    w = [0.2 + r.random() for _ in range(B)]
    got = [1 + int((T - B) * x / sum(w)) for x in w]
    got[0] += T - sum(got)
    return got


def _rope(case):
    rot = case["rot"]
    return (case["D"] - rot if case["tail"] else 0), rot


def _window_span(case):
    """Per sequence: new tokens, cached tokens after them."""
    n = _chunks(case)
    return n, [x + case["past"] * (i % 3) // 2 for i, x in enumerate(n)]


# ------------------------------------------------------------------ inputs

def _quantise(x):
    """E2M1 codes (0..15) and E4M3 scale codes of x [..., D] in blocks of 16 channels."""
    b = x.float().unflatten(-1, (-1, 16))
    scale = (b.abs().amax(-1).double() / 6).clamp(max=448).float().to(torch.float8_e4m3fn)
    s = scale.float().unsqueeze(-1)
    a = torch.where(s > 0, b.abs() / s, torch.zeros_like(b))
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    even = torch.tensor([0, 1, 0, 1, 0, 1, 0], device=x.device, dtype=torch.bool)
    passed = (a.unsqueeze(-1) > mids) | ((a.unsqueeze(-1) == mids) & even)
    code = passed.sum(-1) + 8 * torch.signbit(b).long()
    return code.flatten(-2), scale


def _values(code, scale):
    """The bf16 values that E2M1 codes and E4M3 scales stand for."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=code.device)
    v = table[code].unflatten(-1, (-1, 16)) * scale.float().unsqueeze(-1)
    return v.flatten(-2).to(torch.bfloat16)


def _cache(case, g, lens, fill):
    """Paged cache tensors, its block table (a random permutation of the pages) and lengths."""
    B, page, H, D = len(lens), case["page"], case["Hkv"], case["D"]
    width = max(1, max(-(-n // page) for n in lens))
    pages = B * width + 3
    table = torch.randperm(pages, generator=g, device="cuda")[: B * width].view(B, width).int()
    st = {"table": table, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    for name in ("k",) if case["shared"] else ("k", "v"):
        if case["type"] == "fp4":
            codes = torch.zeros(pages, page, H, D // 2, dtype=torch.uint8, device="cuda")
            scales = torch.zeros(pages, page, H, D // 16, dtype=torch.uint8, device="cuda")
            if fill:
                step = max(1, (1 << 24) // (page * H * D))
                for i in range(0, pages, step):
                    n = min(step, pages - i)
                    x = torch.randn(n, page, H, D, generator=g, device="cuda")
                    c, s = _quantise(x)
                    codes[i:i + n] = (c[..., 0::2] + 16 * c[..., 1::2]).to(torch.uint8)
                    scales[i:i + n] = s.view(torch.uint8)
            st[name], st[name + "_scales"] = codes, scales
        else:
            st[name] = torch.zeros(pages, page, H, D, dtype=TYPES[case["type"]], device="cuda")
            if fill:
                st[name].normal_(generator=g)
    if case["shared"]:
        st["v"], st["v_scales"] = st["k"], st.get("k_scales")
    return st


def _handle(st, case):
    """The library's description of the cache, which a program keeps beside its tensors."""
    import kv_cache_csa2_b200 as K
    st["cache"] = K.PagedKv(st["k"], st["table"], st["lens"], v=None if case["shared"] else st["v"],
                            k_scales=st.get("k_scales"), v_scales=None if case["shared"] else st.get("v_scales"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    op, D = case["op"], case["D"]
    dt = TYPES[case["type"]]
    st = {"case": dict(case)}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)

    if op in ("norm_rope", "append"):
        T = case["T"]
        offset, rot = _rope(case)
        st["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)).float()
        if op == "norm_rope":
            Hq, Hk = case["Hq"], case["Hk"]
            if case["fused"]:
                qkv = normal(T, Hq + 2 * Hk, D)
                st["q"], st["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
            else:
                st["q"], st["k"] = normal(T, Hq, D), normal(T, Hk, D)
            st["q_weight"] = 1 + 0.2 * torch.randn(D, generator=g, device="cuda")
            st["k_weight"] = 1 + 0.2 * torch.randn(D, generator=g, device="cuda")
            st["positions"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
        else:
            n = _chunks(case)
            old = [7919 * (i + 1) % (case["room"] + 1) for i in range(len(n))]      # tokens cached before
            st.update(_cache(case, g, [a + b for a, b in zip(old, n)], False))
            st["seq"] = torch.cat([torch.repeat_interleave(torch.arange(len(n)), torch.tensor(n)),
                                   torch.full((case["pad"],), -1)]).int().cuda()
            st["pos"] = torch.cat([torch.arange(a, a + b) for a, b in zip(old, n)] +
                                  [torch.zeros(case["pad"], dtype=torch.int64)]).int().cuda()
            st["new_k"] = normal(T + case["pad"], case["Hkv"], D)
            st["new_v"] = None if case["shared"] else normal(T + case["pad"], case["Hkv"], D)
    elif op == "decode":
        st.update(_cache(case, g, _lens(case), True))
        st["q"] = normal(case["B"], case["Hq"], D)
    else:
        n, lens = _window_span(case)
        st.update(_cache(case, g, lens, True))
        st["q"] = normal(case["T"], case["Hq"], D)
        st["cu_q"] = torch.tensor([0] + n, device="cuda").cumsum(0).int()
        st["most_q"], st["n"] = max(n), n
    if own:
        if op in ("norm_rope", "append"):
            import kv_cache_csa2_b200 as K
            st["rope"] = K.Rope(st["inv_freq"], offset=_rope(case)[0], interleaved=case["inter"])
        if op != "norm_rope":
            _handle(st, case)
    return st


# ------------------------------------------------------------------ one pass

def _rotate(x, positions, inv_freq, offset, inter):
    """x f32 [T, H, D]; the angles in 64 bits (far positions), their sines rounded to 32."""
    angle = positions.double()[:, None, None] * inv_freq.double()
    cos, sin = angle.cos().float(), angle.sin().float()
    half = inv_freq.numel()
    mid = x[..., offset:offset + 2 * half]
    a, b = (mid[..., 0::2], mid[..., 1::2]) if inter else (mid[..., :half], mid[..., half:])
    a, b = a * cos - b * sin, b * cos + a * sin
    mid = torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)
    return torch.cat((x[..., :offset], mid, x[..., offset + 2 * half:]), -1)


def _norm(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _plain_rows(st, name, count):
    """The first `count` cached rows of every sequence in 32 bits, [B, count, Hkv, D], zero past its end."""
    pos = torch.arange(count, device="cuda")
    page = st["k"].shape[1]
    table = st["table"].long()
    pages = table[:, (pos // page).clamp(max=table.shape[1] - 1)]
    rows = st[name][pages, pos % page]
    if st["case"]["type"] == "fp4":
        code = torch.stack((rows & 15, rows >> 4), -1).flatten(-2).long()
        rows = _values(code, st[name + "_scales"][pages, pos % page].view(torch.float8_e4m3fn))
    rows = rows.float()
    return rows * (pos < st["lens"][:, None])[:, :, None, None]


def _plain_softmax(s, visible):
    """Softmax weights and log sum over the last axis; a row that sees nothing gives 0 and -inf."""
    s = s.masked_fill(~visible, float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m > float("-inf"), m, torch.zeros_like(m)))
    total = p.sum(-1, keepdim=True)
    return p / total.clamp(min=1e-30), (m + total.log()).squeeze(-1)


def _plain_decode(st):
    c = st["case"]
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    k = _plain_rows(st, "k", c["L"])
    v = k if c["shared"] else _plain_rows(st, "v", c["L"])
    q = st["q"].float().view(B, Hkv, Hq // Hkv, D)
    s = torch.einsum("bhgd,blhd->bhgl", q, k) * D ** -0.5
    pos, n = torch.arange(c["L"], device="cuda"), st["lens"].long()[:, None]
    visible = pos < n
    if c["window"]:
        visible = visible & ((pos >= n - c["window"]) | (pos < c["sinks"]))
    p, lse = _plain_softmax(s, visible[:, None, None])
    out = torch.einsum("bhgl,blhd->bhgd", p, v).reshape(B, Hq, D)
    return out.to(st["q"].dtype), lse.view(B, Hq)


def _plain_window(st):
    c = st["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    n, lens = _window_span(c)
    B, most, L = c["B"], max(n), max(lens)
    k = _plain_rows(st, "k", L)
    v = k if c["shared"] else _plain_rows(st, "v", L)
    cu, count = st["cu_q"].long()[:-1], st["cu_q"].long().diff()
    i = torch.arange(most, device="cuda")
    rows = (cu[:, None] + i).clamp(max=c["T"] - 1)
    q = st["q"][rows].float().view(B, most, Hkv, Hq // Hkv, D)
    s = torch.einsum("bthgd,blhd->bhgtl", q, k) * D ** -0.5
    at = (st["lens"].long() - count)[:, None] + i                       # the queries' positions
    pos = torch.arange(L, device="cuda")
    visible = pos <= at[..., None]
    if c["window"]:
        visible = visible & ((pos > at[..., None] - c["window"]) | (pos < c["sinks"]))
    p, lse = _plain_softmax(s, visible[:, None, None])
    del s
    out = torch.einsum("bhgtl,blhd->bthgd", p, v).reshape(B * most, Hq, D)
    seq = torch.bucketize(torch.arange(c["T"], device="cuda"), st["cu_q"].long()[1:], right=True)
    back = seq * most + torch.arange(c["T"], device="cuda") - cu[seq]   # each query's place in the padded batch
    return out[back].to(st["q"].dtype), lse.permute(0, 3, 1, 2).reshape(B * most, Hq)[back]


def _plain_append(st):
    c = st["case"]
    T, page = c["T"], c["page"]
    offset = _rope(c)[0]
    pos, seq = st["pos"][:T].long(), st["seq"][:T].long()
    pages, slots = st["table"][seq, pos // page].long(), pos % page
    k = _rotate(st["new_k"][:T].float(), st["pos"][:T], st["inv_freq"], offset, c["inter"]).to(st["new_k"].dtype)
    got = []
    for name, x in (("k", k),) if c["shared"] else (("k", k), ("v", st["new_v"][:T])):
        if c["type"] == "fp4":
            code, scale = _quantise(x)
            whole = torch.zeros(*st[name].shape[:-1], c["D"], dtype=torch.bfloat16, device="cuda")
            whole[pages, slots] = _values(code, scale)
            got.append(whole)
        else:
            st[name][pages, slots] = x
            got.append(st[name])
    return got


def run(state):
    st, c = state, state["case"]
    op = c["op"]
    if own:
        import kv_cache_csa2_b200 as K
        if op == "norm_rope":
            return K.csa2_qk_norm_rope(st["q"], st["k"], st["positions"], q_weight=st["q_weight"],
                                       k_weight=st["k_weight"], eps=EPS, rope=st["rope"])
        if op == "append":
            K.csa2_paged_append(st["cache"], st["new_k"], st["new_v"], st["seq"], st["pos"], rope=st["rope"])
            names = ("k",) if c["shared"] else ("k", "v")
            if c["type"] == "fp4":
                return [K.csa2_fp4_unpack(st[x], st[x + "_scales"]) for x in names]
            return [st[x] for x in names]
        if op == "decode":
            return K.csa2_paged_decode_attn(st["q"], st["cache"], c["D"] ** -0.5, window=c["window"], sinks=c["sinks"])
        return K.csa2_paged_window_attn(st["q"], st["cu_q"], st["cache"], c["D"] ** -0.5, window=c["window"],
                                        sinks=c["sinks"])
    if op == "norm_rope":
        offset = _rope(c)[0]
        return tuple(_rotate(_norm(st[x].float(), st[x + "_weight"]), st["positions"], st["inv_freq"], offset,
                             c["inter"]).to(st[x].dtype) for x in ("q", "k"))
    if op == "append":
        return _plain_append(st)
    return _plain_decode(st) if op == "decode" else _plain_window(st)


# ------------------------------------------------------------------ what a pass cannot do without

def _row_bytes(case):
    return case["D"] * 9 // 16 if case["type"] == "fp4" else 2 * case["D"]


def work(case):
    D, op = case["D"], case["op"]
    if op == "norm_rope":
        n = case["T"] * (case["Hq"] + case["Hk"]) * D
        return {"bytes": 4 * n + 4 * case["T"] + 8 * D, "flops": 8 * n}
    rows = 1 if case["shared"] else 2
    if op == "append":
        n = case["T"] * case["Hkv"] * rows
        return {"bytes": n * (2 * D + _row_bytes(case)) + 8 * case["T"], "flops": 3 * case["T"] * case["Hkv"] * case["rot"]}
    W, S = case["window"], case["sinks"]
    if op == "decode":
        lens = _lens(case)
        seen = sum(min(n, W) + min(S, max(0, n - W)) if W else n for n in lens)
        held, queries, pairs = seen, case["B"], seen
    else:
        n, lens = _window_span(case)
        pairs = held = 0
        for new, total in zip(n, lens):
            first = total - new                       # position of the first new token
            for p in range(first, total):
                pairs += min(p + 1, W) + min(S, max(0, p + 1 - W)) if W else p + 1
            lo = max(0, first + 1 - W) if W else 0
            held += total - lo + min(S, lo)
        queries = case["T"]
    io = queries * case["Hq"] * (4 * D + 4)
    return {"bytes": held * case["Hkv"] * rows * _row_bytes(case) + io, "flops": 4 * case["Hq"] * D * pairs}


# ------------------------------------------------------------------ the definition, in 64 bits

def _exact_rotation(x, positions, case, inv_freq):
    """Each rotated pair as a complex number times e^(i angle)."""
    offset, rot = _rope(case)
    y = x.clone()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device).expand(x.shape[0], 1, rot // 2),
                       positions.double().view(-1, 1, 1) * inv_freq.double().view(1, 1, -1))
    i = torch.arange(rot // 2, device=x.device)
    first = offset + (2 * i if case["inter"] else i)
    second = first + 1 if case["inter"] else first + rot // 2
    z = torch.complex(x[..., first], x[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_fp4(x):
    """x (values of 16-bit floats) through FP4: nearest E2M1 multiple of the nearest E4M3 scale, as values."""
    grid = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    scales = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()

    def nearest(v, points):                           # ties to the even index
        hi = torch.searchsorted(points, v.contiguous()).clamp(1, len(points) - 1)
        lo = hi - 1
        d = (v - points[lo]) - (points[hi] - v)
        up = (d > 0) | ((d == 0) & (hi % 2 == 0))
        return torch.where(up, hi, lo)

    b = x.unflatten(-1, (-1, 16))
    s = scales[nearest(b.abs().amax(-1) / 6, scales)].unsqueeze(-1)
    v = grid[nearest(torch.where(s > 0, b.abs() / s.clamp(min=1e-300), torch.zeros_like(b)), grid)] * s
    return torch.copysign(v, b).flatten(-2)


def _exact_sequence(st, case, b, n):
    """Keys and values [n, Hkv, D] of sequence b in 64 bits, read page by page."""
    page = case["page"]
    pages = st["table"][b, : -(-n // page)].long()
    got = []
    for name in ("k", "v"):
        rows = st[name][pages].flatten(0, 1)[:n]
        if case["type"] == "fp4":
            scale = st[name + "_scales"][pages].flatten(0, 1)[:n].view(torch.float8_e4m3fn).double()
            grid = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
            pair = torch.stack((rows % 16, rows // 16), -1).flatten(-2).long()
            value = grid[pair % 8] * torch.where(pair >= 8, -1.0, 1.0).double()
            rows = (value.unflatten(-1, (-1, 16)) * scale.unsqueeze(-1)).flatten(-2)
        got.append(rows.double())
    return got


def _exact_attention(q, k, v, at, case):
    """q [n, Hq, D] at positions `at`, over keys [L, Hkv, D]: outputs and log sums, head group by head group."""
    W, S = case["window"], case["sinks"]
    G = case["Hq"] // case["Hkv"]
    out = torch.zeros(q.shape[0], case["Hq"], case["D"], dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], float("-inf"), dtype=torch.float64, device=q.device)
    if k.shape[0] == 0:
        return out, lse
    j = torch.arange(k.shape[0], device=q.device)
    dist = at[:, None] - j
    hidden = dist < 0
    if W:
        hidden |= (dist >= W) & (j >= S)
    for h in range(case["Hkv"]):
        heads = slice(h * G, (h + 1) * G)
        s = torch.matmul(q[:, heads].transpose(0, 1), k[:, h].T) / math.sqrt(case["D"])
        s[:, hidden] = float("-inf")
        lse[:, heads] = torch.logsumexp(s, -1).T
        out[:, heads] = torch.matmul(torch.softmax(s, -1), v[:, h]).transpose(0, 1)
    return out, lse


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm_rope":
        got = []
        for name in ("q", "k"):
            x = st[name].double()
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["D"] + EPS) * st[name + "_weight"].double()
            got.append(_exact_rotation(x, st["positions"], case, st["inv_freq"]))
        return tuple(got)
    if op == "append":
        T, page, got = case["T"], case["page"], []
        place = st["table"].long()[st["seq"][:T].long(), st["pos"][:T].long() // page] * page + st["pos"][:T].long() % page
        for name in ("k",) if case["shared"] else ("k", "v"):
            x = st["new_" + name][:T].double()
            if name == "k":
                x = _exact_rotation(x, st["pos"][:T], case, st["inv_freq"])
            if case["type"] == "fp4":
                x = _exact_fp4(x.to(torch.bfloat16).double())
            whole = torch.zeros(st[name].shape[0] * page, case["Hkv"], case["D"], dtype=torch.float64, device="cuda")
            whole[place] = x
            got.append(whole.unflatten(0, (-1, page)))
        return got
    q, outs, sums = st["q"].double(), [], []
    if op == "decode":
        for b, n in enumerate(_lens(case)):
            k, v = _exact_sequence(st, case, b, n)
            o, s = _exact_attention(q[b:b + 1], k, v, torch.tensor([n - 1], device="cuda"), case)
            outs.append(o)
            sums.append(s)
    else:
        n, lens = _window_span(case)
        start = 0
        for b, (new, total) in enumerate(zip(n, lens)):
            k, v = _exact_sequence(st, case, b, total)
            for i in range(0, new, 1024):
                m = min(1024, new - i)
                at = torch.arange(total - new + i, total - new + i + m, device="cuda")
                o, s = _exact_attention(q[start + i:start + i + m], k, v, at, case)
                outs.append(o)
                sums.append(s)
            start += new
    return torch.cat(outs), torch.cat(sums)
