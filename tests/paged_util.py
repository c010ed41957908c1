"""Helpers of the paged-cache tests: caches with every unused slot poisoned, the
float64 side, and the error bounds.

Bounds.  u = eps / 2 of the 16-bit type: a rounding is off by at most half a step,
u relative (bf16 2^-8, f16 2^-11).

Head norm and rotation: the f32 chain (a sum of up to 512 squares in a tree of
at most 21 additions, rsqrt, four products, one sum) stays within 32 f32 steps,
2^-19, of |a| + |b| of the rotated pair; then one rounding.

Attention, with mag = sum_j p_j |v_j|:
  - a score errs by ds <= (D + 8) 2^-24 scale sum_d |q_d k_d|, a weight by 2 ds
    relative (numerator and sum), plus 2^-20 for the exponential's approximation;
  - weights are rounded to the 16-bit type for the product: u relative, and for
    f16, whose weights below 2^-14 have a fixed step, at most 2^-25 each (the
    largest weight of a row is 1 before normalisation);
  - f32 sums over L tokens, 16 at a time, and one rescale per tile or chunk:
    (L / 8 + 64) 2^-23 relative;
  - out is rounded once: u |out| (and 2^-25 for f16's fixed step).
lse: ds + (L / 8 + 64) 2^-24 + 2^-20 + 2^-22 |lse|.
"""
import numpy as np
import torch

import kv_cache_csa2_b200 as K
import oracle as O

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "fp4": torch.bfloat16}


def f64(t):
    return t.detach().double().cpu().numpy()


def half_step(dt):
    return torch.finfo(dt).eps / 2


def rng_normal(seed, *shape, dt=torch.bfloat16, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)


def make_cache(kind, lens, page, heads, D, shared=False, seed=0, layout="dense", spare=3, max_len=0, std=1.0):
    """A PagedKv over random pages holding N(0, std) rows, every slot that no token
    owns (past an end, unused pages) poisoned with NaN; and the rows in float64:
    per sequence (k [n, heads, D], v)."""
    B = len(lens)
    width = max(1, max(-(-n // page) for n in lens)) + 1      # one table column no token needs
    n_pages = B * width + spare
    g = torch.Generator().manual_seed(1000 + seed)
    perm = torch.randperm(n_pages, generator=g)[:B * width].view(B, width).int()
    own = torch.zeros(n_pages, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(n):
            own[perm[b, j // page], j % page] = True
        perm[b, -(-n // page):] = 2 ** 30                     # entries past the length are never read
    own = own.cuda()
    parts = []
    for i in range(1 if shared else 2):
        rows = rng_normal(seed * 7 + i, n_pages, page, heads, D, dt=DT[kind], std=std)
        if kind == "fp4":
            codes, scales = K.csa2_fp4_pack(rows)
            values = K.csa2_fp4_unpack(codes, scales)
            scales[~own] = 0x7f                               # E4M3 NaN
            parts.append((codes, scales, values))
        else:
            values = rows.clone()
            rows[~own] = float("nan")
            parts.append((rows, None, values))

    def lay(ts):
        """The tensors of `ts` in the wanted layout (same logical shape)."""
        ts = [t for t in ts if t is not None]
        if layout == "dense" or not ts:
            return ts
        if layout == "heads":                                 # [n_pages, heads, page, ..]
            return [t.transpose(1, 2).contiguous().transpose(1, 2) for t in ts]
        both = torch.stack(ts, 1)                             # [n_pages, 2, page, heads, ..]: k and v of a page together
        return [both[:, i] for i in range(len(ts))]

    data = lay([p[0] for p in parts])
    scales = lay([p[1] for p in parts])
    cache = K.PagedKv(data[0], perm.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                      v=None if shared else data[1], k_scales=scales[0] if scales else None,
                      v_scales=scales[1] if scales and not shared else None, max_len=max_len)
    host = []
    vals = [f64(p[2]) for p in parts]
    for b, n in enumerate(lens):
        k = O.paged_rows(vals[0], perm[b].numpy(), n)
        host.append((k, k if shared else O.paged_rows(vals[1], perm[b].numpy(), n)))
    return cache, host


def check_attn(out, lse, want, q, keys, scale, dt, tokens, what=""):
    """out, lse (device) of n query rows against want = causal_attn(...)."""
    o, s, mag = want
    u = half_step(dt)
    got, got_lse = f64(out), f64(lse)
    assert np.array_equal(np.isfinite(got_lse), np.isfinite(s)), f"{what}: lse finiteness"
    G = q.shape[1] // keys.shape[1]
    ds = 0.0
    if len(keys):
        ka = np.abs(keys).max(0).repeat(G, 0)                 # [Hq, D] largest |k_d|
        ds = (q.shape[2] + 8) * 2.0 ** -24 * scale * (np.abs(q) * ka[None]).sum(-1)
    rel = 2 * ds + 2.0 ** -20 + (tokens / 8 + 64) * 2.0 ** -23 + u * 1.01
    tol = (rel[..., None] if np.ndim(rel) else rel) * mag + u * np.abs(o)
    if dt == torch.float16:
        vmax = mag.max(initial=0.0) if not len(keys) else 8.0
        tol = tol + 2.0 ** -25 * (1 + tokens * vmax)
    err = np.abs(got - o)
    assert np.all(err <= tol + 1e-30), f"{what}: out off by {(err - tol).max():.3g} over its bound, worst {err.max():.3g}"
    fin = np.isfinite(s)
    if fin.any():
        ltol = ds + (tokens / 8 + 64) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(fin, s, 0))
        d = np.abs(np.where(fin, got_lse, 0) - np.where(fin, s, 0))
        assert np.all(d <= ltol), f"{what}: lse off by {d.max():.3g}"
