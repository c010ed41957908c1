"""Float64 statements of the head and paged-cache calls (include/csa2.h, part p)."""
import numpy as np


def rotate(x, positions, inv_freq, offset=0, interleaved=False, inverse=False):
    """x [T, H, D]: pair i of channels [offset, offset + 2 * half) turned by positions[t] * inv_freq[i]."""
    x = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    angle = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)[None, :]
    if inverse:
        angle = -angle
    for i in range(half):
        a = offset + (2 * i if interleaved else i)
        b = a + 1 if interleaved else a + half
        c, s = np.cos(angle[:, i])[:, None], np.sin(angle[:, i])[:, None]
        xa, xb = x[:, :, a].copy(), x[:, :, b].copy()
        x[:, :, a] = xa * c - xb * s
        x[:, :, b] = xb * c + xa * s
    return x


def head_norm(x, weight, eps):
    """x [T, H, D] / rms * weight (weight None: x)."""
    x = np.asarray(x, dtype=np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def paged_rows(pages, table_row, n):
    """The first n tokens' rows [n, H, D] of one sequence from pages [n_pages, page_size, H, D]."""
    size = pages.shape[1]
    if n == 0:
        return np.zeros((0,) + pages.shape[2:])
    return np.stack([pages[table_row[j // size], j % size] for j in range(n)]).astype(np.float64)


def causal_attn(q, positions, k, v, scale, window=0, sinks=0):
    """q [n, Hq, D] at the given positions over keys and values [L, Hkv, D].  Query p sees
    token j <= p with p - j < window (window 0: any) or j < sinks.  Returns out, lse,
    and sum_j p_j |v_j| (the magnitude that rounding errors scale with)."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, mag = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse = np.full((n, Hq), -np.inf)
    for i in range(n):
        p = int(positions[i])
        seen = [j for j in range(min(p + 1, len(k))) if window == 0 or p - j < window or j < sinks]
        if not seen:
            continue
        for h in range(k.shape[1]):
            kk, vv = k[seen, h], v[seen, h]
            s = q[i, h * G:(h + 1) * G] @ kk.T * scale
            m = s.max(-1, keepdims=True)
            e = np.exp(s - m)
            w = e / e.sum(-1, keepdims=True)
            out[i, h * G:(h + 1) * G] = w @ vv
            mag[i, h * G:(h + 1) * G] = w @ np.abs(vv)
            lse[i, h * G:(h + 1) * G] = m[:, 0] + np.log(e.sum(-1))
    return out, lse, mag
