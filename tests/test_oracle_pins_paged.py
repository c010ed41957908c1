"""What pins the float64 statements of the head and paged-cache calls (CPU)."""
import numpy as np
import torch

import oracle as O


def test_rotation_hand_worked():
    x = np.zeros((1, 1, 8))
    x[0, 0, 2], x[0, 0, 4] = 1.0, 2.0
    f = [np.pi / 6, np.pi / 4]
    y = O.rotate(x, [2], f, offset=2)                 # pairs (2, 4), (3, 5); angles 60 and 90 degrees
    c, s = 0.5, np.sqrt(3) / 2
    np.testing.assert_allclose(y[0, 0], [0, 0, c - 2 * s, 0, 2 * c + s, 0, 0, 0], atol=1e-12)
    y = O.rotate(x, [2], f, offset=2, interleaved=True)   # pairs (2, 3), (4, 5)
    np.testing.assert_allclose(y[0, 0], [0, 0, c, s, 0, 2, 0, 0], atol=1e-12)
    np.testing.assert_allclose(O.rotate(y, [2], f, 2, True, inverse=True), x, atol=1e-12)


def test_rotated_products_depend_on_distance_only():
    r = np.random.default_rng(0)
    q, k = r.standard_normal((2, 1, 1, 16))
    f = r.random(8)
    dots = [(O.rotate(q, [p + 5], f) * O.rotate(k, [p], f)).sum() for p in (0, 3, 1000)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-10)


def test_norm_gives_unit_rms():
    x = np.random.default_rng(1).standard_normal((3, 2, 32)) * 7
    y = O.head_norm(x, np.ones(32), 0.0)
    np.testing.assert_allclose((y * y).mean(-1), 1.0)
    np.testing.assert_allclose(y * np.sqrt((x * x).mean(-1, keepdims=True)), x)


def test_attention_equals_sdpa_under_its_mask():
    r = np.random.default_rng(2)
    n, Hq, Hk, D, past, W, S = 9, 6, 2, 16, 12, 7, 3
    q, k, v = r.standard_normal((n, Hq, D)), r.standard_normal((past + n, Hk, D)), r.standard_normal((past + n, Hk, D))
    pos = past + np.arange(n)
    out, lse, mag = O.causal_attn(q, pos, k, v, 0.3, W, S)
    j = np.arange(past + n)
    mask = (j <= pos[:, None]) & ((j > pos[:, None] - W) | (j < S))
    t = lambda a: torch.from_numpy(a).transpose(0, 1)
    rep = lambda a: t(a).repeat_interleave(Hq // Hk, 0)
    want = torch.nn.functional.scaled_dot_product_attention(t(q), rep(k), rep(v), torch.from_numpy(mask), scale=0.3)
    np.testing.assert_allclose(out, want.transpose(0, 1).numpy(), atol=1e-12)
    s = torch.einsum("hqd,hkd->hqk", t(q), rep(k)) * 0.3
    s = s.masked_fill(~torch.from_numpy(mask), float("-inf"))
    np.testing.assert_allclose(lse, torch.logsumexp(s, -1).T.numpy(), atol=1e-12)
    assert np.all(mag >= np.abs(out) - 1e-12)
    empty = O.causal_attn(q[:1], [-1], k, v, 0.3)
    assert np.all(empty[0] == 0) and np.all(np.isneginf(empty[1]))


def test_paged_rows_follow_the_table():
    pages = np.arange(5 * 4 * 1 * 2).reshape(5, 4, 1, 2)
    rows = O.paged_rows(pages, np.array([3, 1, 99]), 6)
    np.testing.assert_array_equal(rows, np.concatenate([pages[3], pages[1][:2]]))
    assert O.paged_rows(pages, np.array([99]), 0).shape == (0, 1, 2)
