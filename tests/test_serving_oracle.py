"""Pins of oracle/serving.py: closed forms, finite differences and the pinned
attention oracle (CPU)."""
import numpy as np
import pytest

from oracle import attention as ref
from oracle import serving


def freqs(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2) / max(rot, 1))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_depends_on_distance(interleaved):
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 5, 3, 32))
    f = freqs(16)
    pos = np.array([0, 1, 7, 1000, 123456])
    rq = serving.rotate(q, pos, f, interleaved)
    np.testing.assert_allclose(np.linalg.norm(rq, axis=-1), np.linalg.norm(q, axis=-1), rtol=1e-12)
    np.testing.assert_array_equal(rq[0], q[0])             # position 0 turns nothing
    np.testing.assert_array_equal(rq[..., 16:], q[..., 16:])  # nor are later elements turned
    a = (serving.rotate(q, pos, f, interleaved) * serving.rotate(k, pos + 5, f, interleaved)).sum(-1)
    b = (serving.rotate(q, pos * 0, f, interleaved) *
         serving.rotate(k, pos * 0 + 5, f, interleaved)).sum(-1)
    np.testing.assert_allclose(a, b, atol=1e-9)
    # a quarter turn of the first pair: (a, b) -> (-b, a)
    i, j = serving.pair_index(2, interleaved)
    x = np.array([[[3.0, 4.0]]])
    np.testing.assert_allclose(serving.rotate(x, [1], [np.pi / 2], interleaved)[0, 0, [i[0], j[0]]],
                               [-4.0, 3.0], atol=1e-15)


def test_norm_gives_unit_mean_square():
    rng = np.random.default_rng(1)
    x = 10 * rng.standard_normal((4, 2, 64))
    y = serving.norm(x, np.ones(64), 0.0)
    np.testing.assert_allclose((y * y).mean(-1), 1.0, rtol=1e-12)
    np.testing.assert_array_equal(serving.norm(x, None, 1.0), x)


@pytest.mark.parametrize("interleaved,rot", [(False, 16), (True, 16), (False, 8), (True, 0)])
def test_gradient_matches_finite_differences(interleaved, rot):
    rng = np.random.default_rng(2)
    x, gy = rng.standard_normal((2, 3, 2, 16))
    w = 1 + 0.3 * rng.standard_normal(16)
    pos, f, eps = np.array([0, 5, 91]), freqs(rot), 1e-3
    loss = lambda x, w: (serving.norm_rope(x, pos, f, w, eps, interleaved) * gy).sum()
    gx, gw = serving.norm_rope_backward(x, gy, pos, f, w, eps, interleaved)
    h = 1e-5
    for g, a, at in ((gx, x, lambda v: loss(v, w)), (gw, w, lambda v: loss(x, v))):
        for i in np.ndindex(a.shape):
            up, dn = a.copy(), a.copy()
            up[i] += h
            dn[i] -= h
            assert abs((at(up) - at(dn)) / (2 * h) - g[i]) < 1e-7


def test_paged_equals_dense_and_append_lands_in_place():
    rng = np.random.default_rng(3)
    hkv, hq, d, ps = 2, 4, 16, 4
    new, cached = [3, 0, 5], [6, 2, 0]
    cu = np.cumsum([0] + new)
    table = np.array([[7, 1, 4], [0, 9, 9], [5, 2, 9]])
    kc, vc = rng.standard_normal((2, 10, ps, hkv, d))
    kn, vn = rng.standard_normal((2, 8, hkv, d))
    q = rng.standard_normal((9, hq, d))  # one padding row
    k2, v2 = serving.append(kn, vn, kc, vc, cu, cached, table)
    assert (k2 != kc).any(axis=(1, 2, 3)).sum() == 4  # pages 1, 4 (sequence 0), 5, 2 (sequence 2)
    out, lse, spread = serving.paged_forward(q, k2, v2, cu, cached, table, 0.3, causal=True)
    assert np.isnan(out[8]).all() and np.isnan(lse[:, 8]).all()
    for i in (0, 2):
        k = np.concatenate([kc[table[i]].reshape(-1, hkv, d)[:cached[i]], kn[cu[i]:cu[i + 1]]])
        v = np.concatenate([vc[table[i]].reshape(-1, hkv, d)[:cached[i]], vn[cu[i]:cu[i + 1]]])
        o, l = ref.forward(q[None, cu[i]:cu[i + 1]], k[None], v[None], 0.3, causal=True)
        np.testing.assert_allclose(out[cu[i]:cu[i + 1]], o[0], rtol=1e-12)
        np.testing.assert_allclose(lse[:, cu[i]:cu[i + 1]], l[0], rtol=1e-12)
    assert (spread[:8] >= np.abs(out[:8]) - 1e-12).all()


def test_paged_window_skips_unseen_pages():
    """Table entries of pages that no row sees are not read."""
    rng = np.random.default_rng(4)
    kc, vc = rng.standard_normal((2, 6, 4, 1, 8))
    q = rng.standard_normal((2, 1, 8))
    table = np.array([[3, 1, 4, 5]])
    hidden = np.array([[-77, 1, 4, 5]])
    a = serving.paged_forward(q, kc, vc, [0, 2], [14], table, 1.0, causal=True, win_l=8)
    b = serving.paged_forward(q, kc, vc, [0, 2], [14], hidden, 1.0, causal=True, win_l=8)
    np.testing.assert_array_equal(a[0], b[0])
