"""Float64 CPU oracle of the operators around the attention calls: the per-head
norm with the position rotation and its gradient, the append to a paged cache,
and attention of a ragged chunk over that cache.

TEST INFRASTRUCTURE ONLY, like ``oracle.attention``, whose dense definition the
paged call below evaluates sequence by sequence.  Plain definitions:

* z = w x / sqrt(mean(x^2) + eps) per head; pair j of the first ``rot`` elements
  of z turns by position * inv_freq[j].  Pairs are (j, j + rot/2), or
  (2j, 2j + 1) when interleaved.
* the gradient is the transpose of that map's Jacobian.
* logical token t of sequence i sits in page block_table[i, t // page_size],
  slot t % page_size.
"""
from __future__ import annotations

import numpy as np

from oracle import attention


def pair_index(rot, interleaved):
    """(first, second) element of every rotation pair."""
    j = np.arange(rot // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)


def rotate(x, positions, inv_freq, interleaved=False):
    """x (..., tokens, heads, d), positions (tokens,): the turned copy of x."""
    inv_freq = np.asarray(inv_freq, np.float64)
    a = np.asarray(positions, np.float64)[:, None] * inv_freq[None, :]
    c, s = np.cos(a)[:, None, :], np.sin(a)[:, None, :]
    i, j = pair_index(2 * inv_freq.size, interleaved)
    y = np.array(x, np.float64)
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    return y


def norm(x, weight, eps):
    """x / sqrt(mean(x^2) + eps) * weight over the last dimension; x without a weight."""
    if weight is None:
        return np.array(x, np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight


def norm_rope(x, positions, inv_freq, weight=None, eps=1e-6, interleaved=False):
    return rotate(norm(np.asarray(x, np.float64), weight, eps), positions, inv_freq, interleaved)


def norm_rope_backward(x, gy, positions, inv_freq, weight=None, eps=1e-6, interleaved=False):
    """(gx, gweight) of norm_rope for the output gradient gy; x (tokens, heads, d)."""
    gz = rotate(np.asarray(gy, np.float64), -np.asarray(positions, np.float64), inv_freq, interleaved)
    if weight is None:
        return gz, None
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    gweight = (gz * x * r).reshape(-1, d).sum(0)
    gw = gz * weight
    gx = r * gw - x * r ** 3 * (gw * x).mean(-1, keepdims=True)
    return gx, gweight


def token_positions(cu_seqlens, cache_seqlens):
    """(sequence, position) of every packed row of the call."""
    cu = np.asarray(cu_seqlens, np.int64)
    seq = np.concatenate([np.full(n, i) for i, n in enumerate(np.diff(cu))] or [[]]).astype(np.int64)
    r = np.arange(cu[-1]) - cu[seq] if cu[-1] else np.zeros(0, np.int64)
    return seq, np.asarray(cache_seqlens, np.int64)[seq] + r


def append(k_new, v_new, k_cache, v_cache, cu_seqlens, cache_seqlens, block_table, *, inv_freq=(),
           weight=None, eps=1e-6, interleaved=False):
    """The caches (num_pages, page_size, hkv, d) after the append; block_table
    None means one page per sequence."""
    k_cache, v_cache = np.array(k_cache, np.float64), np.array(v_cache, np.float64)
    seq, pos = token_positions(cu_seqlens, cache_seqlens)
    k = norm_rope(np.asarray(k_new)[:seq.size], pos, inv_freq, weight, eps, interleaved)
    ps = k_cache.shape[1]
    for r, (i, p) in enumerate(zip(seq, pos)):
        page = i if block_table is None else block_table[i][p // ps]
        k_cache[page, p % ps] = k[r]
        v_cache[page, p % ps] = v_new[r]
    return k_cache, v_cache


def gather(cache, block_table, i, length):
    """The first `length` logical rows of sequence i, (length, hkv, d)."""
    ps = cache.shape[1]
    if block_table is None:
        return cache[i, :length]
    n = -(-length // ps)
    return cache[np.asarray(block_table[i][:n], np.int64)].reshape(-1, *cache.shape[2:])[:length]


def paged_forward(q, k_cache, v_cache, cu_seqlens, cache_seqlens, block_table, scale, *,
                  appended=True, causal=False, win_l=-1, win_r=-1, softcap=0.0):
    """(out (Tq,hq,d), lse (hq,Tq), spread (Tq,hq,d)) of the ragged chunk, with
    spread = sum_j P_j |v_j|, the size against which rounding errors of P count.
    Rows behind the last sequence are NaN.  Slots that hold no key of a row's
    sequence are not looked at, and keys that no row sees count as zeros."""
    tq, hq, d = q.shape
    out = np.full((tq, hq, d), np.nan)
    spread = np.full((tq, hq, d), np.nan)
    lse = np.full((hq, tq), np.nan)
    cu = np.asarray(cu_seqlens, np.int64)
    for i in range(cu.size - 1):
        n = int(cu[i + 1] - cu[i])
        if n == 0:
            continue
        length = int(cache_seqlens[i]) + (n if appended else 0)
        first = 0 if win_l < 0 else max(0, length - n - win_l)
        k, v = np.zeros((length,) + k_cache.shape[2:]), np.zeros((length,) + v_cache.shape[2:])
        first = min(first, length)
        ps = k_cache.shape[1]
        for t in range(first, length):
            page = i if block_table is None else block_table[i][t // ps]
            k[t], v[t] = k_cache[page, t % ps], v_cache[page, t % ps]
        rows = slice(int(cu[i]), int(cu[i + 1]))
        args = (scale, causal, win_l, win_r, softcap)
        o, l = attention.forward(q[None, rows], k[None], v[None], *args)
        a, _ = attention.forward(q[None, rows], k[None], np.abs(v)[None], *args)
        out[rows], lse[:, rows], spread[rows] = o[0], l[0], a[0]
    return out, lse, spread
