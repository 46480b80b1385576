"""fp64 CPU oracle for linear attention with a decay for each head and for rotary positions.

TEST INFRASTRUCTURE ONLY, as the rest of this package. Plain definitions in float64 numpy:

* per sequence and value head ``S_t = e^{g_t} S_{t-1} + v_t k_t^T``, ``o_t = scale S_t q_t``, token
  by token; value head h reads q/k head ``h // (H / H_qk)``; an empty sequence's final state is its
  initial state; with ``absolute`` every input is replaced by its absolute value, which gives the
  sums of the terms' sizes that error bounds are made of;
* ``rotate``: the pair (a, b) of channels ``(i, i + r/2)``, or ``(2i, 2i + 1)``, becomes
  ``f (a cos - b sin, a sin + b cos)`` with the angle ``pos * inv_freq[i]``.
"""
from __future__ import annotations

import numpy as np


def linear_forward(q, k, v, g, cu_seqlens, *, scale, initial=None, absolute=False):
    """q, k ``[T, H_qk, K]``, v ``[T, H, V]``, g ``[T, H]``, ``[H]`` or None, initial ``[N, H, V, K]`` or
    None (zero). Returns ``(out [T, H, V], final [N, H, V, K])``; rows behind the last bound are NaN."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    T, H, V = v.shape
    group = H // q.shape[1]
    q, k = np.repeat(q, group, axis=1), np.repeat(k, group, axis=1)
    cu = [int(x) for x in cu_seqlens]
    N = len(cu) - 1
    g = np.zeros((T, H)) if g is None else np.broadcast_to(np.asarray(g, np.float64), (T, H))
    S = np.zeros((N, H, V, q.shape[2])) if initial is None else np.array(initial, np.float64)
    if absolute:
        q, k, v, S, scale = abs(q), abs(k), abs(v), abs(S), abs(scale)
    out = np.full((T, H, V), np.nan)
    for n in range(N):
        for t in range(cu[n], cu[n + 1]):
            S[n] = S[n] * np.exp(g[t])[:, None, None] + v[t][:, :, None] * k[t][:, None, :]
            out[t] = scale * np.einsum("hvk,hk->hv", S[n], q[t])
    return out, S


def rotate(x, positions, inv_freq, *, interleaved=False, factor=1.0, inverse=False):
    """x ``[T, H, D]`` with its first ``2 len(inv_freq)`` channels rotated."""
    x = np.array(x, np.float64)
    r = len(inv_freq)
    theta = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = factor * np.cos(theta)[:, None], factor * np.sin(-theta if inverse else theta)[:, None]
    first = slice(0, 2 * r, 2) if interleaved else slice(0, r)
    second = slice(1, 2 * r, 2) if interleaved else slice(r, 2 * r)
    a, b = x[..., first].copy(), x[..., second].copy()
    x[..., first], x[..., second] = a * c - b * s, a * s + b * c
    return x
