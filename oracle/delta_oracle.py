"""fp64 CPU oracle for the gated delta rule with one decay for each head and for norms of q and k.

TEST INFRASTRUCTURE ONLY, as the rest of this package. Plain definitions in float64 numpy:

* per sequence and value head ``S <- e^{g_t} S``, ``S <- S + beta_t (v_t - S k_t) k_t^T``, ``o_t = scale S q_t``, token by
  token; value head h reads q/k head ``h // (H / H_qk)``; an empty sequence's final state is its initial state;
* ``qk_norm``: a row x becomes ``rotate(x / sqrt(m sum x^2 + eps) (offset + weight))``, m = 1 / D or 1, and
  ``qk_norm_gradient`` its gradient, written from the Jacobian of the normalised row.
"""
from __future__ import annotations

import numpy as np

from .linear_oracle import rotate

NORM_EPS = 1e-6


def unit(x):
    return x / np.sqrt((x * x).sum(-1, keepdims=True) + NORM_EPS)


def delta_forward(q, k, v, g, beta, cu_seqlens, *, scale, initial=None, normalize=False):
    """q, k ``[T, H_qk, K]``, v ``[T, H, V]``, g ``[T, H]``, ``[H]`` or None, beta ``[T, H]``, initial ``[N, H, V, K]`` or None
    (zero). Returns ``(out [T, H, V], final [N, H, V, K], size [N, H])``; size is the largest value of any state element
    or value on a sequence's way; rows behind the last bound are NaN."""
    q, k, v, beta = (np.asarray(x, np.float64) for x in (q, k, v, beta))
    if normalize:
        q, k = unit(q), unit(k)
    T, H, V = v.shape
    group = H // q.shape[1]
    q, k = np.repeat(q, group, axis=1), np.repeat(k, group, axis=1)
    cu = [int(x) for x in cu_seqlens]
    N = len(cu) - 1
    g = np.zeros((T, H)) if g is None else np.broadcast_to(np.asarray(g, np.float64), (T, H))
    S = np.zeros((N, H, V, q.shape[2])) if initial is None else np.array(initial, np.float64)
    out = np.full((T, H, V), np.nan)
    size = abs(S).max((2, 3))
    for n in range(N):
        for t in range(cu[n], cu[n + 1]):
            s = S[n] * np.exp(g[t])[:, None, None]
            learn = beta[t][:, None] * (v[t] - np.einsum("hvk,hk->hv", s, k[t]))
            S[n] = s + learn[:, :, None] * k[t][:, None, :]
            out[t] = scale * np.einsum("hvk,hk->hv", S[n], q[t])
            size[n] = np.maximum(size[n], np.maximum(abs(S[n]).max((1, 2)), abs(v[t]).max(1)))
    return out, S, size


def qk_norm(x, weight=None, positions=None, inv_freq=None, *, l2=False, eps=1e-6, offset=0.0, interleaved=False):
    """x ``[T, H, D]``."""
    x = np.asarray(x, np.float64)
    y = x / np.sqrt((x * x).sum(-1, keepdims=True) * (1 if l2 else 1 / x.shape[-1]) + eps)
    if weight is not None:
        y = y * (offset + np.asarray(weight, np.float64))
    return y if inv_freq is None else rotate(y, positions, inv_freq, interleaved=interleaved)


def qk_norm_gradient(dy, x, weight=None, positions=None, inv_freq=None, *, l2=False, eps=1e-6, offset=0.0, interleaved=False):
    """``(dx, dweight)`` for the result's gradient dy; dweight None without a weight."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    m = 1.0 if l2 else 1.0 / x.shape[-1]
    size = np.sqrt(m * (x * x).sum(-1) + eps)
    z = dy if inv_freq is None else rotate(dy, positions, inv_freq, interleaved=interleaved, inverse=True)
    dweight = None
    u = z
    if weight is not None:
        dweight = np.einsum("thd,thd,th->d", z, x, 1 / size)
        u = z * (offset + np.asarray(weight, np.float64))
    # d (x_i / size) / d x_j = delta_ij / size - m x_i x_j / size^3
    dx = u / size[..., None] - m * x * (np.einsum("thd,thd->th", u, x) / size ** 3)[..., None]
    return dx, dweight
