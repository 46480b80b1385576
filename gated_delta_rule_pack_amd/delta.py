"""The gated delta rule with one decay for each head.

``gated_delta_fwd`` (prompts) and ``gated_delta_step`` (single tokens) serve beside ``linear_fwd`` and
``linear_step`` with the same packed bounds, state pool, slots, checks and errors. They enqueue the kernels of
``libkda.so`` on the current torch stream; nothing synchronises and no metadata is built, so every call can be
captured. They record no gradient, and refuse inputs that require one while gradients are enabled, or that carry a
forward-mode tangent.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .linear import (_BF16, _Call, _check, _context, _fill_linear, _grads_on, _like, _on, _packed, _refuse_gradient, _refuse_tangents,
                     _tangents_on)

__all__ = ["gated_delta_fwd", "gated_delta_step"]

_F16 = torch.float16
_PATHS = {"walk": _lib.KDA_DELTA_WALK, "scan": _lib.KDA_DELTA_SCAN}


def make_gated_delta_args(q, k, v, g, beta, *, N=None, cu_seqlens=None, cu_seqlens_cpu=None, scale=None, normalize=False,
                          initial_state=None, final_state=None, state_cache=None, state_indices=None,
                          has_initial_state=None, out=None, state_k_first=False, path=None) -> "_lib.GatedDeltaArgs":
    """Fill a ``kda_gated_delta_args`` from tensors (no allocation), checking what the C side cannot see."""
    if beta is None:
        raise ValueError("beta is required")
    if beta.requires_grad and _grads_on():
        _refuse_gradient()
    if _tangents_on():
        _refuse_tangents(beta)
    a = _lib.GatedDeltaArgs()
    dtype = q.dtype
    if dtype == _BF16:
        a.dtype = _lib.KDA_BF16
    elif dtype == _F16:
        a.dtype = _lib.KDA_F16
    else:
        raise TypeError(f"q must be bf16 or fp16, got {dtype}")
    lin = a.lin
    _fill_linear(lin, q, k, v, g, dtype, N, cu_seqlens, cu_seqlens_cpu, scale, initial_state, final_state, state_cache,
                 state_indices, has_initial_state, out, state_k_first)
    if beta.dim() == 3 and beta.shape[0] == 1:
        beta = beta[0]
    if beta.dtype == torch.float32:
        a.beta_dtype = _lib.KDA_F32
    elif beta.dtype == _BF16:
        a.beta_dtype = _lib.KDA_BF16
    else:
        raise TypeError(f"beta must be fp32 or bf16, got {beta.dtype}")
    if beta.shape != (lin.T, lin.H) or not beta.is_contiguous():
        raise ValueError(f"beta must be a contiguous [T, H] = {(lin.T, lin.H)}, got {tuple(beta.shape)}")
    a.beta = beta.data_ptr()
    if normalize:
        a.normalize = 1
    if path is not None:
        if path not in _PATHS:
            raise ValueError(f"unknown path {path!r}: None, 'walk' or 'scan'")
        a.path = _PATHS[path]
    return a


def gated_delta_fwd(q, k, v, g, beta, cu_seqlens, *, cu_seqlens_cpu=None, scale=None, normalize=False, initial_state=None,
                    output_final_state=False, state_cache=None, state_indices=None, has_initial_state=None, out=None,
                    workspace=None, stream=None, context=None, state_k_first=False, path=None):
    """The gated delta rule over packed prompts, for each token and head
    ``S <- e^g S``, ``S <- S + beta (v - S k) k^T``, ``o = scale S q``.

    q, k: ``[T, H_qk, K]``, v: ``[T, H, V]`` (or with a leading 1), all bf16 or all fp16, K and V 64 or 128, H_qk
    dividing H; rows may be strided. g: log decays, at most 0, fp32 or bf16, ``[H]`` or ``[T, H]``, or None for no decay.
    beta: step sizes, fp32 or bf16 ``[T, H]``, as they are used (any sigmoid has been applied). ``normalize`` takes q and k
    to unit length first (``x / sqrt(sum x^2 + 1e-6)``, in fp32); without it keys have to be near unit length
    themselves, or at least keep ``|beta| |k|^2 <= 2``, beyond which a step grows the state. (Raw keys may differ
    in length, with step sizes to match; lengths more than 2^12 apart within 64 tokens may leave nothing finite.)
    scale defaults to ``K ** -0.5``.

    cu_seqlens, states, ``out``, ``stream`` and ``context`` as in :func:`linear_fwd`. ``workspace``: a contiguous uint8 tensor at
    a 256-byte address, made here where none is given; one that is too small or lies elsewhere is refused with KDAError. "walk"
    needs none; "scan" keeps a record of every chunk in it, 308 bytes for each token and value head and 4 K for each token and q/k
    head (a chunk more for each sequence): 593 MB for 32768 tokens of 32 heads that share 16. ``path`` overrides the
    choice between one kernel that walks every sequence of a head ("walk") and two that split the work further
    ("scan"), which agree within rounding. The choice looks at the shapes and, where ``cu_seqlens_cpu`` is given, at the
    lengths: give it where a batch mixes long prompts with single tokens. Returns ``(out, final_state)``, final_state
    None unless dense and asked for."""
    with _Call(q, stream) as call:
        _on(call.index, "k v g beta cu_seqlens initial_state state_cache state_indices has_initial_state out workspace",
            k, v, g, beta, cu_seqlens, initial_state, state_cache, state_indices, has_initial_state, out, workspace)
        if cu_seqlens is None:
            raise ValueError("cu_seqlens is required")
        if out is None:
            out = _like(v)
        final_state = None
        if output_final_state and state_cache is None:
            H, V, K = *_packed("v", v).shape[1:], _packed("q", q).shape[2]
            dt = initial_state.dtype if initial_state is not None else torch.float32
            planes = (K, V) if state_k_first else (V, K)
            final_state = torch.empty((cu_seqlens.numel() - 1, H, *planes), dtype=dt, device=q.device)
        a = make_gated_delta_args(q, k, v, g, beta, cu_seqlens=cu_seqlens, cu_seqlens_cpu=cu_seqlens_cpu, scale=scale,
                                  normalize=normalize, initial_state=initial_state, final_state=final_state,
                                  state_cache=state_cache, state_indices=state_indices, has_initial_state=has_initial_state,
                                  out=out, state_k_first=state_k_first, path=path)
        if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()):
            raise TypeError("workspace must be a contiguous uint8 tensor")
        lib, ref, context = _lib.load(), ctypes.byref(a), _context(context, call.index)
        given = (workspace.data_ptr(), workspace.numel()) if workspace is not None else (None, 0)
        # Short calls need no workspace: it is asked for where the call says so, which has enqueued nothing then. (One that is given and
        # does not serve is the caller's to mend.)
        rc = lib.kda_gated_delta_fwd(context, ref, *given, call.handle)
        if rc == _lib.KDA_ERR_WORKSPACE and workspace is None:
            workspace = torch.empty(lib.kda_gated_delta_fwd_workspace_bytes(ref), dtype=torch.uint8, device=call.device)
            rc = lib.kda_gated_delta_fwd(context, ref, workspace.data_ptr(), workspace.numel(), call.handle)
        _check(rc, "kda_gated_delta_fwd")
    return out, final_state


def gated_delta_step(q, k, v, g, beta, *, state_cache, state_indices=None, has_initial_state=None, scale=None,
                     normalize=False, out=None, stream=None, context=None, state_k_first=False):
    """One token of each of N requests: ``S <- e^g S``, ``S <- S + beta (v - S k) k^T``, ``o = scale S q``.

    q, k: ``[N, H_qk, K]``, v: ``[N, H, V]``, g ``[H]``, ``[N, H]`` or None, beta ``[N, H]``, as in
    :func:`gated_delta_fwd`; slots, flags and padding rows as in :func:`linear_step`. Returns out."""
    with _Call(q, stream) as call:
        _on(call.index, "k v g beta state_cache state_indices has_initial_state out", k, v, g, beta, state_cache, state_indices,
            has_initial_state, out)
        if out is None:
            out = _like(v)
        a = make_gated_delta_args(q, k, v, g, beta, scale=scale, normalize=normalize, state_cache=state_cache,
                                  state_indices=state_indices, has_initial_state=has_initial_state, out=out,
                                  state_k_first=state_k_first)
        _check(_lib.load().kda_gated_delta_step(_context(context, call.index), ctypes.byref(a), call.handle),
               "kda_gated_delta_step")
    return out
