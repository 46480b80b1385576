"""Linear attention with a decay for each head, and rotary positions.

``linear_fwd`` (prompts) and ``linear_step`` (single tokens) serve beside ``chunk_fwd`` with the
same packed bounds, state pool and slots; ``rotary`` turns q and k by their positions. All three
marshal tensors into the C ABI of ``libkda.so`` and enqueue its kernels on the current torch
stream; nothing synchronises and no metadata is built, so every call can be captured.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib

__all__ = ["linear_fwd", "linear_step", "rotary", "rotary_frequencies"]

_STATE_DT = {torch.float32: _lib.KDA_F32, torch.float16: _lib.KDA_F16, torch.bfloat16: _lib.KDA_BF16}


def _need(cond, msg, exc=ValueError):
    if not cond:
        raise exc(msg)


def _packed(name, t):
    """[T, H, D] of a [T, H, D] or [1, T, H, D] tensor."""
    if t.dim() == 4 and t.shape[0] == 1:
        t = t[0]
    _need(t.dim() == 3, f"{name} must be [T, H, D] (or [1, T, H, D]), got {tuple(t.shape)}")
    return t


def _strides(name, t):
    """Element strides between tokens and between heads; dense ones stand in where the tensor has
    a single token or head (torch leaves those arbitrary)."""
    T, H, D = t.shape
    st, sh, sd = t.stride()
    _need(sd == 1 or D == 1, f"{name} must have adjacent elements along its last dimension")
    if H == 1:
        sh = D
    if T <= 1:
        st = H * sh
    return st, sh


def _on(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}, got {t.device}")


def _fill_rotation(a, T, limit, positions, inv_freq, interleaved, factor):
    """The rotary fields of either argument struct."""
    _need(positions is not None and inv_freq is not None, "rotary positions need both positions and inv_freq")
    _need(inv_freq.dtype == torch.float64, f"inv_freq must be fp64, got {inv_freq.dtype}", TypeError)
    _need(inv_freq.dim() == 1 and inv_freq.is_contiguous() and 1 <= inv_freq.numel() <= limit // 2,
          f"inv_freq must be a contiguous vector of 1 to {limit // 2} frequencies")
    _need(positions.dtype in (torch.int32, torch.int64), f"positions must be int32 or int64, got {positions.dtype}", TypeError)
    if positions.dim() == 2 and positions.shape[0] == 1:
        positions = positions[0]
    _need(positions.dim() == 1 and positions.is_contiguous() and positions.numel() == T,
          f"positions must be a contiguous vector of T = {T} elements")
    a.rot_dim = 2 * inv_freq.numel()
    a.inv_freq = inv_freq.data_ptr()
    a.positions = positions.data_ptr()
    a.positions_i64 = 1 if positions.dtype == torch.int64 else 0
    a.interleaved = 1 if interleaved else 0
    return float(factor)


def make_linear_args(q, k, v, g, *, N=None, cu_seqlens=None, cu_seqlens_cpu=None, scale=None, initial_state=None,
                     final_state=None, state_cache=None, state_indices=None, has_initial_state=None, out=None,
                     state_k_first=False, positions=None, inv_freq=None, interleaved=False, rotary_factor=1.0,
                     seg_len=0) -> "_lib.LinearArgs":
    """Fill a ``kda_linear_args`` from tensors (no allocation), checking everything the C side
    cannot see: dtypes, shapes, strides and element counts."""
    q, k, v = _packed("q", q), _packed("k", k), _packed("v", v)
    T, H_qk, K = q.shape
    H, V = v.shape[1], v.shape[2]
    _need(k.shape == q.shape, "q and k must have the same shape")
    _need(v.shape[0] == T, "v must have q's token count")
    _need(0 < H_qk <= H and H % H_qk == 0, f"q/k heads ({H_qk}) must divide v heads ({H})")
    a = _lib.LinearArgs()
    if cu_seqlens is not None:
        _need(cu_seqlens.dtype == torch.int32, "cu_seqlens must be int32", TypeError)
        _need(cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 2 and cu_seqlens.is_contiguous(),
              "cu_seqlens must be a contiguous [N+1] vector with N >= 1")
        N = cu_seqlens.numel() - 1
        a.cu_seqlens = cu_seqlens.data_ptr()
        if cu_seqlens_cpu is not None:
            _need(cu_seqlens_cpu.device.type == "cpu" and cu_seqlens_cpu.dtype == torch.int32,
                  "cu_seqlens_cpu must be a CPU int32 tensor", TypeError)
            _need(cu_seqlens_cpu.is_contiguous() and cu_seqlens_cpu.numel() == N + 1,
                  "cu_seqlens_cpu must be contiguous with N+1 elements, like cu_seqlens")
            a.cu_seqlens_host = cu_seqlens_cpu.data_ptr()
    a.T, a.N, a.H, a.H_qk, a.K, a.V = T, N, H, H_qk, K, V
    a.scale = 1.0 / math.sqrt(K) if scale is None else float(scale)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t.dtype == torch.bfloat16, f"{name} must be bf16, got {t.dtype}", TypeError)
    a.q, a.k, a.v = q.data_ptr(), k.data_ptr(), v.data_ptr()
    a.q_stride_t, a.q_stride_h = _strides("q", q)
    a.k_stride_t, a.k_stride_h = _strides("k", k)
    a.v_stride_t, a.v_stride_h = _strides("v", v)
    if out is not None:
        out = _packed("out", out)
        _need(out.dtype == torch.bfloat16, f"out must be bf16, got {out.dtype}", TypeError)
        _need(out.shape == v.shape, f"out must have v's shape {tuple(v.shape)}, got {tuple(out.shape)}")
        a.out = out.data_ptr()
        a.out_stride_t, a.out_stride_h = _strides("out", out)
    if g is not None:
        _need(g.dtype in (torch.float32, torch.bfloat16), f"g must be fp32 or bf16, got {g.dtype}", TypeError)
        if g.dim() == 3 and g.shape[0] == 1:
            g = g[0]
        per_token = g.dim() == 2
        _need(tuple(g.shape) == ((T, H) if per_token else (H,)),
              f"g must be [H] = {(H,)} or [T, H] = {(T, H)}, got {tuple(g.shape)}")
        _need(g.is_contiguous(), "g must be contiguous")
        a.g = g.data_ptr()
        a.g_dtype = _STATE_DT[g.dtype]
        a.g_per_token = 1 if per_token else 0
    plane = (H, K, V) if state_k_first else (H, V, K)
    for name, st in (("initial_state", initial_state), ("final_state", final_state)):
        if st is None:
            continue
        _need(st.dtype in _STATE_DT, f"{name} must be fp32, fp16 or bf16", TypeError)
        _need(tuple(st.shape) == (N, *plane), f"{name} must be {(N, *plane)}, got {tuple(st.shape)}")
        _need(st.is_contiguous(), f"{name} must be contiguous")
        a.state_dtype = _STATE_DT[st.dtype]
    if initial_state is not None and final_state is not None:
        _need(initial_state.dtype == final_state.dtype, "final_state must have initial_state's dtype", TypeError)
    a.initial_state = None if initial_state is None else initial_state.data_ptr()
    a.final_state = None if final_state is None else final_state.data_ptr()
    if state_cache is not None:
        _need(state_cache.dtype in _STATE_DT, "state_cache must be fp32, fp16 or bf16", TypeError)
        _need(state_cache.dim() == 4 and tuple(state_cache.shape[1:]) == plane and state_cache.shape[0] >= 1,
              f"state_cache must be [slots, {', '.join(map(str, plane))}] with at least one slot")
        sizes, strides = state_cache.shape, state_cache.stride()
        _need((H == 1 or strides[1] == K * V) and strides[2:] == (sizes[3], 1), "each state_cache slot plane must be dense")
        stride0 = H * K * V if sizes[0] == 1 else strides[0]
        _need(stride0 >= H * K * V, "state_cache stride(0) must be at least one H*V*K plane")
        a.state_dtype = _STATE_DT[state_cache.dtype]
        a.state_cache, a.num_slots, a.state_cache_stride0 = state_cache.data_ptr(), sizes[0], stride0
        if state_indices is not None:
            _need(state_indices.dtype == torch.int32, f"state_indices must be int32, got {state_indices.dtype}", TypeError)
            _need(state_indices.dim() == 1 and state_indices.is_contiguous() and state_indices.numel() == N,
                  f"state_indices must be a contiguous vector of N = {N} elements")
            a.state_indices = state_indices.data_ptr()
        if has_initial_state is not None:
            _need(has_initial_state.dtype in (torch.bool, torch.uint8),
                  f"has_initial_state must be bool or uint8, got {has_initial_state.dtype}", TypeError)
            _need(has_initial_state.dim() == 1 and has_initial_state.is_contiguous() and has_initial_state.numel() == N,
                  f"has_initial_state must be a contiguous vector of N = {N} elements")
            a.has_initial_state = has_initial_state.data_ptr()
    else:
        _need(state_indices is None and has_initial_state is None, "state_indices and has_initial_state belong to a state_cache")
    a.state_k_first = 1 if state_k_first else 0
    if positions is not None or inv_freq is not None:
        a.rot_factor = _fill_rotation(a, T, K, positions, inv_freq, interleaved, rotary_factor)
    a.seg_len = int(seg_len)
    return a


def _enter(q, stream):
    """(device index, stream handle) of a call on q's device."""
    device = q.device
    if device.type != "cuda":
        raise ValueError("inputs must be on a GPU")
    return device.index, (torch.cuda.current_stream(device) if stream is None else stream).cuda_stream


def _context(context, index):
    if context is not None:
        _need(context.device == index, f"the context is device {context.device}'s, the tensors are on {index}")
        return context.ptr
    from . import get_context
    return get_context(torch.device("cuda", index)).ptr


def _check(rc, where):
    if rc != _lib.KDA_OK:
        from . import KDAError
        raise KDAError(rc, where)


class _On:
    """The call's device current, and its allocations on its stream (entered only where that differs
    from what is current already: the guards cost more than a small kernel)."""

    def __init__(self, index, stream):
        self.guards = []
        if torch.cuda.current_device() != index:
            self.guards.append(torch.cuda.device(index))
        if stream is not None:
            self.guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def linear_fwd(q, k, v, g, cu_seqlens, *, cu_seqlens_cpu=None, scale=None, initial_state=None,
               output_final_state=False, state_cache=None, state_indices=None, has_initial_state=None, out=None,
               workspace=None, stream=None, context=None, state_k_first=False, positions=None, inv_freq=None,
               interleaved=False, rotary_factor=1.0, seg_len=0):
    """Linear attention with a decay for each head over packed prompts:
    ``S_t = e^{g_t} S_{t-1} + v_t k_t^T``, ``o_t = scale S_t q_t``.

    q, k: bf16 ``[T, H_qk, K]``, v: bf16 ``[T, H, V]`` (or with a leading 1), K and V 64 or 128,
    H_qk dividing H; rows may be strided (parts of one projection's output). g: log decays, fp32 or
    bf16, ``[H]`` (constant) or ``[T, H]``, or None for no decay. cu_seqlens: int32 ``[N+1]`` on the
    device; rows from ``cu_seqlens[N]`` on are left as they were. The optional CPU copy is checked.

    State as in ``chunk_fwd``: dense ``initial_state`` (``[N, H, V, K]``) with
    ``output_final_state``, or a paged ``state_cache`` with ``state_indices`` and
    ``has_initial_state``, updated in place (a slot outside the pool: no slot); ``state_k_first``
    for ``[K, V]`` planes.

    With ``positions`` (``[T]``) and ``inv_freq`` (fp64, see :func:`rotary_frequencies`) q and k are
    rotated first, in bf16, by the kernel of :func:`rotary`. ``seg_len`` overrides the segment
    length policy (a multiple of 64). Returns ``(out, final_state)``, final_state None unless dense
    and asked for."""
    index, handle = _enter(q, stream)
    _on(q.device, k=k, v=v, g=g, cu_seqlens=cu_seqlens, initial_state=initial_state, state_cache=state_cache,
        state_indices=state_indices, has_initial_state=has_initial_state, out=out, workspace=workspace,
        positions=positions, inv_freq=inv_freq)
    _need(cu_seqlens is not None, "cu_seqlens is required")
    with _On(index, stream):
        if out is None:
            out = torch.empty(v.shape, dtype=v.dtype, device=v.device)
        final_state = None
        if output_final_state and state_cache is None:
            H, V, K = v.shape[-2], v.shape[-1], q.shape[-1]
            dt = initial_state.dtype if initial_state is not None else torch.float32
            planes = (K, V) if state_k_first else (V, K)
            final_state = torch.empty((cu_seqlens.numel() - 1, H, *planes), dtype=dt, device=q.device)
        a = make_linear_args(q, k, v, g, cu_seqlens=cu_seqlens, cu_seqlens_cpu=cu_seqlens_cpu, scale=scale,
                             initial_state=initial_state, final_state=final_state, state_cache=state_cache,
                             state_indices=state_indices, has_initial_state=has_initial_state, out=out,
                             state_k_first=state_k_first, positions=positions, inv_freq=inv_freq,
                             interleaved=interleaved, rotary_factor=rotary_factor, seg_len=seg_len)
        lib = _lib.load()
        ref = ctypes.byref(a)
        _check(lib.kda_linear_fwd_validate(ref), "kda_linear_fwd_validate")
        need = lib.kda_linear_fwd_workspace_bytes(ref)
        if workspace is not None:
            _need(workspace.dtype == torch.uint8 and workspace.is_contiguous(),
                  "workspace must be a contiguous uint8 tensor", TypeError)
        if need and (workspace is None or workspace.numel() < need):
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        ptr, size = (workspace.data_ptr(), workspace.numel()) if need else (None, 0)
        _check(lib.kda_linear_fwd(_context(context, index), ref, ptr, size, handle), "kda_linear_fwd")
    return out, final_state


def linear_step(q, k, v, g, *, state_cache, state_indices=None, has_initial_state=None, scale=None, out=None,
                stream=None, context=None, state_k_first=False, positions=None, inv_freq=None, interleaved=False,
                rotary_factor=1.0):
    """One token of each of N requests: ``S <- e^g S + v k^T``, ``o = scale S q``.

    q, k: bf16 ``[N, H_qk, K]``, v: ``[N, H, V]``, g as in :func:`linear_fwd` (``[H]``, ``[N, H]`` or
    None). Row n's state is slot ``state_indices[n]`` of ``state_cache`` (slot n without indices),
    updated in place; a row whose index is outside the pool is padding, its row of ``out`` and every
    state left as they were. ``has_initial_state`` false: the slot is taken as zero and not read.
    With ``positions`` and ``inv_freq`` the kernel rotates q and k itself, in fp32. Returns out."""
    index, handle = _enter(q, stream)
    _on(q.device, k=k, v=v, g=g, state_cache=state_cache, state_indices=state_indices,
        has_initial_state=has_initial_state, out=out, positions=positions, inv_freq=inv_freq)
    with _On(index, stream):
        if out is None:
            out = torch.empty(v.shape, dtype=v.dtype, device=v.device)
        a = make_linear_args(q, k, v, g, N=q.shape[-3], scale=scale, state_cache=state_cache,
                             state_indices=state_indices, has_initial_state=has_initial_state, out=out,
                             state_k_first=state_k_first, positions=positions, inv_freq=inv_freq,
                             interleaved=interleaved, rotary_factor=rotary_factor)
        _check(_lib.load().kda_linear_step(_context(context, index), ctypes.byref(a), handle), "kda_linear_step")
    return out


_ROTARY_DT = _STATE_DT


def make_rotary_args(q, k, positions, inv_freq, out_q, out_k, *, interleaved=False, factor=1.0, inverse=False) -> "_lib.RotaryArgs":
    """Fill a ``kda_rotary_args`` from tensors (no allocation), checking what the C side cannot see."""
    q, out_q = _packed("q", q), _packed("out_q", out_q)
    T, H, D = q.shape
    a = _lib.RotaryArgs()
    _need(q.dtype in _ROTARY_DT, f"q must be fp32, fp16 or bf16, got {q.dtype}", TypeError)
    _need(H >= 1 and D >= 2, "q must have heads and at least two channels")
    _need((k is None) == (out_k is None), "out_k goes with k")
    _need(out_q.dtype == q.dtype and out_q.shape == q.shape, "out_q must have q's shape and dtype")
    a.T, a.H_q, a.D, a.dtype = T, H, D, _ROTARY_DT[q.dtype]
    a.q, a.out_q = q.data_ptr(), out_q.data_ptr()
    a.q_stride_t, a.q_stride_h = _strides("q", q)
    a.out_q_stride_t, a.out_q_stride_h = _strides("out_q", out_q)
    if k is not None:
        k, out_k = _packed("k", k), _packed("out_k", out_k)
        _need(k.dtype == q.dtype, "q and k must have the same dtype", TypeError)
        _need(k.shape[0] == T and k.shape[2] == D, "k must have q's token count and head size")
        _need(out_k.dtype == k.dtype and out_k.shape == k.shape, "out_k must have k's shape and dtype")
        a.H_k, a.k, a.out_k = k.shape[1], k.data_ptr(), out_k.data_ptr()
        a.k_stride_t, a.k_stride_h = _strides("k", k)
        a.out_k_stride_t, a.out_k_stride_h = _strides("out_k", out_k)
    a.factor = _fill_rotation(a, T, D, positions, inv_freq, interleaved, factor)
    a.inverse = 1 if inverse else 0
    return a


def rotary(q, k, positions, inv_freq, *, interleaved=False, factor=1.0, inverse=False, out_q=None, out_k=None,
           stream=None, context=None):
    """q and k turned by their positions, as one kernel.

    q: ``[T, H_q, D]``, k: ``[T, H_k, D]`` or None (or with a leading 1), bf16, fp16 or fp32, rows may
    be strided. positions: int32 or int64 ``[T]``. inv_freq: fp64 vector of up to D/2 frequencies
    (radians per position, :func:`rotary_frequencies`); with r twice its length, pair i is channels
    ``(i, i + r/2)``, or ``(2i, 2i + 1)`` when ``interleaved``; channels from r on pass through.
    ``factor`` scales the rotated channels. ``inverse`` applies the transposed rotation: the gradient
    with respect to q and k, given the results' gradients. ``out_q`` / ``out_k`` may be q / k
    themselves (in place). Returns ``(out_q, out_k)``."""
    index, handle = _enter(q, stream)
    _on(q.device, k=k, positions=positions, inv_freq=inv_freq, out_q=out_q, out_k=out_k)
    with _On(index, stream):
        if out_q is None:
            out_q = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if out_k is None and k is not None:
            out_k = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        a = make_rotary_args(q, k, positions, inv_freq, out_q, out_k, interleaved=interleaved, factor=factor, inverse=inverse)
        _check(_lib.load().kda_rotary(_context(context, index), ctypes.byref(a), handle), "kda_rotary")
    return out_q, out_k


def rotary_frequencies(rot_dim, *, base=10000.0, scaling=None, scale=1.0, original_length=None, beta_fast=32.0,
                       beta_slow=1.0, device=None):
    """``(inv_freq, factor)`` for :func:`rotary`: fp64 frequencies ``base^{-2i/rot_dim}`` for
    ``rot_dim`` rotated channels, for a context ``scale`` times as long as the trained one.

    scaling: None; "linear" (positions shrink by ``scale``); "ntk" (a larger base, ``base *
    scale^{d/(d-2)}``: the slowest frequency shrinks by ``scale``, the fastest stays); "yarn" (per
    frequency: kept where it turns more than ``beta_fast`` times over ``original_length`` tokens,
    shrunk by ``scale`` where it turns less than ``beta_slow`` times, a linear ramp over i between;
    factor ``0.1 ln(scale) + 1``). factor is 1 otherwise."""
    rot_dim = int(rot_dim)
    _need(rot_dim >= 2 and rot_dim % 2 == 0, "rot_dim must be even and at least 2")
    _need(base > 1.0 and math.isfinite(base), "base must be finite and above 1")
    _need(scale >= 1.0 and math.isfinite(scale), "scale must be finite and at least 1")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    freq = float(base) ** (-2.0 * i / rot_dim)
    factor = 1.0
    if scaling == "linear":
        freq = freq / scale
    elif scaling == "ntk":
        _need(rot_dim > 2, "ntk scaling needs at least two frequencies")
        freq = (base * scale ** (rot_dim / (rot_dim - 2))) ** (-2.0 * i / rot_dim)
    elif scaling == "yarn":
        _need(original_length is not None and original_length >= 1, "yarn scaling needs original_length")
        _need(beta_fast > beta_slow > 0, "yarn scaling needs beta_fast > beta_slow > 0")
        # The (real) frequency index that turns `turns` times over the original length.
        def at(turns):
            return rot_dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(beta_fast)), 0), min(math.ceil(at(beta_slow)), rot_dim - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        freq = freq * (1 - ramp) + freq / scale * ramp
        factor = 0.1 * math.log(scale) + 1.0
    else:
        _need(scaling is None, f"unknown scaling {scaling!r}: None, 'linear', 'ntk' or 'yarn'")
        _need(scale == 1.0, "scale needs a scaling")
    return freq.to(device) if device is not None else freq, factor
