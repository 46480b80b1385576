"""Linear attention with a decay for each head, and rotary positions.

``linear_fwd`` (prompts) and ``linear_step`` (single tokens) serve beside ``chunk_fwd`` with the
same packed bounds, state pool and slots; ``rotary`` turns q and k by their positions. All three
marshal tensors into the C ABI of ``libkda.so`` and enqueue its kernels on the current torch
stream; nothing synchronises and no metadata is built, so every call can be captured. They record no
gradient, and refuse inputs that require one while gradients are enabled.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib

__all__ = ["linear_fwd", "linear_step", "rotary", "rotary_frequencies"]

_STATE_DT = {torch.float32: _lib.KDA_F32, torch.float16: _lib.KDA_F16, torch.bfloat16: _lib.KDA_BF16}


# The calls are made once for each layer and token, where a kernel of a few microseconds waits for
# them: every check is a plain condition, and a message is made only when it fails.


def _packed(name, t):
    """[T, H, D] of a [T, H, D] or [1, T, H, D] tensor."""
    n = t.dim()
    if n == 3:
        return t
    if n == 4 and t.shape[0] == 1:
        return t[0]
    raise ValueError(f"{name} must be [T, H, D] (or [1, T, H, D]), got {tuple(t.shape)}")


def _strides(name, t, T, H, D):
    """Element strides between tokens and between heads, for tensors that are not contiguous (a call's
    fields left 0, 0 mean dense); dense ones stand in where the tensor has a single token or head (torch
    leaves those arbitrary). One stride of 0 shows a row as several."""
    st, sh, sd = t.stride()
    if sd != 1 and D != 1:
        raise ValueError(f"{name} must have adjacent elements along its last dimension")
    if H == 1:
        sh = D
    if T <= 1:
        st = H * D
    if st == 0 and sh == 0:
        raise ValueError(f"{name} must not be broadcast over both tokens and heads")
    return st, sh


def _on(index, names, *tensors):
    for i, t in enumerate(tensors):
        if t is not None and t.get_device() != index:
            raise ValueError(f"{names.split()[i]} must be on cuda:{index}, got {t.device}")


def _vector(name, t, n, dtypes):
    """A contiguous vector of n elements of one of the dtypes."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d)[6:] for d in dtypes)}, got {t.dtype}")
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} elements, got {tuple(t.shape)}")
    return t.data_ptr()


# The calls record nothing for autograd: rather than return results cut off from inputs that ask for a gradient, they
# refuse. The conditions are written out where they stand: a loop over the tensors takes half a microsecond.
_grads_on = torch.is_grad_enabled


def _refuse_gradient(advice=""):
    raise ValueError("an input requires a gradient, and the call records none: use torch.no_grad() or detach()" + advice)


_I32 = (torch.int32,)
_INTS = (torch.int32, torch.int64)
_BOOLS = (torch.bool, torch.uint8)
_BF16 = torch.bfloat16


def _fill_rotation(a, T, limit, positions, inv_freq, interleaved):
    """The rotary fields of either argument struct."""
    if positions is None or inv_freq is None:
        raise ValueError("rotary positions need both positions and inv_freq")
    if inv_freq.dtype != torch.float64:
        raise TypeError(f"inv_freq must be fp64, got {inv_freq.dtype}")
    if inv_freq.dim() != 1 or not inv_freq.is_contiguous() or not 1 <= inv_freq.shape[0] <= limit // 2:
        raise ValueError(f"inv_freq must be a contiguous vector of 1 to {limit // 2} frequencies")
    if positions.dim() == 2 and positions.shape[0] == 1:
        positions = positions[0]
    a.positions = _vector("positions", positions, T, _INTS)
    a.positions_i64 = positions.dtype == torch.int64
    a.rot_dim = 2 * inv_freq.shape[0]
    a.inv_freq = inv_freq.data_ptr()
    a.interleaved = bool(interleaved)


def make_linear_args(q, k, v, g, *, N=None, cu_seqlens=None, cu_seqlens_cpu=None, scale=None, initial_state=None,
                     final_state=None, state_cache=None, state_indices=None, has_initial_state=None, out=None,
                     state_k_first=False, positions=None, inv_freq=None, interleaved=False, rotary_factor=1.0,
                     seg_len=0) -> "_lib.LinearArgs":
    """Fill a ``kda_linear_args`` from tensors (no allocation), checking everything the C side
    cannot see: dtypes, shapes, strides and element counts."""
    if _grads_on() and (q.requires_grad or k.requires_grad or v.requires_grad or (g is not None and g.requires_grad) or
                        (state_cache is not None and state_cache.requires_grad) or (out is not None and out.requires_grad) or
                        (initial_state is not None and initial_state.requires_grad)):
        _refuse_gradient()
    q, k, v = _packed("q", q), _packed("k", k), _packed("v", v)
    T, H_qk, K = q.shape
    Tv, H, V = v.shape
    if k.shape != q.shape:
        raise ValueError("q and k must have the same shape")
    if Tv != T:
        raise ValueError("v must have q's token count")
    if H_qk < 1 or H % H_qk != 0 or H < 1:
        raise ValueError(f"q/k heads ({H_qk}) must divide v heads ({H})")
    if q.dtype != _BF16 or k.dtype != _BF16 or v.dtype != _BF16:
        raise TypeError(f"q, k and v must be bf16, got {q.dtype}, {k.dtype}, {v.dtype}")
    a = _lib.LinearArgs()
    if N is None:
        N = T
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
        if N < 1:
            raise ValueError("cu_seqlens must be an [N+1] vector with N >= 1")
        a.cu_seqlens = _vector("cu_seqlens", cu_seqlens, N + 1, _I32)
        if cu_seqlens_cpu is not None:
            if cu_seqlens_cpu.device.type != "cpu":
                raise TypeError("cu_seqlens_cpu must be a CPU int32 tensor")
            a.cu_seqlens_host = _vector("cu_seqlens_cpu", cu_seqlens_cpu, N + 1, _I32)
    a.T, a.N, a.H, a.H_qk, a.K, a.V = T, N, H, H_qk, K, V
    a.scale = 1.0 / math.sqrt(K) if scale is None else scale
    a.q, a.k, a.v = q.data_ptr(), k.data_ptr(), v.data_ptr()
    if not q.is_contiguous():
        a.q_stride_t, a.q_stride_h = _strides("q", q, T, H_qk, K)
    if not k.is_contiguous():
        a.k_stride_t, a.k_stride_h = _strides("k", k, T, H_qk, K)
    if not v.is_contiguous():
        a.v_stride_t, a.v_stride_h = _strides("v", v, T, H, V)
    if out is not None:
        out = _packed("out", out)
        if out.dtype != _BF16:
            raise TypeError(f"out must be bf16, got {out.dtype}")
        if out.shape != v.shape:
            raise ValueError(f"out must have v's shape {tuple(v.shape)}, got {tuple(out.shape)}")
        a.out = out.data_ptr()
        if not out.is_contiguous():
            a.out_stride_t, a.out_stride_h = _strides("out", out, T, H, V)
    if g is not None:
        n = g.dim()
        if n == 3 and g.shape[0] == 1:
            g, n = g[0], 2
        if g.dtype == torch.float32:
            a.g_dtype = _lib.KDA_F32
        elif g.dtype == _BF16:
            a.g_dtype = _lib.KDA_BF16
        else:
            raise TypeError(f"g must be fp32 or bf16, got {g.dtype}")
        if g.shape != ((T, H) if n == 2 else (H,)) or not g.is_contiguous():
            raise ValueError(f"g must be a contiguous [H] = {(H,)} or [T, H] = {(T, H)}, got {tuple(g.shape)}")
        a.g = g.data_ptr()
        a.g_per_token = n == 2
    if state_cache is not None:
        if state_cache.dtype not in _STATE_DT:
            raise TypeError("state_cache must be fp32, fp16 or bf16")
        rows, cols = (K, V) if state_k_first else (V, K)
        sizes = state_cache.shape
        if sizes[1:] != (H, rows, cols) or sizes[0] < 1:
            raise ValueError(f"state_cache must be [slots, {H}, {rows}, {cols}] with at least one slot")
        s0, s1, s2, s3 = state_cache.stride()
        plane = H * K * V
        if (H != 1 and s1 != K * V) or s2 != cols or s3 != 1:
            raise ValueError("each state_cache slot plane must be dense")
        if sizes[0] == 1:
            s0 = plane
        if s0 < plane:
            raise ValueError("state_cache stride(0) must be at least one H*V*K plane")
        a.state_dtype = _STATE_DT[state_cache.dtype]
        a.state_cache, a.num_slots, a.state_cache_stride0 = state_cache.data_ptr(), sizes[0], s0
        if state_indices is not None:
            a.state_indices = _vector("state_indices", state_indices, N, _I32)
        if has_initial_state is not None:
            a.has_initial_state = _vector("has_initial_state", has_initial_state, N, _BOOLS)
    elif state_indices is not None or has_initial_state is not None:
        raise ValueError("state_indices and has_initial_state belong to a state_cache")
    if initial_state is not None or final_state is not None:
        shape = (N, H, K, V) if state_k_first else (N, H, V, K)
        for name, st in (("initial_state", initial_state), ("final_state", final_state)):
            if st is None:
                continue
            if st.dtype not in _STATE_DT:
                raise TypeError(f"{name} must be fp32, fp16 or bf16")
            if st.shape != shape or not st.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {shape}, got {tuple(st.shape)}")
            a.state_dtype = _STATE_DT[st.dtype]
        if initial_state is not None:
            a.initial_state = initial_state.data_ptr()
        if final_state is not None:
            a.final_state = final_state.data_ptr()
            if initial_state is not None and initial_state.dtype != final_state.dtype:
                raise TypeError("final_state must have initial_state's dtype")
    if state_k_first:
        a.state_k_first = 1
    if positions is not None or inv_freq is not None:
        _fill_rotation(a, T, K, positions, inv_freq, interleaved)
        a.rot_factor = rotary_factor
    if seg_len:
        a.seg_len = seg_len
    return a


def _check(rc, where):
    if rc:
        from . import KDAError
        raise KDAError(rc, where)


_contexts = {}  # device index -> the device's shared context


def _context(context, index):
    if context is None:
        context = _contexts.get(index)
        if context is None:
            from . import get_context
            context = _contexts[index] = get_context(torch.device("cuda", index))
    elif context.device != index:
        raise ValueError(f"the context is device {context.device}'s, the tensors are on {index}")
    return context.ptr


# The current stream's handle; torch.cuda.current_stream makes an object of it in 2 us.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


class _Call:
    """The call's device current and its allocations on its stream. The guards cost more than a
    small kernel, so they are entered only where they change something."""

    __slots__ = ("device", "index", "handle", "guards")

    def __init__(self, q, stream):
        if not q.is_cuda:
            raise ValueError("inputs must be on a GPU")
        self.device = device = q.device
        self.index, self.guards = device.index, ()
        if torch.cuda.current_device() != self.index:
            self.guards += (torch.cuda.device(self.index),)
        if stream is None:
            self.handle = _raw_stream(self.index)
        else:
            if stream.device != device:
                raise ValueError(f"stream must be on {device}, got {stream.device}")
            self.guards += (torch.cuda.stream(stream),)
            self.handle = stream.cuda_stream

    def __enter__(self):
        for g in self.guards:
            g.__enter__()
        return self

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _like(t):
    """A dense tensor of t's shape, whatever t's strides."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


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
    rotated first, by the kernel of :func:`rotary` and, like its results, rounded to bf16
    (:func:`linear_step` keeps fp32). ``seg_len`` overrides the segment
    length policy (a multiple of 64). Returns ``(out, final_state)``, final_state None unless dense
    and asked for."""
    with _Call(q, stream) as call:
        _on(call.index, "k v g cu_seqlens initial_state state_cache state_indices has_initial_state out workspace positions "
            "inv_freq", k, v, g, cu_seqlens, initial_state, state_cache, state_indices, has_initial_state, out, workspace,
            positions, inv_freq)
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
        a = make_linear_args(q, k, v, g, cu_seqlens=cu_seqlens, cu_seqlens_cpu=cu_seqlens_cpu, scale=scale,
                             initial_state=initial_state, final_state=final_state, state_cache=state_cache,
                             state_indices=state_indices, has_initial_state=has_initial_state, out=out,
                             state_k_first=state_k_first, positions=positions, inv_freq=inv_freq,
                             interleaved=interleaved, rotary_factor=rotary_factor, seg_len=seg_len)
        lib = _lib.load()
        ref = ctypes.byref(a)
        need = lib.kda_linear_fwd_workspace_bytes(ref)  # 0 for a refused call too: the call says why
        if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()):
            raise TypeError("workspace must be a contiguous uint8 tensor")
        if need and (workspace is None or workspace.numel() < need):
            workspace = torch.empty(need, dtype=torch.uint8, device=call.device)
        _check(lib.kda_linear_fwd(_context(context, call.index), ref, workspace.data_ptr() if need else None, need, call.handle),
               "kda_linear_fwd")
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
    with _Call(q, stream) as call:
        _on(call.index, "k v g state_cache state_indices has_initial_state out positions inv_freq",
            k, v, g, state_cache, state_indices, has_initial_state, out, positions, inv_freq)
        if out is None:
            out = _like(v)
        a = make_linear_args(q, k, v, g, scale=scale, state_cache=state_cache,
                             state_indices=state_indices, has_initial_state=has_initial_state, out=out,
                             state_k_first=state_k_first, positions=positions, inv_freq=inv_freq,
                             interleaved=interleaved, rotary_factor=rotary_factor)
        _check(_lib.load().kda_linear_step(_context(context, call.index), ctypes.byref(a), call.handle), "kda_linear_step")
    return out


def make_rotary_args(q, k, positions, inv_freq, out_q, out_k, *, interleaved=False, factor=1.0, inverse=False) -> "_lib.RotaryArgs":
    """Fill a ``kda_rotary_args`` from tensors (no allocation), checking what the C side cannot see."""
    if _grads_on() and (q.requires_grad or out_q.requires_grad or (k is not None and k.requires_grad) or
                        (out_k is not None and out_k.requires_grad)):
        _refuse_gradient(" (the gradient is the call with inverse=True)")
    q, out_q = _packed("q", q), _packed("out_q", out_q)
    T, H, D = q.shape
    dtype = q.dtype
    a = _lib.RotaryArgs()
    if dtype not in _STATE_DT:
        raise TypeError(f"q must be fp32, fp16 or bf16, got {dtype}")
    if H < 1 or D < 2:
        raise ValueError("q must have heads and at least two channels")
    if (k is None) != (out_k is None):
        raise ValueError("out_k goes with k")
    if out_q.dtype != dtype or out_q.shape != q.shape:
        raise ValueError("out_q must have q's shape and dtype")
    a.T, a.H_q, a.D, a.dtype = T, H, D, _STATE_DT[dtype]
    a.q, a.out_q = q.data_ptr(), out_q.data_ptr()
    if not q.is_contiguous():
        a.q_stride_t, a.q_stride_h = _strides("q", q, T, H, D)
    if not out_q.is_contiguous():
        a.out_q_stride_t, a.out_q_stride_h = _strides("out_q", out_q, T, H, D)
    if k is not None:
        k, out_k = _packed("k", k), _packed("out_k", out_k)
        Tk, Hk, Dk = k.shape
        if k.dtype != dtype:
            raise TypeError("q and k must have the same dtype")
        if Tk != T or Dk != D:
            raise ValueError("k must have q's token count and head size")
        if out_k.dtype != dtype or out_k.shape != k.shape:
            raise ValueError("out_k must have k's shape and dtype")
        a.H_k, a.k, a.out_k = Hk, k.data_ptr(), out_k.data_ptr()
        if not k.is_contiguous():
            a.k_stride_t, a.k_stride_h = _strides("k", k, T, Hk, D)
        if not out_k.is_contiguous():
            a.out_k_stride_t, a.out_k_stride_h = _strides("out_k", out_k, T, Hk, D)
    _fill_rotation(a, T, D, positions, inv_freq, interleaved)
    a.factor = factor
    if inverse:
        a.inverse = 1
    return a


def rotary(q, k, positions, inv_freq, *, interleaved=False, factor=1.0, inverse=False, out_q=None, out_k=None,
           stream=None, context=None):
    """q and k turned by their positions, as one kernel.

    q: ``[T, H_q, D]``, k: ``[T, H_k, D]`` or None (or with a leading 1), bf16, fp16 or fp32, rows may
    be strided. positions: int32 or int64 ``[T]``. inv_freq: fp64 vector of up to D/2 frequencies
    (radians per position, :func:`rotary_frequencies`); with r twice its length, pair i is channels
    ``(i, i + r/2)``, or ``(2i, 2i + 1)`` when ``interleaved``; channels from r on pass through.
    ``factor`` scales the rotated channels. ``inverse`` applies the transposed rotation: the gradient
    with respect to q and k, given the results' gradients (the call itself records none, so a training program makes both
    calls under ``torch.no_grad()``, or in the two halves of an autograd function). ``out_q`` / ``out_k`` may be q / k
    themselves (in place) or share no element with either. Returns ``(out_q, out_k)``."""
    with _Call(q, stream) as call:
        _on(call.index, "k positions inv_freq out_q out_k", k, positions, inv_freq, out_q, out_k)
        if out_q is None:
            out_q = _like(q)
        if out_k is None and k is not None:
            out_k = _like(k)
        a = make_rotary_args(q, k, positions, inv_freq, out_q, out_k, interleaved=interleaved, factor=factor, inverse=inverse)
        _check(_lib.load().kda_rotary(_context(context, call.index), ctypes.byref(a), call.handle), "kda_rotary")
    return out_q, out_k


def _need(cond, msg):
    if not cond:
        raise ValueError(msg)


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
