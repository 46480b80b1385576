"""Norms of q and k for each head, with the position rotation in the same pass, and their gradient.

``qk_norm`` stands in front of ``linear_fwd``, ``gated_delta_fwd`` or any attention; ``qk_norm_backward`` is its gradient as a
call of its own, as ``rotary(..., inverse=True)`` is the rotation's. Both enqueue kernels of ``libkda.so`` on the current
torch stream, synchronise nothing and can be captured; they record no gradient, and refuse inputs that require one while
gradients are enabled, or that carry a forward-mode tangent.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .linear import (_STATE_DT, _Call, _check, _context, _fill_rotation, _grads_on, _like, _on, _packed, _refuse_gradient,
                     _refuse_tangents, _strides, _tangents_on)

__all__ = ["qk_norm", "qk_norm_backward"]

_KINDS = {"rms": _lib.KDA_NORM_RMS, "l2": _lib.KDA_NORM_L2}
_ADVICE = " (the gradient is qk_norm_backward)"


def _weight(name, w, D, dtype):
    if w.dtype != dtype and w.dtype != torch.float32:
        raise TypeError(f"{name} must be fp32 or of q's dtype {dtype}, got {w.dtype}")
    if w.dim() != 1 or w.shape[0] != D or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {D} elements, got {tuple(w.shape)}")
    return w.data_ptr()


def _weight_gradient(name, grad, w):
    if grad.dtype != w.dtype or grad.shape != w.shape or not grad.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector like the weight")
    return grad.data_ptr()


def make_qk_norm_args(q, k, q_weight, k_weight, positions, inv_freq, out_q, out_k, *, grad_q=None, grad_k=None,
                      grad_q_weight=None, grad_k_weight=None, kind="rms", eps=1e-6, weight_offset=0.0,
                      interleaved=False) -> "_lib.QkNormArgs":
    """Fill a ``kda_qk_norm_args`` from tensors (no allocation), checking what the C side cannot see."""
    if _grads_on() and (q.requires_grad or out_q.requires_grad or (k is not None and k.requires_grad) or
                        (out_k is not None and out_k.requires_grad) or (q_weight is not None and q_weight.requires_grad) or
                        (k_weight is not None and k_weight.requires_grad) or (grad_q is not None and grad_q.requires_grad) or
                        (grad_k is not None and grad_k.requires_grad)):
        _refuse_gradient(_ADVICE)
    if _tangents_on():
        _refuse_tangents(q, k, q_weight, k_weight, out_q, out_k, grad_q, grad_k)
    q, out_q = _packed("q", q), _packed("out_q", out_q)
    shape, dtype = q.shape, q.dtype
    T, H, D = shape
    a = _lib.QkNormArgs()
    if dtype not in _STATE_DT:
        raise TypeError(f"q must be fp32, fp16 or bf16, got {dtype}")
    if H < 1 or D < 1:
        raise ValueError("q must have heads and channels")
    if (k is None) != (out_k is None):
        raise ValueError("out_k goes with k")
    if out_q.dtype != dtype or out_q.shape != shape:
        raise ValueError("out_q must have q's shape and dtype")
    a.T, a.H_q, a.D, a.dtype = T, H, D, _STATE_DT[dtype]
    a.q, a.out_q = q.data_ptr(), out_q.data_ptr()
    if not q.is_contiguous():
        a.q_stride_t, a.q_stride_h = _strides("q", q, T, H, D)
    if not out_q.is_contiguous():
        a.out_q_stride_t, a.out_q_stride_h = _strides("out_q", out_q, T, H, D)
    if grad_q is not None:
        grad_q = _packed("grad_q", grad_q)
        if grad_q.dtype != dtype or grad_q.shape != shape:
            raise ValueError("grad_q must have q's shape and dtype")
        a.grad_q = grad_q.data_ptr()
        if not grad_q.is_contiguous():
            a.grad_q_stride_t, a.grad_q_stride_h = _strides("grad_q", grad_q, T, H, D)
    if k is not None:
        k, out_k = _packed("k", k), _packed("out_k", out_k)
        shape = k.shape
        Tk, Hk, Dk = shape
        if k.dtype != dtype:
            raise TypeError("q and k must have the same dtype")
        if Tk != T or Dk != D:
            raise ValueError("k must have q's token count and head size")
        if out_k.dtype != dtype or out_k.shape != shape:
            raise ValueError("out_k must have k's shape and dtype")
        a.H_k, a.k, a.out_k = Hk, k.data_ptr(), out_k.data_ptr()
        if not k.is_contiguous():
            a.k_stride_t, a.k_stride_h = _strides("k", k, T, Hk, D)
        if not out_k.is_contiguous():
            a.out_k_stride_t, a.out_k_stride_h = _strides("out_k", out_k, T, Hk, D)
        if grad_k is not None:
            grad_k = _packed("grad_k", grad_k)
            if grad_k.dtype != dtype or grad_k.shape != shape:
                raise ValueError("grad_k must have k's shape and dtype")
            a.grad_k = grad_k.data_ptr()
            if not grad_k.is_contiguous():
                a.grad_k_stride_t, a.grad_k_stride_h = _strides("grad_k", grad_k, T, Hk, D)
    elif k_weight is not None:
        raise ValueError("k_weight goes with k")
    if q_weight is not None:
        a.q_weight, a.weight_dtype = _weight("q_weight", q_weight, D, dtype), _STATE_DT[q_weight.dtype]
        if grad_q_weight is not None:
            a.grad_q_weight = _weight_gradient("grad_q_weight", grad_q_weight, q_weight)
        if k_weight is not None and q_weight.dtype != k_weight.dtype:
            raise TypeError("q_weight and k_weight must have the same dtype")
    if k_weight is not None:
        a.k_weight, a.weight_dtype = _weight("k_weight", k_weight, D, dtype), _STATE_DT[k_weight.dtype]
        if grad_k_weight is not None:
            a.grad_k_weight = _weight_gradient("grad_k_weight", grad_k_weight, k_weight)
    if positions is not None or inv_freq is not None:
        _fill_rotation(a, T, D, positions, inv_freq, interleaved)
    elif interleaved:
        a.interleaved = 1
    if kind != "rms":
        if kind not in _KINDS:
            raise ValueError(f"unknown kind {kind!r}: 'rms' or 'l2'")
        a.kind = _KINDS[kind]
    a.eps, a.weight_offset = eps, weight_offset
    return a


def qk_norm(q, k, q_weight=None, k_weight=None, positions=None, inv_freq=None, *, kind="rms", eps=1e-6, weight_offset=0.0,
            interleaved=False, out_q=None, out_k=None, stream=None, context=None):
    """Every row (one head of one token) of q and k normalised, weighted and turned by its position, as one kernel:
    ``R(position) [x / sqrt(m sum x^2 + eps) * (weight_offset + weight)]``.

    q: ``[T, H_q, D]``, k: ``[T, H_k, D]`` or None (or with a leading 1), bf16, fp16 or fp32, D up to 1024, rows may be
    strided. kind: "rms" (m = 1 / D) or "l2" (m = 1: rows of unit length). q_weight, k_weight: vectors of D, in fp32 or q's
    dtype, or None (no weight; ``weight_offset`` 1 is for weights stored as their distance from 1). positions (``[T]``)
    and inv_freq as in :func:`rotary`; without them nothing is turned. ``out_q`` / ``out_k`` may be q / k themselves (in
    place) or share no element with either. Returns ``(out_q, out_k)``."""
    with _Call(q, stream) as call:
        _on(call.index, "k q_weight k_weight positions inv_freq out_q out_k", k, q_weight, k_weight, positions, inv_freq, out_q, out_k)
        if out_q is None:
            out_q = _like(q)
        if out_k is None and k is not None:
            out_k = _like(k)
        a = make_qk_norm_args(q, k, q_weight, k_weight, positions, inv_freq, out_q, out_k, kind=kind, eps=eps,
                              weight_offset=weight_offset, interleaved=interleaved)
        _check(_lib.load().kda_qk_norm(_context(context, call.index), ctypes.byref(a), call.handle), "kda_qk_norm")
    return out_q, out_k


def qk_norm_backward(grad_q, grad_k, q, k, q_weight=None, k_weight=None, positions=None, inv_freq=None, *, kind="rms",
                     eps=1e-6, weight_offset=0.0, interleaved=False, out_q=None, out_k=None, workspace=None, stream=None,
                     context=None):
    """The gradient of :func:`qk_norm`: given the results' gradients and the call's inputs, ``(dq, dk, dq_weight,
    dk_weight)``, of the inputs' types (None for an input that is None). Weight gradients are summed over all
    rows in fp32 and rounded once. ``out_q`` / ``out_k`` may be grad_q / grad_k themselves, or share no element with any
    input. ``workspace``, for weight gradients: as in :func:`gated_delta_fwd`, at most 4096 bytes for each channel. A training program calls both under ``torch.no_grad()``, or in the two halves of an autograd function."""
    with _Call(q, stream) as call:
        _on(call.index, "grad_q grad_k k q_weight k_weight positions inv_freq out_q out_k workspace", grad_q, grad_k, k, q_weight,
            k_weight, positions, inv_freq, out_q, out_k, workspace)
        if grad_q is None or (grad_k is None) != (k is None):
            raise ValueError("grad_q is required, and grad_k goes with k")
        if out_q is None:
            out_q = _like(q)
        if out_k is None and k is not None:
            out_k = _like(k)
        dqw = torch.empty_like(q_weight) if q_weight is not None else None
        dkw = torch.empty_like(k_weight) if k_weight is not None else None
        a = make_qk_norm_args(q, k, q_weight, k_weight, positions, inv_freq, out_q, out_k, grad_q=grad_q, grad_k=grad_k,
                              grad_q_weight=dqw, grad_k_weight=dkw, kind=kind, eps=eps, weight_offset=weight_offset,
                              interleaved=interleaved)
        lib = _lib.load()
        ref = ctypes.byref(a)
        need = lib.kda_qk_norm_backward_workspace_bytes(ref)  # 0 for a refused call too: the call says why
        if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()):
            raise TypeError("workspace must be a contiguous uint8 tensor")
        if need and workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=call.device)
        given = (workspace.data_ptr(), workspace.numel()) if need else (None, 0)
        _check(lib.kda_qk_norm_backward(_context(context, call.index), ref, *given, call.handle), "kda_qk_norm_backward")
    return out_q, out_k, dqw, dkw
