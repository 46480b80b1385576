"""CPU tests of the q/k norm's entry points (no GPU): argument checks of the C ABI and of the binding, workspace, launches through a
recording fake runtime, and the oracle's gradient against differences."""
import ctypes
import math

import numpy as np
import pytest
import torch

import gated_delta_rule_pack_amd as kda
from gated_delta_rule_pack_amd import _lib
from oracle import qk_norm, qk_norm_gradient
from tests.test_abi_cpu import FakeBufs
from tests.test_linear_cpu import ALIAS, INV, UNS, _set, fake, lib  # noqa: F401 (fixtures)

ROWS = ("q", "k", "out_q", "out_k")


def _norm(b, T=10, Hq=4, Hk=2, D=64, back=False, weight=True):
    a = _lib.QkNormArgs()
    a.T, a.H_q, a.H_k, a.D, a.rot_dim, a.dtype, a.weight_dtype, a.eps = T, Hq, Hk, D, 32, _lib.KDA_BF16, _lib.KDA_F32, 1e-6
    for n in ROWS + (("grad_q", "grad_k") if back else ()):
        setattr(a, n, b.buf(T * (Hq if n.endswith("q") else max(Hk, 1)) * D * 2).ctypes.data)
    a.positions, a.inv_freq = b.buf(4 * T).ctypes.data, b.buf(8 * 16).ctypes.data
    if weight:
        for n in ("q_weight", "k_weight") + (("grad_q_weight", "grad_k_weight") if back else ()):
            setattr(a, n, b.buf(4 * D).ctypes.data)
    return a


def _shift(name, by):
    return lambda a, b: setattr(a, name, getattr(a, name) + by)


def _same(name, of):
    return lambda a, b: setattr(a, name, getattr(a, of))


REFUSED = {
    "tokens": (_set(T=-1), INV), "many tokens": (_set(T=2 ** 31 - 1), UNS), "heads": (_set(H_q=0), INV), "many heads": (_set(H_q=1 << 17), UNS),
    "size": (_set(D=2048), UNS), "no size": (_set(D=0), INV), "type": (_set(dtype=9), UNS), "kind": (_set(kind=2), INV),
    "eps 0": (_set(eps=0.0), INV), "eps": (_set(eps=math.nan), INV), "offset": (_set(weight_offset=math.inf), INV),
    "odd": (_set(rot_dim=31), INV), "frequencies of nothing": (_set(rot_dim=0), INV), "wide": (_set(rot_dim=66), INV),
    "layout": (_set(interleaved=2), INV), "layout alone": (_set(interleaved=2, rot_dim=0, inv_freq=None), INV),
    "no positions": (_set(positions=None), INV), "no frequencies": (_set(inv_freq=None), INV),
    "odd frequencies": (_shift("inv_freq", 4), INV), "weight type": (_set(weight_dtype=_lib.KDA_F16), UNS),
    "odd weight": (_shift("k_weight", 2), INV), "no q": (_set(q=None), INV), "no out_k": (_set(out_k=None), INV),
    "odd q": (_shift("q", 1), INV), "weight of no k": (_set(H_k=0), INV),
    "huge stride": (_set(q_stride_t=2 ** 33, q_stride_h=64), INV), "negative stride": (_set(k_stride_t=-128, k_stride_h=64), INV),
    "out rows overlap": (_set(out_q_stride_t=64, out_q_stride_h=64), ALIAS), "both results": (_same("out_k", "out_q"), ALIAS),
    "q's result over k": (_same("out_q", "k"), ALIAS), "result over a weight": (_same("q_weight", "out_k"), ALIAS),
}
REFUSED_FORWARD = {"shifted in place": (lambda a, b: setattr(a, "out_q", a.q + 128), ALIAS),
                   "other strides in place": (lambda a, b: (_same("out_q", "q")(a, b), _set(out_q_stride_t=64, out_q_stride_h=640)(a, b)), ALIAS),
                   "a gradient": (lambda a, b: setattr(a, "grad_q_weight", b.buf(256).ctypes.data), INV)}
REFUSED_BACKWARD = {
    "no gradient": (_set(grad_q=None), INV), "no gradient of k": (_set(grad_k=None), INV), "no weight gradient": (_set(grad_q_weight=None), INV),
    "weight gradient without weight": (_set(k_weight=None), INV), "odd gradient": (_shift("grad_q", 1), INV),
    "odd weight gradient": (_shift("grad_k_weight", 2), INV), "in place of q": (_same("out_q", "q"), ALIAS),
    "in place of k's gradient": (_same("out_q", "grad_k"), ALIAS), "shifted in place": (lambda a, b: setattr(a, "out_q", a.grad_q + 128), ALIAS),
    "both weight gradients": (_same("grad_k_weight", "grad_q_weight"), ALIAS), "weight gradient in place": (_same("grad_q_weight", "q_weight"), ALIAS),
    "weight gradient over rows": (_same("grad_q_weight", "k"), ALIAS),
}


@pytest.mark.parametrize("case", sorted(REFUSED) + sorted(REFUSED_FORWARD))
def test_refusals(lib, fake, case):  # noqa: F811
    b = FakeBufs()
    a = _norm(b)
    mutate, code = {**REFUSED, **REFUSED_FORWARD}[case]
    mutate(a, b)
    assert lib.kda_qk_norm_validate(ctypes.byref(a)) == code
    assert lib.kda_qk_norm(fake.ctx, ctypes.byref(a), None) == code
    assert fake.launches == []


@pytest.mark.parametrize("case", sorted(REFUSED) + sorted(REFUSED_BACKWARD))
def test_backward_refusals(lib, fake, case):  # noqa: F811
    b = FakeBufs()
    a = _norm(b, back=True)
    mutate, code = {**REFUSED, **REFUSED_BACKWARD}[case]
    mutate(a, b)
    ref = ctypes.byref(a)
    assert lib.kda_qk_norm_backward_validate(ref) == code and lib.kda_qk_norm_backward_workspace_bytes(ref) == 0
    assert lib.kda_qk_norm_backward(fake.ctx, ref, b.buf(1 << 16).ctypes.data, 1 << 16, None) == code
    assert fake.launches == []


def test_null_arguments(lib, fake):  # noqa: F811
    assert lib.kda_qk_norm_validate(None) == INV and lib.kda_qk_norm_backward_validate(None) == INV
    b = FakeBufs()
    a = _norm(b)
    assert lib.kda_qk_norm(None, ctypes.byref(a), None) == INV
    assert lib.kda_qk_norm_backward(None, ctypes.byref(a), None, 0, None) == INV
    assert fake.launches == []


def test_launches_and_workspace(lib, fake):  # noqa: F811
    b = FakeBufs()
    a = _norm(b)
    assert lib.kda_qk_norm(fake.ctx, ctypes.byref(a), 0x10) == _lib.KDA_OK
    assert fake.launches == [(12, 0x10)] and fake.syncs() == []
    a.T = 0
    fake.launches.clear()
    assert lib.kda_qk_norm(fake.ctx, ctypes.byref(a), 0x10) == _lib.KDA_OK and fake.launches == []
    g = _norm(b, back=True)
    ref = ctypes.byref(g)
    need = lib.kda_qk_norm_backward_workspace_bytes(ref)
    assert need == 10 * 2 * 64 * 4  # a workgroup's sums for each token, of 64 channels
    ws = b.buf(need)
    for ptr, size in ((None, need), (ws.ctypes.data, need - 1), (ws.ctypes.data + 128, need)):
        assert lib.kda_qk_norm_backward(fake.ctx, ref, ptr, size, 0x10) == _lib.KDA_ERR_WORKSPACE
    assert fake.launches == []
    assert lib.kda_qk_norm_backward(fake.ctx, ref, ws.ctypes.data, need, 0x10) == _lib.KDA_OK and fake.launches == [(13, 0x10)]
    fake.launches.clear()
    n = _norm(b, back=True, weight=False)
    assert lib.kda_qk_norm_backward_workspace_bytes(ctypes.byref(n)) == 0
    assert lib.kda_qk_norm_backward(fake.ctx, ctypes.byref(n), None, 0, 0x10) == _lib.KDA_OK and fake.launches == [(13, 0x10)]


def test_one_projections_rows_in_place(lib, fake):  # noqa: F811
    b = FakeBufs()
    a = _norm(b)
    buf = b.buf(10 * 8 * 64 * 2).ctypes.data
    a.q = a.out_q = buf
    a.k = a.out_k = buf + 4 * 64 * 2
    for n in ROWS:
        setattr(a, f"{n}_stride_t", 8 * 64)
        setattr(a, f"{n}_stride_h", 64)
    assert lib.kda_qk_norm(fake.ctx, ctypes.byref(a), 0x20) == _lib.KDA_OK and fake.launches == [(12, 0x20)]
    a.k = a.out_k = buf + 3 * 64 * 2  # k's first head is q's last
    assert lib.kda_qk_norm_validate(ctypes.byref(a)) == ALIAS


# ------------------------------------------------------------------------------ binding
def _call(**kw):
    base = dict(q=torch.zeros(5, 4, 8), k=torch.zeros(5, 2, 8), q_weight=torch.ones(8), k_weight=torch.ones(8), positions=torch.arange(5),
                inv_freq=torch.ones(4, dtype=torch.float64), out_q=torch.zeros(5, 4, 8), out_k=torch.zeros(5, 2, 8))
    return {**base, **kw}


@pytest.mark.parametrize("kw,exc", [
    (dict(q=torch.zeros(5, 4, 8, dtype=torch.int32)), TypeError), (dict(k=torch.zeros(4, 2, 8)), ValueError),
    (dict(k=torch.zeros(5, 2, 16)), ValueError), (dict(k=torch.zeros(5, 2, 8).half()), TypeError), (dict(out_q=torch.zeros(5, 3, 8)), ValueError),
    (dict(out_k=torch.zeros(5, 2, 8).half()), ValueError), (dict(k=None), ValueError), (dict(k=None, out_k=None), ValueError),
    (dict(q_weight=torch.ones(7)), ValueError), (dict(q_weight=torch.ones(8).half()), TypeError), (dict(k_weight=torch.ones(16)[::2]), ValueError),
    (dict(q=torch.zeros(5, 4, 8).half(), k=torch.zeros(5, 2, 8).half(), out_q=torch.zeros(5, 4, 8).half(), out_k=torch.zeros(5, 2, 8).half(),
          q_weight=torch.ones(8).half()), TypeError),
    (dict(positions=torch.arange(4)), ValueError), (dict(positions=None), ValueError), (dict(inv_freq=torch.ones(4)), TypeError),
    (dict(inv_freq=torch.ones(5, dtype=torch.float64)), ValueError), (dict(kind="mean"), ValueError),
    (dict(q=torch.zeros(5, 4, 16)[..., ::2]), ValueError), (dict(q=torch.zeros(5, 0, 8), out_q=torch.zeros(5, 0, 8)), ValueError),
    (dict(grad_q=torch.zeros(5, 4, 9), grad_k=torch.zeros(5, 2, 8)), ValueError),
    (dict(grad_q=torch.zeros(5, 4, 8), grad_k=torch.zeros(5, 2, 8).half()), ValueError),
])
def test_binding_refusals(kw, exc):
    a = kda.make_qk_norm_args(**_call())
    assert (a.T, a.H_q, a.H_k, a.D, a.rot_dim, a.weight_dtype) == (5, 4, 2, 8, 8, _lib.KDA_F32)
    with pytest.raises(exc):
        kda.make_qk_norm_args(**_call(**kw))


def test_binding_fills_strides_and_kinds():
    row = torch.zeros(5, 6 * 8)
    q, k = row.split([32, 16], 1)
    a = kda.make_qk_norm_args(**_call(q=q.unflatten(1, (4, 8)), k=k.unflatten(1, (2, 8)), kind="l2", weight_offset=1.0, interleaved=True))
    assert (a.q_stride_t, a.q_stride_h, a.k_stride_t, a.k_stride_h) == (48, 8, 48, 8)
    assert a.kind == _lib.KDA_NORM_L2 and a.weight_offset == 1.0 and a.interleaved == 1
    a = kda.make_qk_norm_args(**_call(positions=None, inv_freq=None, q_weight=None, k_weight=None))
    assert a.rot_dim == 0 and not a.q_weight


@pytest.mark.parametrize("name", ["q", "k", "q_weight", "k_weight", "out_q", "out_k"])
def test_no_gradient_is_recorded(name):
    kw = _call()
    kw[name].requires_grad_()
    with pytest.raises(ValueError, match="qk_norm_backward"):
        kda.make_qk_norm_args(**kw)
    with torch.no_grad():
        assert kda.make_qk_norm_args(**kw).T == 5


def test_cpu_tensors_are_refused():
    kw = _call()
    with pytest.raises(ValueError, match="GPU"):
        kda.qk_norm(kw["q"], kw["k"])
    with pytest.raises(ValueError, match="GPU"):
        kda.qk_norm_backward(kw["q"], kw["k"], kw["q"], kw["k"])


# ------------------------------------------------------------------------------ oracle
def test_oracle_rows():
    r = np.random.default_rng(1)
    x, w = r.normal(size=(4, 2, 6)), r.normal(size=6)
    y = qk_norm(x, l2=True, eps=1e-30)
    assert np.allclose(np.linalg.norm(y, axis=-1), 1) and np.allclose(y * np.linalg.norm(x, axis=-1, keepdims=True), x)
    assert np.allclose((qk_norm(x, eps=1e-30) ** 2).mean(-1), 1)
    assert np.allclose(qk_norm(x, w, offset=1.0), qk_norm(x) * (1 + w))
    assert np.allclose(qk_norm(np.zeros((1, 1, 6)), w), 0)


@pytest.mark.parametrize("l2", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_gradient_against_differences(l2, interleaved):
    r = np.random.default_rng(2)
    x, dy, w = r.normal(size=(3, 2, 8)), r.normal(size=(3, 2, 8)), r.normal(size=8)
    kw = dict(positions=np.array([0, 5, 77]), inv_freq=np.array([1.0, 0.1, 0.01]), l2=l2, offset=1.0, interleaved=interleaved)
    dx, dw = qk_norm_gradient(dy, x, w, **kw)
    h = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        slope = (dy * (qk_norm(x + e, w, **kw) - qk_norm(x - e, w, **kw))).sum() / (2 * h)
        assert abs(slope - dx[i]) < 1e-8
    for j in range(8):
        e = np.zeros(8)
        e[j] = h
        slope = (dy * (qk_norm(x, w + e, **kw) - qk_norm(x, w - e, **kw))).sum() / (2 * h)
        assert abs(slope - dw[j]) < 1e-8
