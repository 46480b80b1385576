"""CPU tests of the linear-attention and rotary entry points (no GPU): argument checks of the C
ABI and of the binding, workspace and segment policy, the launch sequence through a recording fake
runtime, the frequency helper, and the oracle's own pins."""
import ctypes
import math

import numpy as np
import pytest
import torch

import gated_delta_rule_pack_amd as kda
from gated_delta_rule_pack_amd import _lib
from oracle import linear_forward, rotate
from tests.test_abi_cpu import FakeBufs, FakeRuntime

INV, UNS, STATE, STRIDE, ALIAS = (_lib.KDA_ERR_INVALID_ARG, _lib.KDA_ERR_UNSUPPORTED, _lib.KDA_ERR_STATE_MODE,
                                  _lib.KDA_ERR_STRIDE, _lib.KDA_ERR_ALIAS)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


@pytest.fixture
def fake(lib):
    f = FakeRuntime()
    ctx = ctypes.c_void_p()
    assert lib.kda_ctx_create_with_runtime(ctypes.byref(f.rt), 256, ctypes.byref(ctx)) == _lib.KDA_OK
    f.ctx = ctx
    f.log = []
    yield f
    lib.kda_ctx_destroy(ctx)


def _args(b, T=100, N=3, H=4, H_qk=2, K=128, V=64, step=False):
    a = _lib.LinearArgs()
    a.T, a.N, a.H, a.H_qk, a.K, a.V, a.scale = T, N, H, H_qk, K, V, 0.1
    a.q, a.k = (b.buf(max(T * H_qk * K * 2, 16)).ctypes.data for _ in range(2))
    a.v, a.out = (b.buf(max(T * H * V * 2, 16)).ctypes.data for _ in range(2))
    a.g, a.g_dtype, a.g_per_token = b.buf(max(T * H * 4, 16)).ctypes.data, _lib.KDA_F32, 1
    if not step:
        cu = np.linspace(0, T, N + 1).astype(np.int32)
        host = b.buf(4 * (N + 1), 16).view(np.int32)
        host[:] = cu
        a.cu_seqlens = a.cu_seqlens_host = host.ctypes.data
        a.host = host
    a.state_cache, a.num_slots, a.state_cache_stride0 = b.buf(4 * 8 * H * K * V).ctypes.data, 8, H * K * V
    a.state_indices, a.has_initial_state = b.buf(4 * N, 16).ctypes.data, b.buf(N, 16).ctypes.data
    a.state_dtype = _lib.KDA_F32
    return a


def _rot(a, b):
    a.rot_dim, a.inv_freq, a.rot_factor = 64, b.buf(8 * 32).ctypes.data, 1.0
    a.positions = b.buf(8 * max(a.T, 1)).ctypes.data


def _dense(a, b, both=True):
    a.state_cache = a.state_indices = a.has_initial_state = None
    n = 4 * a.N * a.H * a.K * a.V
    a.initial_state = b.buf(n).ctypes.data
    if both:
        a.final_state = b.buf(n).ctypes.data


def _set(**kw):
    def f(a, b):
        for k, v in kw.items():
            setattr(a, k, v)
    return f


def _host(*cu):
    def f(a, b):
        a.host[:] = cu
    return f


REFUSED = {
    "no rows": (_set(N=0), INV), "negative tokens": (_set(T=-1), INV), "no heads": (_set(H=0), INV),
    "too many tokens": (_set(T=2 ** 31 - 1), UNS), "too many rows": (_set(N=2 ** 20 + 1), INV),
    "K": (_set(K=96), UNS), "V": (_set(V=256), UNS),
    "scale": (_set(scale=math.inf), INV), "heads do not divide": (_set(H_qk=3), INV), "more q/k heads": (_set(H_qk=8), INV),
    "k first": (_set(state_k_first=2), INV), "per token": (_set(g_per_token=2), INV),
    "fp16 g": (_set(g_dtype=_lib.KDA_F16), UNS), "misaligned g": (lambda a, b: setattr(a, "g", a.g + 2), INV),
    "state dtype": (_set(state_dtype=5), UNS),
    "odd stride": (_set(q_stride_t=260, q_stride_h=128), INV), "negative stride": (_set(v_stride_t=-256, v_stride_h=64), INV),
    "huge stride": (_set(k_stride_t=2 ** 33, k_stride_h=128), INV),
    "out rows overlap": (_set(out_stride_t=64, out_stride_h=64), ALIAS), "out heads overlap": (_set(out_stride_t=256, out_stride_h=32), ALIAS),
    "no q": (_set(q=None), INV), "no out": (_set(out=None), INV), "misaligned v": (lambda a, b: setattr(a, "v", a.v + 8), INV),
    "out is v": (lambda a, b: setattr(a, "out", a.v), ALIAS), "out over k": (lambda a, b: setattr(a, "out", a.k + 16 * 64), ALIAS),
    "out over q": (lambda a, b: setattr(a, "out", a.q), ALIAS),
    "dense and pool": (lambda a, b: setattr(a, "initial_state", a.v), STATE),
    "no slots": (_set(num_slots=0), INV), "short stride0": (_set(state_cache_stride0=4 * 128 * 64 - 1), STRIDE),
    "unaligned stride0": (_set(state_cache_stride0=4 * 128 * 64 + 2), INV),
    "misaligned pool": (lambda a, b: setattr(a, "state_cache", a.state_cache + 8), INV),
    "odd rotation": (lambda a, b: (_rot(a, b), setattr(a, "rot_dim", 33)), INV),
    "wide rotation": (lambda a, b: (_rot(a, b), setattr(a, "rot_dim", 130)), INV),
    "no positions": (lambda a, b: (_rot(a, b), setattr(a, "positions", None)), INV),
    "rotation factor": (lambda a, b: (_rot(a, b), setattr(a, "rot_factor", math.nan)), INV),
    "position type": (lambda a, b: (_rot(a, b), setattr(a, "positions_i64", 3)), INV),
}
REFUSED_FWD = {
    "no bounds": (_set(cu_seqlens=None), INV), "no indices": (_set(state_indices=None), INV),
    "no flags": (_set(has_initial_state=None), INV),
    "odd segment": (_set(seg_len=100), INV), "negative segment": (_set(seg_len=-64), INV),
    "bounds fall": (_host(0, 50, 40, 100), INV), "bounds start late": (_host(1, 50, 60, 100), INV),
    "bounds past T": (_host(0, 50, 60, 101), INV),
    "states overlap": (lambda a, b: (_dense(a, b), setattr(a, "final_state", a.initial_state + 64)), ALIAS),
}
REFUSED_STEP = {
    "rows differ": (_set(N=2), INV), "no pool": (_set(state_cache=None), INV),
    "few slots without indices": (_set(state_indices=None, num_slots=2), INV),
    "dense states": (lambda a, b: _dense(a, b), INV),
}


@pytest.mark.parametrize("case", sorted(REFUSED) + sorted(REFUSED_FWD))
def test_forward_refusals(lib, fake, case):
    b = FakeBufs()
    a = _args(b)
    mutate, code = {**REFUSED, **REFUSED_FWD}[case]
    mutate(a, b)
    assert lib.kda_linear_fwd_validate(ctypes.byref(a)) == code
    assert lib.kda_linear_fwd_workspace_bytes(ctypes.byref(a)) == 0 and lib.kda_linear_seg_len(ctypes.byref(a)) == 0
    assert lib.kda_linear_fwd(fake.ctx, ctypes.byref(a), None, 0, None) == code
    assert fake.launches == []


@pytest.mark.parametrize("case", sorted(REFUSED) + sorted(REFUSED_STEP))
def test_step_refusals(lib, fake, case):
    b = FakeBufs()
    a = _args(b, T=3, N=3, step=True)
    mutate, code = {**REFUSED, **REFUSED_STEP}[case]
    mutate(a, b)
    if case in ("out over k", "out rows overlap"):  # their offsets are made for more rows
        a.T = a.N = 100
        a.state_indices = b.buf(4 * 100, 16).ctypes.data
    got = lib.kda_linear_step_validate(ctypes.byref(a))
    assert got == code if case not in ("too many tokens", "negative tokens", "no rows", "too many rows") else got != _lib.KDA_OK
    assert lib.kda_linear_step(fake.ctx, ctypes.byref(a), None) == got
    assert fake.launches == []


def test_null_arguments(lib, fake):
    assert lib.kda_linear_fwd_validate(None) == INV and lib.kda_linear_step_validate(None) == INV
    assert lib.kda_rotary_validate(None) == INV
    b = FakeBufs()
    a = _args(b)
    assert lib.kda_linear_fwd(None, ctypes.byref(a), None, 0, None) == INV
    assert lib.kda_linear_step(None, ctypes.byref(a), None) == INV
    assert lib.kda_rotary(None, None, None) == INV


def test_forward_launches_and_workspace(lib, fake):
    b = FakeBufs()
    a = _args(b)
    # 100 tokens and two more sequences of 128 * 64 fp32 state each (K V 4 2 / ((K + V) 4) tokens' worth):
    # the policy's one segment for so little work.
    a.seg_len = 64 * 64
    assert lib.kda_linear_fwd_workspace_bytes(ctypes.byref(a)) == 0
    assert lib.kda_linear_fwd(fake.ctx, ctypes.byref(a), None, 0, 0x10) == _lib.KDA_OK
    assert fake.launches == [(7, 0x10)] and fake.syncs() == [] and fake.log == []
    fake.launches.clear()
    a.seg_len = 64
    axis = 100 + 2 * (128 * 64 * 4 * 2 // ((128 + 64) * 4))
    borders = -(-axis // 64) - 1
    def up(x):
        return -(-x // 256) * 256
    plane = 4 * 128 * 64 * 4
    want = 2 * up(borders * plane) + up(borders * 4 * 4) + up(borders * 4)
    need = lib.kda_linear_fwd_workspace_bytes(ctypes.byref(a))
    assert need == want
    ws = b.buf(need)
    for ptr, size in ((None, need), (ws.ctypes.data, need - 1), (ws.ctypes.data + 128, need)):
        assert lib.kda_linear_fwd(fake.ctx, ctypes.byref(a), ptr, size, 0x10) == _lib.KDA_ERR_WORKSPACE
    assert fake.launches == []
    assert lib.kda_linear_fwd(fake.ctx, ctypes.byref(a), ws.ctypes.data, need, 0x10) == _lib.KDA_OK
    assert [k for k, _ in fake.launches] == [5, 6, 7]
    fake.launches.clear()
    _rot(a, b)
    more = lib.kda_linear_fwd_workspace_bytes(ctypes.byref(a)) - need
    assert more == 2 * up(100 * 2 * 128 * 2)
    ws = b.buf(need + more)
    assert lib.kda_linear_fwd(fake.ctx, ctypes.byref(a), ws.ctypes.data, need + more, 0x10) == _lib.KDA_OK
    assert [k for k, _ in fake.launches] == [9, 5, 6, 7]
    # No rows: nothing to rotate, the states still move.
    z = _args(FakeBufs(), T=0)
    z.host[:] = 0
    z.q = z.k = z.v = z.out = z.g = None
    assert lib.kda_linear_fwd_validate(ctypes.byref(z)) == _lib.KDA_OK


def test_launch_failures_are_reported(lib, fake):
    b = FakeBufs()
    a = _args(b)
    a.seg_len = 4096
    fake.rt.launch = _lib.LAUNCH(lambda *x: 1)
    ctx = ctypes.c_void_p()
    assert lib.kda_ctx_create_with_runtime(ctypes.byref(fake.rt), 256, ctypes.byref(ctx)) == _lib.KDA_OK
    assert lib.kda_linear_fwd(ctx, ctypes.byref(a), None, 0, None) == _lib.KDA_ERR_HIP
    s = _args(b, T=3, N=3, step=True)
    assert lib.kda_linear_step(ctx, ctypes.byref(s), None) == _lib.KDA_ERR_HIP
    lib.kda_ctx_destroy(ctx)


def test_policy_gives_whole_chunks_and_covers_the_axis(lib):
    b = FakeBufs()
    for T, N, H in ((1, 1, 1), (37, 1, 12), (100, 3, 4), (4096, 1, 12), (16384, 1, 12), (32768, 1, 32), (131072, 128, 12)):
        a = _args(b, T=8, N=1, H=4)
        a.T, a.N, a.H, a.H_qk = T, N, H, H  # sizes only; nothing is read, the addresses are far apart
        a.q, a.k, a.v, a.out = (i << 42 for i in range(1, 5))
        a.cu_seqlens_host = None
        a.num_slots, a.state_cache_stride0 = N, H * 128 * 64
        L = lib.kda_linear_seg_len(ctypes.byref(a))
        assert L > 0 and L % 64 == 0


def _sizes_only(a, T, N, H):
    """Sizes alone change: nothing is read, and the addresses are far apart."""
    a.T, a.N, a.H, a.H_qk = T, N, H, H
    a.q, a.k, a.v, a.out = (i << 46 for i in range(1, 5))
    a.cu_seqlens_host = None
    a.num_slots, a.state_cache_stride0 = N, H * 128 * 64


def test_launches_stay_within_32_bits_of_work_items(lib, fake):
    b = FakeBufs()
    for N, H, code in ((1 << 20, 15, _lib.KDA_OK), (1 << 20, 16, UNS), (1 << 18, 63, _lib.KDA_OK), (1 << 12, 1 << 13, UNS)):
        a = _args(b, T=3, N=3, step=True)
        _sizes_only(a, N, N, H)
        assert lib.kda_linear_step_validate(ctypes.byref(a)) == code, (N, H)
    for T, H, code in ((1 << 22, 127, _lib.KDA_OK), (1 << 22, 128, UNS), (1 << 29, 1, UNS), (1 << 30, 1, UNS)):
        a = _args(b)
        _sizes_only(a, T, 1, H)
        a.seg_len = 64
        assert lib.kda_linear_fwd_validate(ctypes.byref(a)) == code, (T, H)
        a.seg_len = 0  # the policy stays far below
        assert lib.kda_linear_fwd_validate(ctypes.byref(a)) == _lib.KDA_OK
    assert fake.launches == []


# ------------------------------------------------------------------------------ rotary
def _rotary_args(b, T=10, Hq=4, Hk=2, D=64):
    a = _lib.RotaryArgs()
    a.T, a.H_q, a.H_k, a.D, a.rot_dim, a.dtype, a.factor = T, Hq, Hk, D, 32, _lib.KDA_BF16, 1.0
    a.q, a.out_q = (b.buf(T * Hq * D * 2).ctypes.data for _ in range(2))
    a.k, a.out_k = (b.buf(T * max(Hk, 1) * D * 2).ctypes.data for _ in range(2))
    a.positions, a.inv_freq = b.buf(4 * T).ctypes.data, b.buf(8 * 16).ctypes.data
    return a


ROTARY_REFUSED = {
    "tokens": (_set(T=-1), INV), "heads": (_set(H_q=0), INV), "size": (_set(D=2048), UNS), "type": (_set(dtype=9), UNS),
    "odd": (_set(rot_dim=31), INV), "zero": (_set(rot_dim=0), INV), "wide": (_set(rot_dim=66), INV),
    "factor": (_set(factor=math.nan), INV), "layout": (_set(interleaved=2), INV), "inverse": (_set(inverse=-1), INV),
    "no positions": (_set(positions=None), INV), "no frequencies": (_set(inv_freq=None), INV),
    "odd frequencies": (lambda a, b: setattr(a, "inv_freq", a.inv_freq + 4), INV),
    "odd positions": (lambda a, b: (setattr(a, "positions_i64", 1), setattr(a, "positions", a.positions + 4)), INV),
    "no q": (_set(q=None), INV), "no out_k": (_set(out_k=None), INV), "odd q": (lambda a, b: setattr(a, "q", a.q + 1), INV),
    "out rows overlap": (_set(out_q_stride_t=64, out_q_stride_h=64), ALIAS),
    "shifted in place": (lambda a, b: setattr(a, "out_q", a.q + 128), ALIAS),
    "in place, other strides": (lambda a, b: (setattr(a, "out_q", a.q), setattr(a, "out_q_stride_t", 64), setattr(a, "out_q_stride_h", 640)), ALIAS),
    "q's result over k": (lambda a, b: setattr(a, "out_q", a.k), ALIAS),
    "both results": (lambda a, b: setattr(a, "out_k", a.out_q), ALIAS),
}


@pytest.mark.parametrize("case", sorted(ROTARY_REFUSED))
def test_rotary_refusals(lib, fake, case):
    b = FakeBufs()
    a = _rotary_args(b)
    mutate, code = ROTARY_REFUSED[case]
    mutate(a, b)
    assert lib.kda_rotary_validate(ctypes.byref(a)) == code
    assert lib.kda_rotary(fake.ctx, ctypes.byref(a), None) == code
    assert fake.launches == []


def test_rotary_accepts_one_projections_rows_in_place(lib, fake):
    b = FakeBufs()
    a = _rotary_args(b)
    buf = b.buf(10 * 8 * 64 * 2).ctypes.data
    a.q = a.out_q = buf
    a.k = a.out_k = buf + 4 * 64 * 2
    for n in ("q", "k", "out_q", "out_k"):
        setattr(a, f"{n}_stride_t", 8 * 64)
        setattr(a, f"{n}_stride_h", 64)
    assert lib.kda_rotary(fake.ctx, ctypes.byref(a), 0x20) == _lib.KDA_OK
    assert fake.launches == [(9, 0x20)]
    a.k = a.out_k = buf + 3 * 64 * 2  # k's first head is q's last
    assert lib.kda_rotary_validate(ctypes.byref(a)) == ALIAS
    a.T = 0
    fake.launches.clear()
    assert lib.kda_rotary(fake.ctx, ctypes.byref(a), 0x20) == _lib.KDA_OK and fake.launches == []


# ------------------------------------------------------------------------------ binding
BF = torch.bfloat16


def _tensors(T=20, H=4, H_qk=2, K=128, V=64, N=2):
    return (dict(q=torch.zeros(T, H_qk, K, dtype=BF), k=torch.zeros(T, H_qk, K, dtype=BF), v=torch.zeros(T, H, V, dtype=BF),
                 g=torch.zeros(T, H)),
            dict(cu_seqlens=torch.tensor([0, 7, T], dtype=torch.int32), state_cache=torch.zeros(3, H, V, K),
                 state_indices=torch.zeros(N, dtype=torch.int32), has_initial_state=torch.zeros(N, dtype=torch.bool),
                 out=torch.zeros(T, H, V, dtype=BF)))


def test_binding_fills_strides_and_types():
    row = torch.zeros(20, 2 * 2 * 128 + 4 * 64, dtype=BF)
    q, k, v = row.split([256, 256, 256], 1)
    t, kw = _tensors()
    a = kda.make_linear_args(q.unflatten(1, (2, 128)), k.unflatten(1, (2, 128)), v.unflatten(1, (4, 64)), t["g"], **kw)
    assert (a.q_stride_t, a.q_stride_h, a.v_stride_t, a.v_stride_h) == (768, 128, 768, 64)
    assert (a.T, a.N, a.H, a.H_qk, a.K, a.V) == (20, 2, 4, 2, 128, 64) and a.g_per_token == 1 and a.num_slots == 3
    a = kda.make_linear_args(t["q"][None], t["k"][None], t["v"][None], t["g"][0].bfloat16(), **kw)
    assert a.g_per_token == 0 and a.g_dtype == _lib.KDA_BF16
    assert a.scale == pytest.approx(128 ** -0.5)


def test_binding_of_broadcast_rows():
    # Strides 0, 0 mean dense to the library: a broadcast row must not be passed as such.
    t, kw = _tensors()
    one, many = torch.zeros(1, 1, 128, dtype=BF), torch.zeros(20, 1, 128, dtype=BF)
    a = kda.make_linear_args(t["q"], many.expand(-1, 2, -1), t["v"], t["g"], **kw)
    assert (a.k_stride_t, a.k_stride_h) == (128, 0)
    with pytest.raises(ValueError, match="broadcast"):
        kda.make_linear_args(t["q"], one.expand(20, 2, -1), t["v"], t["g"], **kw)
    step = dict(N=1, state_cache=kw["state_cache"], out=torch.zeros(1, 4, 64, dtype=BF))
    a = kda.make_linear_args(one.expand(-1, 2, -1), one.expand(-1, 2, -1), t["v"][:1], t["g"][:1], **step)
    assert a.q_stride_h == a.k_stride_h == 0 and a.q_stride_t == a.k_stride_t == 256
    pos, inv = torch.zeros(20, dtype=torch.int32), torch.ones(8, dtype=torch.float64)
    with pytest.raises(ValueError, match="broadcast"):
        kda.make_rotary_args(one.expand(20, 3, -1), None, pos, inv, torch.zeros(20, 3, 128, dtype=BF), None)
    with pytest.raises(ValueError, match="broadcast"):
        kda.make_rotary_args(torch.zeros(20, 3, 128, dtype=BF), None, pos, inv, one.expand(20, 3, -1), None)
    a = kda.make_rotary_args(one.expand(1, 3, -1), None, pos[:1], inv, torch.zeros(1, 3, 128, dtype=BF), None)
    assert (a.q_stride_t, a.q_stride_h) == (384, 0)
    a = kda.make_rotary_args(torch.zeros(1, 3, 128, dtype=BF).expand(20, -1, -1), None, pos, inv, torch.zeros(20, 3, 128, dtype=BF), None)
    assert (a.q_stride_t, a.q_stride_h) == (0, 128)


def _m(name, value):
    return lambda t, kw: (t if name in t else kw).__setitem__(name, value)


BINDING_REFUSED = {
    "fp16 q": (_m("q", torch.zeros(20, 2, 128, dtype=torch.float16)), TypeError),
    "k shape": (_m("k", torch.zeros(20, 4, 128, dtype=BF)), ValueError),
    "v tokens": (_m("v", torch.zeros(19, 4, 64, dtype=BF)), ValueError),
    "heads": (_m("v", torch.zeros(20, 3, 64, dtype=BF)), ValueError),
    "no heads": (lambda t, kw: (t.update(q=torch.zeros(20, 0, 128, dtype=BF), k=torch.zeros(20, 0, 128, dtype=BF))), ValueError),
    "strided channels": (_m("q", torch.zeros(20, 2, 256, dtype=BF)[..., ::2]), ValueError),
    "g shape": (_m("g", torch.zeros(20, 3)), ValueError), "g type": (_m("g", torch.zeros(20, 4, dtype=torch.float16)), TypeError),
    "strided g": (_m("g", torch.zeros(20, 8)[:, ::2]), ValueError),
    "bounds type": (_m("cu_seqlens", torch.tensor([0, 7, 20])), TypeError),
    "short indices": (_m("state_indices", torch.zeros(1, dtype=torch.int32)), ValueError),
    "int64 indices": (_m("state_indices", torch.zeros(2, dtype=torch.int64)), TypeError),
    "float flags": (_m("has_initial_state", torch.zeros(2)), TypeError),
    "pool planes": (_m("state_cache", torch.zeros(3, 4, 128, 64)), ValueError),
    "pool strides": (_m("state_cache", torch.zeros(3, 4, 128, 64).transpose(2, 3)), ValueError),
    "empty pool": (_m("state_cache", torch.zeros(0, 4, 64, 128)), ValueError),
    "fp32 out": (_m("out", torch.zeros(20, 4, 64)), TypeError), "out shape": (_m("out", torch.zeros(20, 4, 128, dtype=BF)), ValueError),
    "dense with indices": (lambda t, kw: kw.update(state_cache=None), ValueError),
    "positions alone": (lambda t, kw: kw.update(positions=torch.arange(20)), ValueError),
    "fp32 frequencies": (lambda t, kw: kw.update(positions=torch.arange(20), inv_freq=torch.zeros(4)), TypeError),
    "many frequencies": (lambda t, kw: kw.update(positions=torch.arange(20), inv_freq=torch.zeros(65, dtype=torch.float64)), ValueError),
    "float positions": (lambda t, kw: kw.update(positions=torch.zeros(20), inv_freq=torch.zeros(4, dtype=torch.float64)), TypeError),
    "short positions": (lambda t, kw: kw.update(positions=torch.arange(19), inv_freq=torch.zeros(4, dtype=torch.float64)), ValueError),
}


@pytest.mark.parametrize("case", sorted(BINDING_REFUSED))
def test_binding_refusals(case):
    t, kw = _tensors()
    mutate, exc = BINDING_REFUSED[case]
    mutate(t, kw)
    with pytest.raises(exc):
        kda.make_linear_args(t["q"], t["k"], t["v"], t["g"], **kw)


def test_cpu_tensors_are_refused():
    t, kw = _tensors()
    for call in (lambda: kda.linear_fwd(t["q"], t["k"], t["v"], t["g"], kw["cu_seqlens"]),
                 lambda: kda.linear_step(t["q"], t["k"], t["v"], t["g"], state_cache=kw["state_cache"]),
                 lambda: kda.rotary(t["q"], t["k"], torch.arange(20), torch.zeros(4, dtype=torch.float64))):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("kw,exc", [
    (dict(q=torch.zeros(5, 2, 8, dtype=torch.int32)), TypeError), (dict(k=torch.zeros(4, 2, 8)), ValueError),
    (dict(k=torch.zeros(5, 2, 16)), ValueError), (dict(k=torch.zeros(5, 2, 8, dtype=BF)), TypeError),
    (dict(out_q=torch.zeros(5, 3, 8)), ValueError), (dict(out_k=torch.zeros(5, 2, 8, dtype=BF)), ValueError),
    (dict(positions=torch.arange(4)), ValueError), (dict(inv_freq=torch.zeros(5, dtype=torch.float64)), ValueError),
    (dict(inv_freq=torch.zeros(0, dtype=torch.float64)), ValueError), (dict(k=None), ValueError),
])
def test_rotary_binding_refusals(kw, exc):
    base = dict(q=torch.zeros(5, 2, 8), k=torch.zeros(5, 2, 8), positions=torch.arange(5), inv_freq=torch.ones(4, dtype=torch.float64),
                out_q=torch.zeros(5, 2, 8), out_k=torch.zeros(5, 2, 8))
    assert kda.make_rotary_args(**base).rot_dim == 8
    with pytest.raises(exc):
        kda.make_rotary_args(**{**base, **kw})


# ------------------------------------------------------------------------------ frequencies
def test_frequencies():
    inv, f = kda.rotary_frequencies(8)
    assert inv.dtype == torch.float64 and f == 1.0
    assert torch.allclose(inv, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14)
    assert torch.equal(kda.rotary_frequencies(8, scaling="linear", scale=4.0)[0], inv / 4)
    ntk, f = kda.rotary_frequencies(8, scaling="ntk", scale=4.0)
    assert f == 1.0 and ntk[0] == 1.0 and ntk[-1].item() == pytest.approx(inv[-1].item() / 4, rel=1e-12)
    full = kda.rotary_frequencies(128)[0]
    yarn, f = kda.rotary_frequencies(128, scaling="yarn", scale=8.0, original_length=4096)
    assert f == pytest.approx(0.1 * math.log(8.0) + 1)
    turns = full * 4096 / (2 * math.pi)
    assert torch.equal(yarn[turns > 40], full[turns > 40])  # well above beta_fast: kept
    assert torch.allclose(yarn[turns < 0.8], full[turns < 0.8] / 8, rtol=1e-14)  # below beta_slow: shrunk
    between = (yarn <= full * (1 + 1e-15)) & (yarn >= full / 8 * (1 - 1e-15))
    assert bool(between.all()) and bool((yarn[1:] < yarn[:-1]).all())


@pytest.mark.parametrize("kw", [dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, base=1.0), dict(rot_dim=8, scale=0.5),
                                dict(rot_dim=8, scale=2.0), dict(rot_dim=8, scaling="other", scale=2.0),
                                dict(rot_dim=2, scaling="ntk", scale=2.0), dict(rot_dim=8, scaling="yarn", scale=2.0)])
def test_frequency_refusals(kw):
    with pytest.raises(ValueError):
        kda.rotary_frequencies(**kw)


# ------------------------------------------------------------------------------ oracle pins
def test_oracle_closed_form():
    """Against the sum it stands for: o_t = scale sum_s e^{G_t - G_s} (q_t k_s) v_s + the initial state's part."""
    r = np.random.default_rng(0)
    T, H, K, V = 7, 2, 3, 4
    q, k, v, g = r.normal(size=(T, 1, K)), r.normal(size=(T, 1, K)), r.normal(size=(T, H, V)), -r.random((T, H))
    S0 = r.normal(size=(1, H, V, K))
    out, S = linear_forward(q, k, v, g, [0, T], scale=0.5, initial=S0)
    G = np.cumsum(g, 0)
    for h in range(H):
        for t in range(T):
            o = np.exp(G[t, h]) * S0[0, h] @ q[t, 0] + sum(np.exp(G[t, h] - G[s, h]) * (q[t, 0] @ k[s, 0]) * v[s, h] for s in range(t + 1))
            assert np.allclose(out[t, h], 0.5 * o, rtol=1e-12)
        want = np.exp(G[-1, h]) * S0[0, h] + sum(np.exp(G[-1, h] - G[s, h]) * np.outer(v[s, h], k[s, 0]) for s in range(T))
        assert np.allclose(S[0, h], want, rtol=1e-12)


def test_oracle_sequences_do_not_meet():
    r = np.random.default_rng(1)
    a = [r.normal(size=(9, 1, 2)) for _ in range(3)]
    out, S = linear_forward(*a, None, [0, 4, 4, 9], scale=1.0)
    o0, S0 = linear_forward(*(x[:4] for x in a), None, [0, 4], scale=1.0)
    o1, S1 = linear_forward(*(x[4:] for x in a), None, [0, 5], scale=1.0)
    assert np.array_equal(out, np.concatenate([o0, o1])) and np.array_equal(S[0], S0[0]) and np.array_equal(S[2], S1[0])
    assert not S[1].any()


@pytest.mark.parametrize("il", [False, True])
def test_oracle_rotation_keeps_distances_and_turns_back(il):
    r = np.random.default_rng(2)
    x, y = r.normal(size=(5, 2, 10)), r.normal(size=(5, 2, 10))
    inv = kda.rotary_frequencies(6)[0].numpy()
    pos = np.array([0, 3, 50, 7, 900])
    rx = rotate(x, pos, inv, interleaved=il)
    assert np.allclose(rotate(rx, pos, inv, interleaved=il, inverse=True), x) and np.array_equal(rx[..., 6:], x[..., 6:])
    assert np.array_equal(rx[0], x[0]) and not np.allclose(rx[1], x[1])
    # q at position p against k at position p' depends on p - p' alone.
    a = (rotate(x, pos, inv, interleaved=il) * rotate(y, pos + 5, inv, interleaved=il)).sum(-1)
    b = (rotate(x, pos + 11, inv, interleaved=il) * rotate(y, pos + 16, inv, interleaved=il)).sum(-1)
    assert np.allclose(a, b)
