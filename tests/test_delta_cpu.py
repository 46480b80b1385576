"""CPU tests of the gated delta rule's entry points (no GPU): argument checks of the C ABI and of the binding, workspace, path
policy, the launch sequence through a recording fake runtime, and the oracle's own pins."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_pack_amd as kda
from gated_delta_rule_pack_amd import _lib
from oracle import delta_forward
from tests.test_abi_cpu import FakeBufs
from tests.test_linear_cpu import (BF, BINDING_REFUSED, INV, REFUSED, REFUSED_FWD, REFUSED_STEP, UNS, _args, _set, _sizes_only, _tensors,
                                   fake, lib)  # noqa: F401 (fixtures)

WORKSPACE = _lib.KDA_ERR_WORKSPACE


def _delta(a, b, path=0):
    """A gated delta call around the linear fields a."""
    d = _lib.GatedDeltaArgs()
    d.lin = a
    d.beta, d.beta_dtype, d.dtype, d.path = b.buf(max(4 * a.T * a.H, 16)).ctypes.data, _lib.KDA_F32, _lib.KDA_BF16, path
    return d


OWN_REFUSED = {
    "no beta": (_set(beta=None), INV), "misaligned beta": (lambda d, b: setattr(d, "beta", d.beta + 2), INV),
    "fp16 beta": (_set(beta_dtype=_lib.KDA_F16), UNS), "fp32 tokens": (_set(dtype=_lib.KDA_F32), UNS), "type": (_set(dtype=7), UNS),
    "normalize": (_set(normalize=2), INV), "path": (_set(path=3), INV), "negative path": (_set(path=-1), INV),
}


@pytest.mark.parametrize("path", [0, 1, 2])
@pytest.mark.parametrize("case", sorted(REFUSED) + sorted(REFUSED_FWD) + sorted(OWN_REFUSED))
def test_forward_refusals(lib, fake, case, path):  # noqa: F811
    b = FakeBufs()
    a = _args(b)
    own = case in OWN_REFUSED
    mutate, code = {**REFUSED, **REFUSED_FWD, **OWN_REFUSED}[case]
    if own:
        d = _delta(a, b, path)
        mutate(d, b)
    else:
        mutate(a, b)
        beta = FakeBufs()
        d = _delta(_args(beta), beta, path)
        d.lin = a
    ref = ctypes.byref(d)
    assert lib.kda_gated_delta_fwd_validate(ref) == code
    assert lib.kda_gated_delta_fwd_workspace_bytes(ref) == 0
    assert lib.kda_gated_delta_fwd(fake.ctx, ref, None, 0, None) == code
    assert fake.launches == []


@pytest.mark.parametrize("case", sorted(REFUSED) + sorted(REFUSED_STEP) + sorted(set(OWN_REFUSED)))
def test_step_refusals(lib, fake, case):  # noqa: F811
    b = FakeBufs()
    a = _args(b, T=3, N=3, step=True)
    mutate, code = {**REFUSED, **REFUSED_STEP, **OWN_REFUSED}[case]
    d = _delta(a, b)
    if case in OWN_REFUSED:
        mutate(d, b)
    else:
        mutate(a, b)
        if case in ("out over k", "out rows overlap"):  # their offsets are made for more rows
            a.T = a.N = 100
            a.state_indices = b.buf(4 * 100, 16).ctypes.data
        d.lin = a
    got = lib.kda_gated_delta_step_validate(ctypes.byref(d))
    assert got == code if case not in ("too many tokens", "negative tokens", "no rows", "too many rows") else got != _lib.KDA_OK
    assert lib.kda_gated_delta_step(fake.ctx, ctypes.byref(d), None) == got
    assert fake.launches == []


def test_null_arguments(lib, fake):  # noqa: F811
    assert lib.kda_gated_delta_fwd_validate(None) == INV and lib.kda_gated_delta_step_validate(None) == INV
    assert lib.kda_gated_delta_fwd_workspace_bytes(None) == 0
    b = FakeBufs()
    d = _delta(_args(b), b)
    assert lib.kda_gated_delta_fwd(None, ctypes.byref(d), None, 0, None) == INV
    assert lib.kda_gated_delta_step(None, ctypes.byref(d), None) == INV
    assert fake.launches == []


def test_launches_and_workspace(lib, fake):  # noqa: F811
    b = FakeBufs()
    a = _args(b)  # 100 tokens, 3 sequences, H = 4 over H_qk = 2, K = 128
    d = _delta(a, b, _lib.KDA_DELTA_WALK)
    ref = ctypes.byref(d)
    assert lib.kda_gated_delta_fwd_workspace_bytes(ref) == 0
    assert lib.kda_gated_delta_fwd(fake.ctx, ref, None, 0, 0x10) == _lib.KDA_OK
    assert fake.launches == [(10, 0x10)] and fake.syncs() == []
    fake.launches.clear()
    d.path = _lib.KDA_DELTA_SCAN

    def up(x):
        return -(-x // 256) * 256

    places = 100 // 64 + 3
    want = up(places * 4 * 19712) + 2 * up(places * 2 * 64 * 128 * 2)
    need = lib.kda_gated_delta_fwd_workspace_bytes(ref)
    assert need == want
    ws = b.buf(need)
    for ptr, size in ((None, need), (ws.ctypes.data, need - 1), (ws.ctypes.data + 128, need)):
        assert lib.kda_gated_delta_fwd(fake.ctx, ref, ptr, size, 0x10) == WORKSPACE
    assert fake.launches == []
    assert lib.kda_gated_delta_fwd(fake.ctx, ref, ws.ctypes.data, need, 0x10) == _lib.KDA_OK
    assert fake.launches == [(14, 0x10), (15, 0x10)] and fake.syncs() == []
    fake.launches.clear()
    s = _delta(_args(b, T=3, N=3, step=True), b)
    assert lib.kda_gated_delta_step(fake.ctx, ctypes.byref(s), 0x20) == _lib.KDA_OK
    assert fake.launches == [(11, 0x20)]
    # No tokens: nothing to read, the states still move.
    z = _args(FakeBufs(), T=0)
    z.host[:] = 0
    z.q = z.k = z.v = z.out = z.g = None
    for path in (0, 1, 2):
        zd = _delta(z, b, path)
        zd.beta = None
        assert lib.kda_gated_delta_fwd_validate(ctypes.byref(zd)) == _lib.KDA_OK


def test_launch_failures_are_reported(lib, fake):  # noqa: F811
    b = FakeBufs()
    fake.rt.launch = _lib.LAUNCH(lambda *x: 1)
    ctx = ctypes.c_void_p()
    assert lib.kda_ctx_create_with_runtime(ctypes.byref(fake.rt), 256, ctypes.byref(ctx)) == _lib.KDA_OK
    d = _delta(_args(b), b, _lib.KDA_DELTA_WALK)
    assert lib.kda_gated_delta_fwd(ctx, ctypes.byref(d), None, 0, None) == _lib.KDA_ERR_HIP
    d.path = _lib.KDA_DELTA_SCAN
    ws = b.buf(lib.kda_gated_delta_fwd_workspace_bytes(ctypes.byref(d)))
    assert lib.kda_gated_delta_fwd(ctx, ctypes.byref(d), ws.ctypes.data, ws.size, None) == _lib.KDA_ERR_HIP
    s = _delta(_args(b, T=3, N=3, step=True), b)
    assert lib.kda_gated_delta_step(ctx, ctypes.byref(s), None) == _lib.KDA_ERR_HIP
    lib.kda_ctx_destroy(ctx)


def _path(lib, lengths, H, V=128, host=True):  # noqa: F811
    b = FakeBufs()
    N, T = len(lengths), sum(lengths)
    a = _args(b, T=8, N=1, H=4, V=V)
    _sizes_only(a, T, N, H)
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    at = b.buf(4 * (N + 1)).view(np.int32)
    at[:] = cu
    a.cu_seqlens_host = at.ctypes.data if host else None
    a.state_cache_stride0 = H * 128 * 128
    d = _delta(a, b)
    assert lib.kda_gated_delta_fwd_validate(ctypes.byref(d)) == _lib.KDA_OK
    return "scan" if lib.kda_gated_delta_fwd_workspace_bytes(ctypes.byref(d)) else "walk"


@pytest.mark.parametrize("lengths,H,V,want", [
    ([1], 12, 128, "walk"), ([64], 12, 128, "walk"), ([128], 12, 128, "walk"), ([192], 12, 128, "scan"), ([4096], 12, 128, "scan"),
    ([32768], 32, 128, "scan"), ([1024] * 4, 12, 128, "scan"), ([1024] * 16, 12, 128, "walk"), ([1024] * 16, 6, 64, "scan"),
    ([64] * 8, 12, 128, "walk"), ([4096] * 8, 32, 128, "walk"), ([1] * 64, 12, 128, "walk"), ([0, 0, 0], 4, 128, "walk"),
    ([8192, 4096, 2048, 1024, 512, 256, 128, 64], 12, 128, "scan")])
def test_policy(lib, lengths, H, V, want):  # noqa: F811
    assert _path(lib, lengths, H, V) == want


def test_policy_tells_a_long_prompt_among_single_tokens_by_the_host_bounds(lib):  # noqa: F811
    lengths = [1] * 20 + [4096] + [1] * 11
    assert _path(lib, lengths, 12) == "scan" and _path(lib, lengths, 12, host=False) == "walk"
    assert _path(lib, [1] * 127 + [512], 24) == "walk"
    for equal in ([4096], [1024] * 16, [64] * 8):  # nothing to tell
        assert _path(lib, equal, 12) == _path(lib, equal, 12, host=False)


def test_launches_stay_within_32_bits_of_work_items(lib):  # noqa: F811
    def status(T, N, H, path, step=False):
        b = FakeBufs()
        a = _args(b, T=3, N=3, step=step)
        _sizes_only(a, T, N, H)
        d = _delta(a, FakeBufs(), path) if T * H < 1 << 20 else _delta(_args(b), b, path)
        d.lin = a
        return (lib.kda_gated_delta_step_validate if step else lib.kda_gated_delta_fwd_validate)(ctypes.byref(d))

    assert status(1 << 20, 1 << 20, 15, 0, True) == _lib.KDA_OK and status(1 << 20, 1 << 20, 16, 0, True) == UNS
    assert status(1 << 20, 1 << 20, 3, _lib.KDA_DELTA_WALK) == _lib.KDA_OK and status(1 << 20, 1 << 20, 4, _lib.KDA_DELTA_WALK) == UNS
    # The scan: a workgroup for each chunk's place and head, and V / 16 of 512 threads for each sequence and head.
    assert status(1 << 22, 1, 128, _lib.KDA_DELTA_SCAN) == _lib.KDA_OK and status(1 << 22, 1, 256, _lib.KDA_DELTA_SCAN) == UNS
    assert status(1 << 20, 1 << 20, 1, _lib.KDA_DELTA_SCAN) == _lib.KDA_OK and status(1 << 20, 1 << 20, 2, _lib.KDA_DELTA_SCAN) == UNS
    assert status(1 << 22, 1, 256, 0) == _lib.KDA_OK  # the policy stays inside


# ------------------------------------------------------------------------------ binding
def _call(**kw):
    t, more = _tensors()
    return {**t, "beta": torch.zeros(20, 4), **more, **kw}


# The rule takes fp16 tokens, and no positions.
@pytest.mark.parametrize("case", sorted(c for c in BINDING_REFUSED if c != "fp16 q" and "position" not in c and "frequenc" not in c))
def test_binding_refusals(case):
    mutate, exc = BINDING_REFUSED[case]
    t, kw = _tensors()
    mutate(t, kw)
    with pytest.raises(exc):
        kda.make_gated_delta_args(**t, beta=torch.zeros(20, 4), **kw)


@pytest.mark.parametrize("kw,exc", [
    (dict(beta=None), ValueError), (dict(beta=torch.zeros(20, 3)), ValueError), (dict(beta=torch.zeros(19, 4)), ValueError),
    (dict(beta=torch.zeros(4)), ValueError), (dict(beta=torch.zeros(20, 4, dtype=torch.float16)), TypeError),
    (dict(beta=torch.zeros(20, 8)[:, ::2]), ValueError), (dict(q=torch.zeros(20, 2, 128)), TypeError),
    (dict(q=torch.zeros(20, 2, 128, dtype=torch.float16)), TypeError), (dict(path="both"), ValueError),
])
def test_own_binding_refusals(kw, exc):
    assert kda.make_gated_delta_args(**_call()).lin.T == 20
    with pytest.raises(exc):
        kda.make_gated_delta_args(**_call(**kw))


def test_binding_fills_types():
    a = kda.make_gated_delta_args(**_call(beta=torch.zeros(1, 20, 4, dtype=BF), normalize=True, path="scan"))
    assert (a.beta_dtype, a.dtype, a.normalize, a.path) == (_lib.KDA_BF16, _lib.KDA_BF16, 1, _lib.KDA_DELTA_SCAN)
    h = {n: t.half() if t.dtype == BF else t for n, t in _call().items()}
    a = kda.make_gated_delta_args(**h)
    assert a.dtype == _lib.KDA_F16 and a.path == _lib.KDA_DELTA_POLICY and a.lin.N == 2


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "out", "state_cache"])
def test_no_gradient_is_recorded(name):
    kw = _call()
    kw[name].requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        kda.make_gated_delta_args(**kw)
    with torch.no_grad():
        assert kda.make_gated_delta_args(**kw).lin.T == 20


def test_cpu_tensors_are_refused():
    kw = _call()
    with pytest.raises(ValueError, match="GPU"):
        kda.gated_delta_fwd(kw["q"], kw["k"], kw["v"], kw["g"], kw["beta"], kw["cu_seqlens"])
    with pytest.raises(ValueError, match="GPU"):
        kda.gated_delta_step(kw["q"], kw["k"], kw["v"], kw["g"], kw["beta"], state_cache=kw["state_cache"])


# ------------------------------------------------------------------------------ oracle
def _inputs(T, H=2, H_qk=1, K=5, V=3, seed=0):
    r = np.random.default_rng(seed)
    k = r.normal(size=(T, H_qk, K))
    return (r.normal(size=(T, H_qk, K)), k / np.linalg.norm(k, axis=-1, keepdims=True), r.normal(size=(T, H, V)), -r.random((T, H)),
            r.random((T, H)), r.normal(size=(1, H, V, K)))


def test_oracle_learns_what_it_is_shown():
    q, k, v, g, beta, S0 = _inputs(1)
    out, S, _ = delta_forward(k, k, v, g, np.ones_like(beta), [0, 1], scale=1.0, initial=S0)
    assert np.allclose(out, v)  # a full step with a unit key replaces what the key read
    out, S, _ = delta_forward(q, k, v, g, 0 * beta, [0, 1], scale=0.5, initial=S0)
    assert np.allclose(S, np.exp(g[0])[None, :, None, None] * S0) and np.allclose(out[0], 0.5 * np.einsum("hvk,k->hv", S[0], q[0, 0]))


def test_oracle_agrees_with_the_chunked_form():
    """The kernels' form, in 64 bits: T = (I + A)^-1 and products of whole chunks."""
    n = 12
    q, k, v, g, beta, S0 = _inputs(n, seed=4)
    out, S, size = delta_forward(q, k, v, g, beta, [0, n], scale=0.3, initial=S0)
    assert size[0].max() >= abs(S).max()
    for h in range(2):
        K, Q, V, b = k[:, 0], q[:, 0], v[:, h], beta[:, h]
        G = np.cumsum(g[:, h])
        decay = np.tril(np.exp(G[:, None] - G[None, :]))
        A = np.tril(b[:, None] * (K @ K.T) * decay, -1)
        D = np.linalg.solve(np.eye(n) + A, b[:, None] * (V - np.exp(G)[:, None] * (K @ S0[0, h].T)))
        O = 0.3 * (np.exp(G)[:, None] * (Q @ S0[0, h].T) + ((Q @ K.T) * decay) @ D)
        assert np.allclose(O, out[:, h], rtol=1e-12, atol=1e-13)
        assert np.allclose(np.exp(G[-1]) * S0[0, h] + D.T @ (np.exp(G[-1] - G)[:, None] * K), S[0, h], rtol=1e-12, atol=1e-13)


def test_oracle_sequences_and_groups():
    q, k, v, g, beta, _ = _inputs(9, H=4, H_qk=2, seed=8)
    out, S, _ = delta_forward(q, k, v, g, beta, [0, 4, 4, 9], scale=1.0, normalize=True)
    assert np.all(S[1] == 0)
    for n, (a, b) in enumerate(((0, 4), (4, 4), (4, 9))):
        for h in range(4):
            one = (x[a:b, h // 2:h // 2 + 1] for x in (q, k))
            o, s, _ = delta_forward(*one, v[a:b, h:h + 1], g[a:b, h:h + 1], beta[a:b, h:h + 1], [0, b - a], scale=1.0, normalize=True)
            assert np.allclose(o, out[a:b, h:h + 1]) and np.allclose(s[0, 0], S[n, h])
