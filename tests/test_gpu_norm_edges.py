"""The q/k norm's calls at the edges of what they allow: sizes far from one, values that are not finite, layouts, streams, captured
calls, token counts around the workgroups' shares, and the gradient against differences of the forward pass."""
import threading

import numpy as np
import pytest
import torch

import gated_delta_rule_pack_amd as kda
from oracle import qk_norm, qk_norm_gradient
from tests.linear_harness import DT, HALF, TINY, f64, same_bits
from tests.test_gpu_norm import make, near, oracle_kw

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def on_device(s):
    return {n: None if t is None else t.cuda() for n, t in s.items()}


def forward(d, kw, **more):
    return kda.qk_norm(d["q"], d["k"], d["qw"], d["kw"], d["pos"], d["freq"], **kw, **more)


def backward(d, kw, **more):
    return kda.qk_norm_backward(d["gq"], d["gk"], d["q"], d["k"], d["qw"], d["kw"], d["pos"], d["freq"], **kw, **more)


def check_forward(s, kw, q, k):
    for n, got, w in (("q", q, "qw"), ("k", k, "kw")):
        if got is not None:
            want = qk_norm(f64(s[n]), None if s[w] is None else f64(s[w]), **oracle_kw(s, kw))
            near(n, f64(got), want, HALF[got.dtype] * np.abs(want) + 2.0 ** -20 * np.abs(want).max(-1, keepdims=True) + TINY[got.dtype])


# Sizes of x whose squares leave 32 bits at either end, in a wide and a narrow layout.
@pytest.mark.parametrize("kind", ["rms", "l2"])
@pytest.mark.parametrize("D,dtype", [(128, "f32"), (72, "f32"), (200, "f32"), (128, "bf16"), (128, "f16")])
@pytest.mark.parametrize("size", [2.0 ** 120, 2.0 ** 60, 2.0 ** 14, 2.0 ** -14, 2.0 ** -60])
def test_rows_of_any_size(size, D, dtype, kind):
    if dtype == "f16" and not 2.0 ** -15 < size < 2.0 ** 13:
        size = 2.0 ** 12 if size > 1 else 2.0 ** -12
    s, kw = make(T=5, D=D, rot=0 if D == 200 else D, dtype=dtype, kind=kind)
    for n in "qk":
        x = s[n].float()
        s[n] = (x / x.abs().amax(-1, keepdim=True) * size).to(DT[dtype])
    d = on_device(s)
    check_forward(s, kw, *forward(d, kw))


@pytest.mark.parametrize("D", [64, 65, 128, 200])
def test_zero_rows(D):
    s, kw = make(T=4, D=D, rot=0, offset=1.0)
    s["q"][2], s["k"][0, 1] = 0, 0
    d = on_device(s)
    q, k = forward(d, kw)
    assert torch.all(q[2] == 0) and torch.all(k[0, 1] == 0)
    dq, dk, _, _ = backward(d, kw)
    # There r = 1 / sqrt(eps) and dx = r u.
    want = f64(s["gq"])[2] * (1 + f64(s["qw"])) * 1e3
    near("dq", f64(dq)[2], want, (2.0 ** -8 + 2.0 ** -18) * np.abs(want) + 1e-3)


@pytest.mark.parametrize("D", [128, 65, 200])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_what_is_not_finite_stays_in_its_row(D, bad):
    s, kw = make(T=9, D=D, rot=0)
    d = on_device(s)
    q, k = forward(d, kw)
    dq, dk, dqw, dkw = backward(d, kw)
    d["q"][4, 3, 7] = bad
    q2, k2 = forward(d, kw)
    dq2, dk2, dqw2, dkw2 = backward(d, kw)
    rest = torch.ones(9, 6, dtype=torch.bool, device="cuda")
    rest[4, 3] = False
    assert same_bits(q2[rest], q[rest]) and same_bits(k2, k) and torch.isnan(q2[4, 3]).all()
    assert same_bits(dq2[rest], dq[rest]) and same_bits(dk2, dk) and torch.isnan(dq2[4, 3]).all()
    assert same_bits(dkw2, dkw) and torch.isnan(dqw2).all()


# Shares of the workgroups' walks: 512 and 1024 of them, up to 4 or 8 tokens at a time.
@pytest.mark.parametrize("T", [1, 2, 511, 513, 1023, 1025, 2047, 4097, 5003])
def test_token_counts(T):
    s, kw = make(T=T, Hq=3, Hk=1, D=64)
    d = on_device(s)
    check_forward(s, kw, *forward(d, kw))
    dq, dk, dqw, dkw = backward(d, kw)
    for n, got, gw, w in (("q", dq, dqw, "qw"), ("k", dk, dkw, "kw")):
        x, dy, wide = f64(s[n]), f64(s["g" + n]), f64(s[w])
        want, wantw = qk_norm_gradient(dy, x, wide, **oracle_kw(s, kw))
        size = np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
        u = np.sqrt((dy * dy).sum(-1, keepdims=True)) * np.abs(wide).max()
        near("d" + n, f64(got), want, 2.0 ** -8 * np.abs(want) + (2.0 ** -20 + 64 * 2.0 ** -24) * u / size)
        rows = x.shape[0] * x.shape[1]
        terms = np.sqrt(((np.abs(dy).max(-1, keepdims=True) * x / size) ** 2).sum((0, 1))) * 2 ** 0.5
        near("d" + w, f64(gw), wantw, 2.0 ** -8 * np.abs(wantw) + rows ** 0.5 * (2.0 ** -20 + rows ** 0.5 * 2.0 ** -23) * terms)


@pytest.mark.parametrize("Hq,Hk,D", [(1, 0, 128), (64, 8, 128), (7, 5, 256), (300, 1, 16), (1, 1, 8)])
def test_head_counts(Hq, Hk, D):
    s, kw = make(T=33, Hq=Hq, Hk=Hk, D=D)
    d = on_device(s)
    check_forward(s, kw, *forward(d, kw))
    dq, _, _, _ = backward(d, kw)
    want, _ = qk_norm_gradient(f64(s["gq"]), f64(s["q"]), f64(s["qw"]), **oracle_kw(s, kw))
    x = f64(s["q"])
    room = np.sqrt((f64(s["gq"]) ** 2).sum(-1, keepdims=True)) * np.abs(f64(s["qw"])).max() / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
    near("dq", f64(dq), want, 2.0 ** -8 * np.abs(want) + (2.0 ** -20 + D * 2.0 ** -24) * room)


def test_no_tokens():
    s, kw = make(T=3)
    d = on_device(s)
    for n in ("q", "k", "gq", "gk", "pos"):
        d[n] = d[n][:0]
    q, k = forward(d, kw)
    assert q.shape == (0, 6, 128) and k.shape == (0, 2, 128)
    _, _, dqw, dkw = backward(d, kw)
    assert torch.all(dqw == 0) and torch.all(dkw == 0)


# ------------------------------------------------------------------------------ layouts
@pytest.mark.parametrize("offset", [0, 1, 2, 4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_columns_of_one_projection_in_place(offset, dtype):
    """q and k are columns of one row, at addresses of every alignment; the rest of the row stays as it was."""
    s, kw = make(T=21, Hq=4, Hk=2, D=64, dtype=dtype)
    width = 4 * 64 + 2 * 64 + 24
    row = torch.full((21, width), 7.0, dtype=DT[dtype], device="cuda")
    q = row[:, offset:offset + 256].unflatten(1, (4, 64))
    k = row[:, offset + 256:offset + 384].unflatten(1, (2, 64))
    q.copy_(s["q"]), k.copy_(s["k"])
    d = dict(on_device(s), q=q, k=k)
    forward(d, kw, out_q=q, out_k=k)
    check_forward(s, kw, q, k)
    assert torch.all(row[:, :offset] == 7.0) and torch.all(row[:, offset + 384:] == 7.0)


@pytest.mark.parametrize("D,rot", [(128, 128), (65, 0), (200, 50)])
def test_backward_in_place_of_the_gradients(D, rot):
    s, kw = make(T=700, Hq=5, Hk=2, D=D, rot=rot)
    d = on_device(s)
    want = backward(d, kw)
    got = backward(d, kw, out_q=d["gq"], out_k=d["gk"])
    assert got[0] is d["gq"] and all(same_bits(a, b) for a, b in zip(got, want))


def test_heads_of_q_and_k_in_turn():
    s, kw = make(T=30, Hq=3, Hk=3, D=64)
    both = torch.stack([s["q"], s["k"]], 2).cuda()  # [T, H, 2, D]
    d = dict(on_device(s), q=both[:, :, 0], k=both[:, :, 1])
    forward(d, kw, out_q=d["q"], out_k=d["k"])
    check_forward(s, kw, d["q"], d["k"])


def test_strided_gradients_and_broadcast_rows():
    s, kw = make(T=40, Hq=4, Hk=2)
    d = on_device(s)
    want = backward(d, kw)
    wide = torch.zeros(40, 4, 256, dtype=torch.bfloat16, device="cuda")
    wide[..., :128] = d["gq"]
    got = backward(dict(d, gq=wide[..., :128]), kw)
    assert all(same_bits(a, b) for a, b in zip(got, want))
    one = d["gq"][:, :1]  # a gradient that every head shares
    got = backward(dict(d, gq=one.expand(-1, 4, -1)), kw)
    want = backward(dict(d, gq=one.repeat(1, 4, 1)), kw)
    assert all(same_bits(a, b) for a, b in zip(got, want))


def test_offsets_past_32_bits():
    T = 300
    s, kw = make(T=T, Hq=2, Hk=1)
    d = on_device(s)
    want = forward(d, kw), backward(d, kw)
    rows = torch.empty(T << 23, dtype=torch.bfloat16, device="cuda")  # 5 GB, 2^23 elements between tokens
    q = rows.as_strided((T, 2, 128), (1 << 23, 128, 1))
    q.copy_(d["q"])
    out = rows.as_strided((T, 2, 128), (1 << 23, 128, 1), 1 << 12)
    far = dict(d, q=q)
    assert same_bits(forward(far, kw, out_q=out)[0], want[0][0])
    assert all(same_bits(a, b) for a, b in zip(backward(far, kw, out_q=out), want[1]))


# ------------------------------------------------------------------------------ streams
def test_other_stream_and_given_workspace():
    s, kw = make(T=600)
    d = on_device(s)
    want = backward(d, kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = backward(d, kw, stream=side, workspace=torch.empty(8 << 20, dtype=torch.uint8, device="cuda"))
    q, k = forward(d, kw, stream=side)
    side.synchronize()
    assert all(same_bits(a, b) for a, b in zip(got, want))
    check_forward(s, kw, q, k)


def test_two_threads():
    sets = [make(T=900, seed=i) for i in range(2)]
    data = [on_device(s) for s, _ in sets]
    want = [backward(d, kw) for d, (_, kw) in zip(data, sets)]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(20):
                got[i] = backward(data[i], sets[i][1], stream=stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i in range(2):
        assert all(same_bits(a, b) for a, b in zip(got[i], want[i]))


def test_captured_calls_replay():
    """Both passes in one graph, with other rows and positions at each replay and the program's own work between."""
    s, kw = make(T=1300, Hq=3, Hk=1, weight="f32")
    d = on_device(s)
    forward(d, kw), backward(d, kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            got = (*forward(d, kw), *backward(d, kw))
    torch.cuda.current_stream().wait_stream(side)
    for r in range(4):
        t, _ = make(T=1300, Hq=3, Hk=1, weight="f32", seed=100 + r)
        e = on_device(t)
        for n, x in e.items():
            d[n].copy_(x)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = (*forward(e, kw), *backward(e, kw))
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(got, want)), f"replay {r}"


# ------------------------------------------------------------------------------ the gradient
@pytest.mark.parametrize("kind", ["rms", "l2"])
@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (64, 32, True), (65, 20, False), (72, 36, True), (200, 50, False)])
def test_gradient_against_differences(D, rot, interleaved, kind):
    """Along a direction e: (dy . (y(x + h e) - y(x - h e))) / 2 h of the formula in 64 bits against dx . e, h = 1e-5: the
    difference is off by h^2 times a third derivative (below 1e-7 of the sizes' product), the gradient by its fp32 roundings."""
    s, kw = make(T=6, D=D, rot=rot, interleaved=interleaved, dtype="f32", kind=kind, offset=1.0)
    d = on_device(s)
    dq, dk, dqw, dkw = backward(d, kw)
    gen = np.random.default_rng(D)
    ok = oracle_kw(s, kw)
    for n, dx, dw, w in (("q", dq, dqw, "qw"), ("k", dk, dkw, "kw")):
        x, dy, wide = f64(s[n]), f64(s["g" + n]), f64(s[w])
        e = gen.normal(size=x.shape) * np.abs(x).max(-1, keepdims=True)
        h = 1e-5
        slope = (dy * (qk_norm(x + h * e, wide, **ok) - qk_norm(x - h * e, wide, **ok))).sum((1, 2)) / (2 * h)
        size = np.sqrt((dy ** 2).sum((1, 2)) * (e ** 2).sum((1, 2))) * np.abs(1 + wide).max()
        size /= np.sqrt((x * x).sum(-1).min(-1) * (1 if ok["l2"] else 1 / D))
        assert np.all(np.abs((f64(dx) * e).sum((1, 2)) - slope) < 1e-5 * size)
        e = gen.normal(size=D)
        slope = (dy * (qk_norm(x, wide + h * e, **ok) - qk_norm(x, wide - h * e, **ok))).sum() / (2 * h)
        assert abs((f64(dw) * e).sum() - slope) < 1e-5 * np.sqrt((dy ** 2).sum() * (e ** 2).sum() * x.shape[0] * x.shape[1]) * max(1, D ** 0.5 if not ok["l2"] else 1)


def test_gradient_through_an_autograd_function():
    """The two halves of a training program's own function, beside the formula's gradient by the library."""
    s, kw = make(T=12, D=64, dtype="f32")
    d = on_device(s)

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, qw, kw_):
            ctx.save_for_backward(q, k, qw, kw_)
            return kda.qk_norm(q, k, qw, kw_, d["pos"], d["freq"])

        @staticmethod
        def backward(ctx, gq, gk):
            return kda.qk_norm_backward(gq.contiguous(), gk.contiguous(), *ctx.saved_tensors, d["pos"], d["freq"])

    leaves = [d[n].detach().clone().requires_grad_() for n in ("q", "k", "qw", "kw")]
    q, k = Norm.apply(*leaves)
    torch.autograd.backward([q, k], [d["gq"], d["gk"]])
    want = backward(d, kw)
    assert all(same_bits(t.grad, w) for t, w in zip(leaves, want))


def test_refused_calls_on_the_device():
    s, kw = make(T=5)
    d = on_device(s)
    with pytest.raises(kda.KDAError):
        forward(d, kw, out_q=torch.empty_like(d["q"]), out_k=d["q"][:, :2])
    with pytest.raises(kda.KDAError):
        backward(d, kw, out_q=d["q"])
    with pytest.raises(ValueError):
        kda.qk_norm_backward(None, d["gk"], d["q"], d["k"])
    with pytest.raises(ValueError):
        forward(dict(d, qw=d["qw"].cpu()), kw)
    with pytest.raises(TypeError):
        backward(d, kw, workspace=torch.empty(4, device="cuda"))
    with pytest.raises(ValueError):
        forward(dict(d, q=d["q"].float().requires_grad_()), kw)


def test_a_given_workspace_that_does_not_serve_is_refused():
    q = torch.randn(600, 3, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    big = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for ws in (big[:1000], big[128:]):
        with pytest.raises(kda.KDAError, match="workspace"):
            kda.qk_norm_backward(q, None, q, None, w, workspace=ws)
    got = kda.qk_norm_backward(q, None, q, None, w, workspace=big)
    want = kda.qk_norm_backward(q, None, q, None, w)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    assert kda.qk_norm_backward(q, None, q, None, workspace=big[:1])[2] is None  # no weights: none is needed


@pytest.mark.parametrize("T,H,D,rot,interleaved", [(1001, 12, 72, 36, True), (1001, 12, 72, 36, False), (513, 3, 65, 64, False), (4096, 8, 128, 128, False)])
def test_weight_gradients_sum_in_pairs(T, H, D, rot, interleaved):
    """n terms of one size and random signs: with e = 0.735 2^-24 (the half step's share of a value is 2^-24 at its lowest, 0.735 of that in
    the mean square over all values) a chain of m partial sums is off by e sqrt(m / 6) of its result, rms, pairs of pairs by e sqrt(log2(m) /
    3). The terms carry five roundings each, 1.3 e. Here chains hold at most 16 rows of a lane (1.6) and 8 in each four of a workgroup's
    groups (1.1 and 0.8), then two in each four of a channel's 8 workgroups (0.6 and 0.8), and pairs of 64 (1.4): 3.1 e = 2.3 2^-24 in all at
    most. One chain of 64 (3.3) instead of pairs makes 2.8 2^-24 and more."""
    gen = torch.Generator().manual_seed(12)
    q, gq = (torch.randn(T, H, D, generator=gen) for _ in range(2))
    w = 1 + 0.2 * torch.randn(D, generator=gen)
    pos, freq = torch.arange(T), 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    _, _, got, _ = kda.qk_norm_backward(gq.cuda(), None, q.cuda(), None, w.cuda(), None, pos.cuda(), freq.cuda(), interleaved=interleaved)
    _, want = qk_norm_gradient(f64(gq), f64(q), f64(w), positions=f64(pos), inv_freq=f64(freq), interleaved=interleaved)
    rel = np.linalg.norm(f64(got) - want) / np.linalg.norm(want)
    print(f"  dw: rel-L2 {rel * 2 ** 24:.2f} 2^-24", flush=True)
    assert rel < 2.5 * 2.0 ** -24
