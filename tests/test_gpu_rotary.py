"""Rotary positions on the GPU against the fp64 oracle.

A result is rounded once to its type (half a step of its value), after fp32 arithmetic: two products,
their sum and the functions, each within 2^-24 of (|a| + |b|) factor; cos and sin are within 2 2^-24 of
1 for an angle reduced in 64 bits, the reduced angle's own rounding pi 2^-24."""
import numpy as np
import pytest
import torch

import gated_delta_rule_pack_amd as kda
from tests.linear_harness import DT, HALF, TINY, f64, rotate, same_bits

pytestmark = pytest.mark.gpu


def _within(name, got, x, pos, inv, dtype, **kw):
    want = rotate(f64(x), pos.numpy(), inv.numpy(), **kw)
    factor = abs(kw.get("factor", 1.0))
    r, il = inv.numel(), kw.get("interleaved", False)
    a = np.abs(f64(x))
    size = np.zeros_like(a)
    first, second = (slice(0, 2 * r, 2), slice(1, 2 * r, 2)) if il else (slice(0, r), slice(r, 2 * r))
    size[..., first] = size[..., second] = factor * (a[..., first] + a[..., second])
    room = HALF[dtype] * np.abs(want) + 12 * 2.0 ** -24 * size * (1 + HALF[dtype]) + (TINY[dtype] if dtype != torch.float32 else 0)
    off = np.abs(f64(got) - want)
    share = float(np.max(off / np.maximum(room, 1e-300))) if off.size else 0.0
    print(f"  {name}: worst element at {share:.2f} of its bound", flush=True)
    assert share <= 1.0, f"{name}: {share}"
    assert same_bits(got[..., 2 * r:].contiguous(), x[..., 2 * r:].contiguous().to(got.device))


def _inputs(T, Hq, Hk, D, dtype, seed):
    gen = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(T, Hq, D, generator=gen).to(dtype), torch.randn(T, Hk, D, generator=gen).to(dtype) if Hk else None,
            torch.randint(0, 1 << 20, (T,), generator=gen))


CASES = [
    # T, Hq, Hk, D, rot, interleaved, dtype
    (1, 1, 0, 64, 64, False, "bf16"), (1, 32, 8, 128, 128, True, "bf16"), (7, 3, 1, 128, 64, False, "f16"),
    (33, 4, 4, 80, 32, True, "f32"), (5, 2, 2, 96, 96, False, "f32"), (3, 5, 1, 256, 16, True, "f16"),
    (4, 2, 1, 10, 6, False, "bf16"), (4, 2, 1, 10, 6, True, "f32"), (9, 1, 1, 2, 2, True, "bf16"),
    (6, 2, 2, 130, 128, False, "bf16"), (2, 3, 2, 1024, 1024, False, "bf16"), (2, 3, 2, 1023, 1022, True, "f16"),
    (4100, 2, 1, 64, 64, False, "bf16"), (4099, 1, 1, 72, 40, True, "f16"), (300, 12, 12, 64, 8, False, "f32"),
]


@pytest.mark.parametrize("T,Hq,Hk,D,rot,il,dt", CASES)
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary(T, Hq, Hk, D, rot, il, dt, inverse):
    q, k, pos = _inputs(T, Hq, Hk, D, DT[dt], T + D)
    inv, _ = kda.rotary_frequencies(rot)
    print(f"case rotary {T}x({Hq}+{Hk})x{D} rot={rot} interleaved={il} {dt} inverse={inverse}", flush=True)
    kw = dict(interleaved=il, factor=1.1, inverse=inverse)
    oq, ok = kda.rotary(q.cuda(), None if k is None else k.cuda(), pos.cuda(), inv.cuda(), **kw)
    torch.cuda.synchronize()
    _within("q", oq, q, pos, inv, DT[dt], **kw)
    if k is None:
        assert ok is None
    else:
        _within("k", ok, k, pos, inv, DT[dt], **kw)


@pytest.mark.parametrize("scaling,kw", [("linear", dict(scale=8.0)), ("ntk", dict(scale=8.0)),
                                        ("yarn", dict(scale=16.0, original_length=4096))])
def test_far_positions_of_scaled_contexts(scaling, kw):
    inv, factor = kda.rotary_frequencies(128, base=500000.0, scaling=scaling, **kw)
    q, k, _ = _inputs(64, 2, 1, 128, torch.float32, 3)
    pos = torch.arange(64) * 65_537 + 3_000_000_000 * (torch.arange(64) % 2)  # past 32 bits
    oq, ok = kda.rotary(q.cuda(), k.cuda(), pos.cuda(), inv.cuda(), factor=factor)
    torch.cuda.synchronize()
    _within("q", oq, q, pos, inv, torch.float32, factor=factor)
    _within("k", ok, k, pos, inv, torch.float32, factor=factor)


def test_negative_positions():
    inv, _ = kda.rotary_frequencies(64)
    q, _, _ = _inputs(16, 2, 0, 64, torch.float32, 4)
    pos = -torch.arange(16, dtype=torch.int32) * 1000
    oq, _ = kda.rotary(q.cuda(), None, pos.cuda(), inv.cuda())
    torch.cuda.synchronize()
    _within("q", oq, q, pos, inv, torch.float32)


@pytest.mark.parametrize("D,rot,offset", [(128, 128, 0), (128, 64, 0), (64, 64, 1), (66, 60, 0)])
def test_in_place_in_the_rows_of_one_projection(D, rot, offset):
    """q and k are parts of one row buffer and are rotated in place; v and the rest stay as they were.
    offset 1 puts the rows off the 16-byte grid."""
    T, Hq, Hk = 37, 4, 2
    gen = torch.Generator("cpu").manual_seed(D)
    width = (Hq + 2 * Hk) * D
    buf = torch.randn(T * width + 8, generator=gen).bfloat16()
    rows = buf[offset: offset + T * width].view(T, width)
    dev = buf.cuda()
    drows = dev[offset: offset + T * width].view(T, width)
    q, k = (drows[:, a:b].unflatten(1, (-1, D)) for a, b in ((0, Hq * D), (Hq * D, (Hq + Hk) * D)))
    hq, hk = (rows[:, a:b].unflatten(1, (-1, D)) for a, b in ((0, Hq * D), (Hq * D, (Hq + Hk) * D)))
    pos = torch.arange(T) + 5
    inv, _ = kda.rotary_frequencies(rot)
    oq, ok = kda.rotary(q, k, pos.cuda(), inv.cuda(), out_q=q, out_k=k)
    torch.cuda.synchronize()
    assert oq is q and ok is k
    _within("q", q, hq, pos, inv, torch.bfloat16)
    _within("k", k, hk, pos, inv, torch.bfloat16)
    assert same_bits(drows[:, (Hq + Hk) * D:], rows[:, (Hq + Hk) * D:].cuda())
    assert same_bits(dev[:offset], buf[:offset].cuda()) and same_bits(dev[offset + T * width:], buf[offset + T * width:].cuda())


def test_strided_in_and_out():
    q, k, pos = _inputs(20, 3, 2, 64, torch.float16, 9)
    inv, _ = kda.rotary_frequencies(32)
    wide = torch.full((20, 7, 72), 3.0, dtype=torch.float16, device="cuda")
    kt = k.cuda().transpose(0, 1).contiguous().transpose(0, 1)  # heads outside tokens
    oq, ok = kda.rotary(q.cuda(), kt, pos.int().cuda(), inv.cuda(), interleaved=True, out_q=wide[:, 1:4, :64])
    torch.cuda.synchronize()
    _within("q", oq, q, pos, inv, torch.float16, interleaved=True)
    _within("k", ok, k, pos, inv, torch.float16, interleaved=True)
    keep = torch.ones_like(wide, dtype=torch.bool)
    keep[:, 1:4, :64] = False
    assert torch.all(wide[keep] == 3.0)


@pytest.mark.parametrize("il", [False, True])
def test_gradient(il):
    """The inverse rotation of the results' gradients is the gradient: against the formula and against
    differences (the rotation is linear in q, so a step of any size has no truncation error)."""
    T, H, D, r = 5, 2, 16, 8
    q, dy, pos = _inputs(T, H, H, D, torch.float32, 21)
    inv, _ = kda.rotary_frequencies(r)
    kw = dict(interleaved=il, factor=1.3)
    dq, _ = kda.rotary(dy.cuda(), None, pos.cuda(), inv.cuda(), inverse=True, **kw)
    y0, _ = kda.rotary(q.cuda(), None, pos.cuda(), inv.cuda(), **kw)
    torch.cuda.synchronize()
    _within("dq", dq, dy, pos, inv, torch.float32, inverse=True, **kw)
    base = float((f64(y0) * f64(dy)).sum())
    # Each loss is a sum over T H D products of values within 12 2^-24 of their pairs: 1e-6 of the sums of sizes.
    size = float((1.3 * 2 * np.abs(f64(q)).max() + 1) * np.abs(f64(dy)).sum())
    for t, h, d in ((0, 0, 0), (1, 1, 3), (4, 0, 7), (2, 1, 12)):
        e = q.clone()
        e[t, h, d] += 64.0
        y1, _ = kda.rotary(e.cuda(), None, pos.cuda(), inv.cuda(), **kw)
        torch.cuda.synchronize()
        diff = (float((f64(y1) * f64(dy)).sum()) - base) / 64.0
        # The changed pair's values are as large as 64 * 1.3: their fp32 errors, over 64.
        assert abs(diff - float(f64(dq)[t, h, d])) <= 1e-6 * (size / 64 + 4 * np.abs(f64(dy)).max())


def test_captured_rotation_replays():
    q, k, pos = _inputs(50, 4, 2, 128, torch.bfloat16, 30)
    q, k, pos = q.cuda(), k.cuda(), pos.cuda()
    inv, _ = kda.rotary_frequencies(128, device="cuda")
    kda.rotary(q, k, pos, inv)
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            oq, ok = kda.rotary(q, k, pos, inv)
    for i in range(3):
        pos.add_(i * 17)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        rq, rk = kda.rotary(q, k, pos, inv)
        torch.cuda.synchronize()
        assert same_bits(oq, rq) and same_bits(ok, rk)


def test_offsets_past_32_bits():
    """Rows whose element offsets pass 2^31, on both access paths."""
    for D, far in ((64, 1 << 30), (60, (1 << 30) + 2)):
        q, _, pos = _inputs(4, 2, 0, D, torch.bfloat16, 40)
        inv, _ = kda.rotary_frequencies(D)
        rows = torch.empty(3 * far + 2 * D, dtype=torch.bfloat16, device="cuda").as_strided((4, 2, D), (far, D, 1))
        rows.copy_(q)
        kda.rotary(rows, None, pos.cuda(), inv.cuda(), out_q=rows)
        torch.cuda.synchronize()
        _within("q", rows, q, pos, inv, torch.bfloat16)


@pytest.mark.parametrize("D, rot", [(6, 4), (16, 16)])
def test_more_tokens_than_one_launch_takes(D, rot):
    T = (1 << 22) + 1000
    inv, _ = kda.rotary_frequencies(rot, device="cuda")
    gen = torch.Generator("cuda").manual_seed(31)
    q = torch.randn(T, 1, D, device="cuda", generator=gen).bfloat16()
    k = torch.randn(T, 1, D, device="cuda", generator=gen).bfloat16()
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    out = kda.rotary(q, k, pos, inv)
    for first in (0, (1 << 22) - 500, (1 << 22) - 1, 1 << 22, T - 700):  # alone, the same tokens give the same bits
        part = slice(first, first + 700)
        want = kda.rotary(q[part], k[part], pos[part], inv)
        for got, ref in zip(out, want):
            assert torch.equal(got[part], ref)


def test_other_stream():
    q, k, pos = _inputs(50, 4, 2, 128, torch.bfloat16, 31)
    inv, _ = kda.rotary_frequencies(128)
    s = torch.cuda.Stream()
    qd, kd, pd, fd = q.cuda(), k.cuda(), pos.cuda(), inv.cuda()
    s.wait_stream(torch.cuda.current_stream())
    oq, ok = kda.rotary(qd, kd, pd, fd, stream=s)
    s.synchronize()
    _within("q", oq, q, pos, inv, torch.bfloat16)
    _within("k", ok, k, pos, inv, torch.bfloat16)
