"""Rotary positions in memory whose rows interleave: results beside each other or beside their inputs, one in place."""
import pytest
import torch

import gated_delta_rule_pack_amd as kda
from tests.linear_harness import DT, same_bits

pytestmark = pytest.mark.gpu

T = 37


def _call(D, dt):
    gen = torch.Generator("cpu").manual_seed(D)
    rows = torch.randn(T, 8, D, generator=gen).to(DT[dt]).cuda()  # 4 heads of q, 2 of k, 2 of v
    pos = (torch.arange(T) * 7 + 3).cuda()
    inv, _ = kda.rotary_frequencies(D // 4 * 2, device="cuda")
    want = kda.rotary(rows[:, :4].contiguous(), rows[:, 4:6].contiguous(), pos, inv)
    torch.cuda.synchronize()
    return rows, pos, inv, want


@pytest.mark.parametrize("D,dt", [(128, "bf16"), (64, "f32"), (66, "f16")])
@pytest.mark.parametrize("layout", ["columns", "beside", "q in place", "k in place", "in turn"])
def test_rows_that_interleave(layout, D, dt):
    print(f"case {layout} D={D} {dt}", flush=True)
    rows, pos, inv, want = _call(D, dt)
    before = rows.clone()
    q, k, kept = rows[:, :4], rows[:, 4:6], slice(6, 8)
    if layout == "columns":
        both = torch.full((T, 7, D), 3.0, dtype=rows.dtype, device="cuda")
        out = both[:, :4], both[:, 4:6]
        rest = [(both[:, 6], torch.full_like(both[:, 6], 3.0)), (rows, before)]
    elif layout == "beside":
        wide = torch.full((T, 16, D), 3.0, dtype=rows.dtype, device="cuda")
        wide[:, :8] = rows
        q, k, out = wide[:, :4], wide[:, 4:6], (wide[:, 8:12], wide[:, 14:16])
        rest = [(wide[:, :8], before), (wide[:, 12:14], torch.full_like(wide[:, 12:14], 3.0))]
    elif layout == "q in place":
        out = q, torch.empty_like(k, memory_format=torch.contiguous_format)
        rest = [(rows[:, 4:], before[:, 4:])]
    elif layout == "k in place":
        out = torch.empty_like(q, memory_format=torch.contiguous_format), k
        rest = [(rows[:, :4], before[:, :4]), (rows[:, 6:], before[:, 6:])]
    else:  # heads of q, k and v in turn
        turn = torch.full((T, 4, 3, D), 3.0, dtype=rows.dtype, device="cuda")
        turn[:, :, 0], turn[:, :2, 1] = rows[:, :4], rows[:, 4:6]
        q, k = turn[:, :, 0], turn[:, :2, 1]
        out = q, k
        rest = [(turn[:, 2:, 1], torch.full_like(turn[:, 2:, 1], 3.0)), (turn[:, :, 2], torch.full_like(turn[:, :, 2], 3.0))]
    got = kda.rotary(q, k, pos, inv, out_q=out[0], out_k=out[1])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert same_bits(a, b)
    for a, b in rest:
        assert same_bits(a, b)


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_through_an_autograd_function(interleaved):
    """Both calls in the halves of a function; asked for a gradient directly, the call refuses."""
    class Turn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, pos, inv):
            ctx.save_for_backward(pos, inv)
            return kda.rotary(q, None, pos, inv, interleaved=interleaved)[0]

        @staticmethod
        def backward(ctx, dy):
            return kda.rotary(dy, None, *ctx.saved_tensors, interleaved=interleaved, inverse=True)[0], None, None

    gen = torch.Generator("cpu").manual_seed(3)
    q, w = (torch.randn(9, 3, 16, generator=gen).cuda() for _ in range(2))
    pos, (inv, _) = torch.arange(9).cuda() * 11, kda.rotary_frequencies(8, device="cuda")
    leaf = q.clone().requires_grad_()
    with pytest.raises(ValueError, match="inverse=True"):
        kda.rotary(leaf, None, pos, inv, interleaved=interleaved)
    (Turn.apply(leaf, pos, inv) * w).sum().backward()
    # The same in 64 bits by torch's own derivatives.
    x = q.double().requires_grad_()
    angle = (pos.double()[:, None] * inv)[:, None]
    a, b = (x[..., 0:8:2], x[..., 1:8:2]) if interleaved else (x[..., :4], x[..., 4:8])
    pair = (a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos())
    y = torch.cat([torch.stack(pair, -1).flatten(-2) if interleaved else torch.cat(pair, -1), x[..., 8:]], -1)
    (y * w.double()).sum().backward()
    # Two products and a sum of terms no larger than w's, functions within 2 2^-24 of 1, an angle within pi 2^-24.
    assert (leaf.grad.double() - x.grad).abs().max() <= 12 * 2.0 ** -24 * 2 * w.abs().max()


@pytest.mark.parametrize("interleaved,inverse,D,rot", [(True, True, 64, 64), (False, False, 64, 64), (False, True, 66, 62)])
def test_fp32_results_lose_nothing_to_their_angles(interleaved, inverse, D, rot):
    """cos and sin are rounded to fp32 once, and then two products and their sum are: 2 2^-24 of the terms' sizes, and
    2^-24 of the result. Against 64 bits, at positions up to 2^20."""
    gen = torch.Generator("cpu").manual_seed(D + rot)
    x = torch.randn(3000, 4, D, generator=gen).cuda()
    pos = torch.randint(0, 1 << 20, (3000,), generator=gen).cuda()
    inv, _ = kda.rotary_frequencies(rot, device="cuda")
    factor = 1.25
    got, _ = kda.rotary(x, None, pos, inv, interleaved=interleaved, inverse=inverse, factor=factor)
    torch.cuda.synchronize()
    angle = (pos.double()[:, None] * inv)[:, None] * (-1 if inverse else 1)
    c, s = factor * angle.cos(), factor * angle.sin()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    ya, yb = (got[..., 0:rot:2], got[..., 1:rot:2]) if interleaved else (got[..., :rot // 2], got[..., rot // 2:rot])
    a, b = a.double(), b.double()
    for y, u, v in ((ya, a * c, -b * s), (yb, a * s, b * c)):
        room = 2.0 ** -24 * (2 * (u.abs() + v.abs()) + (u + v).abs()) * 1.001 + 1e-14
        share = ((y.double() - (u + v)).abs() / room).max().item()
        print(f"  worst element at {share:.2f} of its bound", flush=True)
        assert share <= 1.0
