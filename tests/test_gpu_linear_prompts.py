"""Prompts of linear_fwd on the GPU, beside tests/test_gpu_linear.py: what the outputs are rounded to, and every
walk and combine that the call's sizes choose, against the fp64 oracle."""
import numpy as np
import pytest
import torch

import gated_delta_rule_pack_amd as kda
from tests.linear_harness import HALF, TINY, Case, close, f64, same_bits

pytestmark = pytest.mark.gpu

U = HALF[torch.bfloat16]
# P and the state enter the products that make an output as two bf16 terms: the first is cut off (it leaves less
# than 2^-7 of the value), the second rounds what is left (2^-8 of it).
TERMS = 2.0 ** -15


def _say(msg):
    print(msg, flush=True)


def _check_out(case, out, longest=None):
    """Outputs elementwise within one rounding, the terms' rest and the fp32 sums; and all together as far off as one
    rounding is: an error uniform in half a step to either side has a mean square of step^2 / 12."""
    o, S, oa, Sa = case.oracle()
    rows = int(case.cu[-1])
    got, o, oa = f64(out).reshape(o.shape)[:rows], o[:rows], oa[:rows]
    rel = close("out", got, o, oa, TERMS, longest or max(case.lengths), U, TINY[torch.bfloat16])
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(o), 1e-30))) - 7)
    want = np.sqrt((step ** 2).sum() / 12) / np.linalg.norm(o)
    # A sum of n squares of uniform errors is off by about sqrt(0.8 / n): 1 % at 10^4, and half as much of its root.
    assert o.size >= 10_000 and rel <= 1.05 * want, f"out: rel-L2 {rel:.3e}, one rounding makes {want:.3e}"
    return S, Sa


@pytest.mark.parametrize("H,kw", [
    (2, dict()), (2, dict(K=64)), (4, dict(V=64)), (4, dict(K=64, V=64)), (2, dict(state_dtype="bf16", k_first=True)),
    (2, dict(state="none")), (2, dict(state="dense", decay="head")), (4, dict(decay="none", H_qk=2)), (14, dict()),
    (28, dict(K=64, H_qk=4)),
], ids=str)
def test_outputs_are_rounded_once(H, kw):
    case = Case([300, 70], H=H, seed=H, **kw)
    _say(f"case H={H} {kw}")
    d = case.device()
    out, final = case.forward(d, seg_len=64)
    torch.cuda.synchronize()
    _check_out(case, out)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("H,kw", [(2, dict()), (12, dict()), (2, dict(K=64)), (3, dict(V=64)), (3, dict(K=64, V=64)),
                                  (2, dict(k_first=True, state_dtype="bf16"))], ids=str)
def test_values_that_are_not_finite_reach_no_earlier_token(H, kw, bad):
    """The form is causal: such a value takes its own channel from its own token on, and nothing else."""
    case = Case([200, 100, 64, 1], H=H, seed=5, flags="all", decay="resets", **kw)
    _say(f"case H={H} {kw} bad={bad}")
    begin, end = case.cu[:-1].tolist(), case.cu[1:].tolist()
    clean = case.device()
    out, _ = case.forward(clean, seg_len=64)
    # (sequence, token in it, head, channel): in every token tile and both halves of a tile's rows, in whole and
    # short chunks, first and later ones.
    places = [(0, 0, 0, 3), (0, 15, 0, 17), (0, 16, 1, 33), (0, 62, 1, 63), (0, 63, 0, 40), (0, 64, 1, 5), (0, 100, 1, 6),
              (0, 199, 0, 7), (1, 31, 0, 8), (1, 32, 0, 9), (1, 99, 1, 10), (1, 33, 0, 9), (2, 47, 1, 62), (2, 48, 1, 61), (3, 0, 0, 1)]
    d = case.device()
    touched = torch.zeros(case.v.shape, dtype=torch.bool, device="cuda")
    channels = torch.zeros(case.N, H, case.V, dtype=torch.bool, device="cuda")
    for n, t, h, c in places:
        d["v"][begin[n] + t, h, c] = bad
        touched[begin[n] + t:end[n], h, c] = True
        channels[n, h, c] = True
    got, _ = case.forward(d, seg_len=64)
    torch.cuda.synchronize()
    assert not torch.isfinite(got[touched].float()).any()
    assert same_bits(got[~touched], out[~touched])
    planes, ref = (case.planes(x["store"])[case.indices.long().cuda()] for x in (d, clean))
    if case.k_first:
        planes, ref = planes.transpose(-1, -2), ref.transpose(-1, -2)
    assert not torch.isfinite(planes[channels].float()).any()
    assert same_bits(planes[~channels], ref[~channels])


@pytest.mark.parametrize("name", ["q", "k", "g"])
@pytest.mark.parametrize("H,V", [(2, 128), (12, 128), (2, 64)])
def test_rows_that_are_not_finite_reach_no_earlier_token(name, H, V):
    """A row of q takes its own output, one of k or g everything of its head from its token on."""
    case = Case([150, 70], H=H, V=V, seed=6, flags="all")
    clean = case.device()
    out, _ = case.forward(clean, seg_len=64)
    d = case.device()
    touched = torch.zeros(case.T, H, dtype=torch.bool, device="cuda")
    heads = torch.zeros(case.N, H, dtype=torch.bool, device="cuda")
    for n, t, end, h in ((0, 70, 150, 0), (1, 150 + 17, 220, 1)):
        d[name][t, h] = float("nan") if name == "g" else torch.tensor([float("inf"), float("nan")], device="cuda").repeat(64)
        touched[t:(t + 1 if name == "q" else end), h] = True
        heads[n, h] = name != "q"
    got, _ = case.forward(d, seg_len=64)
    torch.cuda.synchronize()
    assert torch.isnan(got[touched].float()).all()
    assert same_bits(got[~touched], out[~touched])
    planes, ref = (case.planes(x["store"])[case.indices.long().cuda()] for x in (d, clean))
    assert same_bits(planes[~heads], ref[~heads]) and (name == "q" or not torch.isfinite(planes[heads]).all(-1).any())


@pytest.mark.parametrize("entry", ["prompt", "step"])
def test_one_token_of_heads_that_lie_far_apart(entry):
    case = Case([1], H=32, seed=7, flags="all")
    d, e = case.device(), case.device()
    for n in "qkv":
        rows = torch.zeros(32, 5000, 128, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
        rows[4321] = e[n][0]
        e[n] = rows[4321:4322]
    outs = []
    for x in (d, e):
        if entry == "prompt":
            outs.append(case.forward(x)[0])
        else:
            outs.append(kda.linear_step(x["q"], x["k"], x["v"], x["g"], state_cache=x["cache"], state_indices=x["indices"]))
    torch.cuda.synchronize()
    assert same_bits(*outs) and same_bits(d["store"], e["store"])
