"""Prompts of linear_fwd on the GPU, beside tests/test_gpu_linear.py: what the outputs are rounded to, and every
walk and combine that the call's sizes choose, against the fp64 oracle."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_pack_amd as kda
from gated_delta_rule_pack_amd import _lib
from tests.linear_harness import HALF, TINY, Case, check, close, f64, same_bits

pytestmark = pytest.mark.gpu

U = HALF[torch.bfloat16]
# P and the state enter the products that make an output as two bf16 terms: the first is cut off (it leaves less
# than 2^-7 of the value), the second rounds what is left (2^-8 of it).
TERMS = 2.0 ** -15


def _say(msg):
    print(msg, flush=True)


def _once(case):
    """The oracle is the test's longest part: computed once for all its checks."""
    kept = case.oracle()
    case.oracle = lambda q=None, k=None: kept
    return case


def _check_out(case, out):
    """Outputs elementwise within one rounding, the terms' rest and the fp32 sums; and all together as far off as one
    rounding is: an error uniform in half a step to either side has a mean square of step^2 / 12."""
    o, S, oa, Sa = case.oracle()
    rows = int(case.cu[-1])
    got, o, oa = f64(out).reshape(o.shape)[:rows], o[:rows], oa[:rows]
    rel = close("out", got, o, oa, TERMS, max(case.lengths), U, TINY[torch.bfloat16])
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(o), 1e-30))) - 7)
    want = np.sqrt((step ** 2).sum() / 12) / np.linalg.norm(o)
    # A sum of n squares of uniform errors is off by about sqrt(0.8 / n): 1 % at 10^4, and half as much of its root.
    assert o.size >= 10_000 and rel <= 1.05 * want, f"out: rel-L2 {rel:.3e}, one rounding makes {want:.3e}"


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


# ------------------------------------------------------------------------------ the kernels that sizes choose
def _plan(case, seg_len):
    """(segments, segments times heads, elements of all heads' states): what the library chooses its kernels by."""
    cost = 2 if case.state == "none" else case.K * case.V * (case.initial if case.store is None else case.store).element_size() * 2 // (
        (case.K + case.V) * 4)
    axis = max(case.T, 1) + cost * (case.N - 1)
    n = -(-axis // seg_len)
    return n, n * case.H, case.H * case.K * case.V


# V = 128 and more than 128 units: the walk of all 128 state rows. At least 2^17 state elements: the combine that moves
# four at a time and 16 segments together, with a sequence that crosses more borders than that.
WHOLE = {
    "fp32 pool": dict(),
    "bf16 pool, K first": dict(state_dtype="bf16", k_first=True, pad=64),
    "fp16 pool": dict(state_dtype="f16"),
    "fp32 pool, K first": dict(k_first=True),
    "dense": dict(state="dense"),
    "dense, fp16, K first": dict(state="dense", state_dtype="f16", k_first=True),
    "no state": dict(state="none"),
    "resets": dict(decay="resets"),
    "decay for each head": dict(decay="head", g_dtype="bf16"),
    "no decay, shared q and k": dict(decay="none", H_qk=4),
    "rows of one projection": dict(fused=True, H_qk=6),
    "K = 64": dict(K=64, H=16),
    "K = 64, bf16 pool, K first": dict(K=64, H=16, state_dtype="bf16", k_first=True),
}


@pytest.mark.parametrize("name", sorted(WHOLE))
def test_walk_of_all_rows_and_wide_combine(name):
    kw = {"H": 12, **WHOLE[name]}
    case = _once(Case([1300, 0, 1, 90], seed=len(name), flags="all" if name == "resets" else "some", **kw))
    n, units, elems = _plan(case, 64)
    assert units > 128 and elems >= 1 << 17 and n > 1300 // 64 > 16
    _say(f"case {name}: {n} segments, {units} workgroups")
    d = case.device()
    out, final = case.forward(d, seg_len=64)
    torch.cuda.synchronize()
    _check_out(case, out)
    check(case, out, d, final)
    # Again, bit for bit, and with the policy's own segments.
    e = case.device()
    again, last = case.forward(e, seg_len=64)
    torch.cuda.synchronize()
    assert same_bits(again, out) and (final is None or same_bits(last, final)) and ("store" not in d or same_bits(d["store"], e["store"]))
    f = case.device()
    own, final = case.forward(f)
    torch.cuda.synchronize()
    check(case, own, f, final)


@pytest.mark.parametrize("H,K,V", [(1, 128, 64), (2, 64, 64), (1, 64, 128)])
def test_narrow_combine_over_many_segments(H, K, V):
    """Few heads: one element a thread and 32 segments together, with a sequence that crosses two such groups' borders."""
    case = _once(Case([40, 64 * 70 + 9, 0, 300], H=H, K=K, V=V, seed=K + V, decay="head"))
    n, units, elems = _plan(case, 64)
    assert elems < 1 << 17 and n > 2 * 32
    d = case.device()
    out, final = case.forward(d, seg_len=64)
    torch.cuda.synchronize()
    _check_out(case, out)
    check(case, out, d, final)


def test_middle_prompt_by_the_policy():
    """4096 tokens at 12 heads: more units than slices are for, in segments that the policy chose."""
    case = _once(Case([4096], H=12, H_qk=2, seed=8, decay="head"))
    d = case.device()
    out, final = case.forward(d)
    torch.cuda.synchronize()
    _check_out(case, out)
    check(case, out, d, final)
    e = case.device()
    again, _ = case.forward(e)
    torch.cuda.synchronize()
    assert same_bits(again, out) and same_bits(d["store"], e["store"])


def test_dense_state_in_place_of_the_walk_of_all_rows():
    case = Case([700, 0, 130], H=12, state="dense", seed=9)
    assert _plan(case, 64)[1] > 128
    d = case.device()
    state, out = d["initial"].clone(), torch.empty_like(d["v"])
    a = kda.make_linear_args(d["q"], d["k"], d["v"], d["g"], cu_seqlens=d["cu"], scale=case.scale, initial_state=state,
                             final_state=state, out=out, seg_len=64)
    lib = _lib.load()
    ws = torch.empty(lib.kda_linear_fwd_workspace_bytes(ctypes.byref(a)), dtype=torch.uint8, device="cuda")
    assert lib.kda_linear_fwd(kda.get_context("cuda:0").ptr, ctypes.byref(a), ws.data_ptr(), ws.numel(),
                              torch.cuda.current_stream().cuda_stream) == _lib.KDA_OK
    torch.cuda.synchronize()
    check(case, out, d, state)


def test_captured_prompts_of_the_walk_of_all_rows():
    """One graph, replayed with other bounds and inputs, against the eager call."""
    cases = [Case(lens, H=12, seed=30 + i, slots=8, extra_rows=900 - sum(lens)) for i, lens in enumerate(([600, 1, 299], [0, 900, 0], [64, 500, 3]))]
    assert _plan(cases[0], 64)[1] > 128
    d = cases[0].device()
    cases[0].forward(cases[0].device(), seg_len=64)
    torch.cuda.synchronize()
    out = torch.empty_like(d["v"])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            cases[0].forward(d, out=out, seg_len=64)
    torch.cuda.current_stream().wait_stream(side)
    for case in cases + cases[:1]:
        e = case.device()
        for n in ("q", "k", "v", "g", "cu", "store", "indices", "flags"):
            d[n].copy_(e[n])
        out.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref, _ = case.forward(e, out=torch.full_like(out, 7.0), seg_len=64)
        torch.cuda.synchronize()
        assert same_bits(out, ref) and same_bits(d["store"], e["store"])
        check(case, out, d, None)


@pytest.mark.parametrize("seg_len", [0, 1 << 20], ids=["policy", "one segment"])
def test_slow_decay_over_a_long_prompt(seg_len):
    """40000 tokens whose old terms live on: every chunk multiplies the state by a rounded e^{G_C}, always the same one
    where the decay is constant, so the roundings add up. Terms of one sign, so that their sums bound the results
    closely: the error stays within the harness's 3 2^-24 a chunk, 1.4e-4 here."""
    case = Case([40000], H=1, K=64, V=64, seed=10, decay="head", state="dense")
    case.g[:] = -1e-5
    case.q, case.k, case.v, case.initial = case.q.abs(), case.k.abs(), case.v.abs(), case.initial.abs()
    _once(case)
    d = case.device()
    out, final = case.forward(d, seg_len=seg_len)
    torch.cuda.synchronize()
    check(case, out, d, final)
    _check_out(case, out)


@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_tensors_of_too_few_dimensions_are_refused(name):
    case = Case([3, 4], H=2, seed=11, state="dense")
    d = case.device()
    d[name] = d[name].reshape(-1)
    with pytest.raises(ValueError, match=name):
        case.forward(d)
    with pytest.raises(ValueError, match=name):
        kda.linear_step(d["q"], d["k"], d["v"], d["g"], state_cache=torch.zeros(7, 2, 128, 128, device="cuda"))
    with pytest.raises(ValueError):
        kda.rotary(d["q"].reshape(-1), None, torch.arange(7, device="cuda"), torch.ones(4, dtype=torch.float64, device="cuda"))
