"""Linear attention with a decay for each head on the GPU: prompts (linear_fwd) and single tokens
(linear_step), against the fp64 oracle, with elementwise bounds (tests/linear_harness.py)."""
import numpy as np
import pytest
import torch

import gated_delta_rule_pack_amd as kda
from tests.linear_harness import DT, HALF, TINY, Case, check, close, f64, rotate, same_bits

pytestmark = pytest.mark.gpu


def _say(msg):
    print(msg, flush=True)


PROMPTS = {
    # Lengths around the 64-token chunk and the segment borders, empty sequences first, last and between.
    "one_token": dict(lengths=[1]),
    "short": dict(lengths=[5, 0, 17]),
    "chunk_edges": dict(lengths=[63, 64, 65, 127, 128, 129]),
    "empties": dict(lengths=[0, 0, 40, 0, 1, 0, 90, 0]),
    "all_empty": dict(lengths=[0, 0, 0]),
    "ragged": dict(lengths=[300, 1, 0, 77, 200, 2], H=3),
    "singles": dict(lengths=[1] * 70, H=1),
    "k64": dict(lengths=[100, 31], K=64, V=128),
    "v64": dict(lengths=[100, 31], K=128, V=64),
    "kv64": dict(lengths=[100, 31], K=64, V=64, H=3),
    "grouped": dict(lengths=[150, 40], H=6, H_qk=2),
    "one_qk_head": dict(lengths=[70, 3], H=5, H_qk=1, V=64),
    "head_decay": dict(lengths=[200, 70], decay="head"),
    "no_decay": dict(lengths=[200, 70], decay="none"),
    "resets": dict(lengths=[200, 70, 1, 64], decay="resets"),
    "bf16_decay": dict(lengths=[130], g_dtype="bf16"),
    "bf16_head_decay": dict(lengths=[130], decay="head", g_dtype="bf16"),
    "fused_rows": dict(lengths=[100, 29], H=4, H_qk=2, fused=True),
    "dense": dict(lengths=[90, 0, 65], state="dense"),
    "dense_f16_kfirst": dict(lengths=[90, 0, 65], state="dense", state_dtype="f16", k_first=True),
    "no_state": dict(lengths=[90, 0, 65], state="none"),
    "bf16_pool": dict(lengths=[90, 0, 65], state_dtype="bf16", pad=64),
    "f16_pool_kfirst": dict(lengths=[90, 0, 65], state_dtype="f16", k_first=True, pad=8),
    "f32_pool_kfirst_v64": dict(lengths=[90, 0, 65], V=64, k_first=True),
    "rows_behind": dict(lengths=[33, 40], extra_rows=9),
    "growth": dict(lengths=[130, 1], decay="growth"),
    "singles_among_prompts": dict(lengths=[1, 70, 1, 0, 1, 1, 2, 1, 130], H=4, H_qk=2, state_dtype="f16", k_first=True),
    "singles_no_state": dict(lengths=[1, 1, 3, 1], state="none", decay="none"),
}


@pytest.mark.parametrize("seg_len", [0, 64, 128], ids=["policy", "seg64", "seg128"])
@pytest.mark.parametrize("name", sorted(PROMPTS))
def test_prompts(name, seg_len):
    case = Case(**PROMPTS[name], seed=len(name))
    _say(f"case {name} seg_len={seg_len}")
    d = case.device()
    out = torch.full_like(d["v"], 7.0, memory_format=torch.contiguous_format)
    before = None if case.state != "paged" else d["store"].clone()
    got, final = case.forward(d, out=out, seg_len=seg_len)
    torch.cuda.synchronize()
    assert got is out
    check(case, got, d, final)
    rows = int(case.cu[-1])
    assert torch.all(got[rows:] == 7.0)  # rows behind the last sequence
    if before is not None:  # other slots and the padding between slots keep their bits
        used = set(case.indices.tolist())
        for s in range(case.slots):
            if s not in used:
                assert same_bits(d["store"][s], before[s])
            assert same_bits(d["store"][s, case.H * case.K * case.V:], before[s, case.H * case.K * case.V:])


def test_long_prompt_many_segments():
    case = Case([1500, 0, 700], H=2, decay="head", seed=3)
    d = case.device()
    out, final = case.forward(d)
    torch.cuda.synchronize()
    check(case, out, d, final)


def test_segments_do_not_change_single_segment_results_beyond_rounding():
    """A state carried over a border is the fp32 state a single walk would hold, up to fp32 sums."""
    case = Case([400], H=1, state="dense", seed=5)
    d = case.device()
    finals = [case.forward(d, seg_len=L)[1] for L in (64, 192, 448)]
    torch.cuda.synchronize()
    _, S, _, Sa = case.oracle()
    for f in finals:
        close("state", f64(f), S, Sa, 0.0, 400, HALF[torch.float32])


def test_calls_repeat_bit_for_bit():
    case = Case([300, 20, 500], H=3, seed=6)
    d = case.device()
    store = d["store"].clone()
    first = case.forward(d, seg_len=64)[0].clone()
    after = d["store"].clone()
    for _ in range(3):
        d["store"].copy_(store)
        again, _ = case.forward(d, seg_len=64)
        assert same_bits(again, first) and same_bits(d["store"], after)


def test_dense_state_in_place():
    """initial_state and final_state may be the same memory, also where a sequence spans segments."""
    case = Case([300, 0, 40], H=2, state="dense", seed=7)
    d = case.device()
    state = d["initial"].clone()
    out = torch.empty_like(d["v"])
    a = kda.make_linear_args(d["q"], d["k"], d["v"], d["g"], cu_seqlens=d["cu"], initial_state=state, final_state=state,
                             out=out, seg_len=64)
    from gated_delta_rule_pack_amd import _lib
    import ctypes
    lib = _lib.load()
    ws = torch.empty(lib.kda_linear_fwd_workspace_bytes(ctypes.byref(a)), dtype=torch.uint8, device="cuda")
    rc = lib.kda_linear_fwd(kda.get_context("cuda:0").ptr, ctypes.byref(a), ws.data_ptr(), ws.numel(),
                            torch.cuda.current_stream().cuda_stream)
    assert rc == _lib.KDA_OK
    torch.cuda.synchronize()
    check(case, out, d, state)


def test_slots_outside_the_pool_are_no_slots():
    case = Case([80, 30, 0, 1], H=2, seed=8, flags="all")
    case.indices[1], case.indices[2] = -1, case.slots
    d = case.device()
    before = d["store"].clone()
    out, _ = case.forward(d, seg_len=64)
    torch.cuda.synchronize()
    check(case, out, d, None)
    used = {int(case.indices[0]), int(case.indices[3])}
    for s in range(case.slots):
        if s not in used:
            assert same_bits(d["store"][s], before[s])


def test_strided_output_and_padded_heads():
    case = Case([70, 20], H=3, seed=9, V=64)
    d = case.device()
    wide = torch.full((case.T, 4, 80), 7.0, dtype=torch.bfloat16, device="cuda")
    out, _ = case.forward(d, out=wide[:, :3, :64])
    torch.cuda.synchronize()
    check(case, out, d, None)
    assert torch.all(wide[:, 3] == 7.0) and torch.all(wide[:, :, 64:] == 7.0)


def test_another_stream_and_given_workspace():
    case = Case([200, 90], H=2, seed=10)
    d = case.device()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, _ = case.forward(d, stream=side, seg_len=64, workspace=torch.empty(64 << 20, dtype=torch.uint8, device="cuda"))
    side.synchronize()
    check(case, out, d, None)


def test_broadcast_rows():
    """q and k with stride 0 over heads (one head's rows shown as several)."""
    case = Case([100], H=3, H_qk=1, seed=11)
    d = case.device()
    shared = dict(d, q=d["q"].expand(-1, 3, -1), k=d["k"].expand(-1, 3, -1))
    out, _ = case.forward(shared)
    torch.cuda.synchronize()
    check(case, out, d, None)


@pytest.mark.parametrize("entry", ["prompt", "step"])
def test_broadcast_row_of_one_token(entry):
    """One token whose q and k heads are one row (all strides 0)."""
    case = Case([1], H=3, H_qk=1, seed=61, flags="all")
    shared = {n: getattr(case, n).cuda().expand(-1, 3, -1) for n in "qk"}
    outs = []
    for q, k in ((case.q.cuda(), case.k.cuda()), (shared["q"], shared["k"])):
        d = dict(case.device(), q=q, k=k)
        if entry == "prompt":
            out, _ = case.forward(d)
        else:
            out = kda.linear_step(q, k, d["v"], d["g"], state_cache=d["cache"], state_indices=d["indices"])
        outs.append((out, d["store"]))
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_prompts_with_rotary_positions():
    case = Case([150, 40], H=4, H_qk=2, K=128, seed=12, state="dense")
    d = case.device()
    inv, _ = kda.rotary_frequencies(64, device="cuda")
    pos = torch.cat([torch.arange(150) + 1000, torch.arange(40)])
    out, final = case.forward(d, positions=pos.cuda(), inv_freq=inv, interleaved=True)
    torch.cuda.synchronize()
    q, k = (rotate(f64(x), pos.numpy(), inv.cpu().numpy(), interleaved=True) for x in (case.q, case.k))
    # Rotated q and k are rounded to bf16: a term of the rotation is at most |a| + |b| <= sqrt(2) of its
    # pair's length, which the sums of absolute rotated values do not bound elementwise, so the call is
    # held to the same call on rows that the rotary kernel has rounded.
    rq, rk = kda.rotary(d["q"], d["k"], pos.cuda(), inv, interleaved=True)
    torch.cuda.synchronize()
    assert np.linalg.norm(f64(rq) - q) <= 2 ** -8 * np.linalg.norm(q)
    check(case, out, d, final, q=f64(rq), k=f64(rk))


def test_prompt_then_single_tokens():
    """The operators as they are used: prompts fill the pool, then requests go on token by token, with
    rotated q and k throughout."""
    steps, H, H_qk, K = 5, 4, 2, 128
    lens = [70, 0, 33]
    whole = Case([n + steps for n in lens], H=H, H_qk=H_qk, seed=13, state="none")
    inv, factor = kda.rotary_frequencies(K, scaling="yarn", scale=4.0, original_length=64, device="cuda")
    cache = torch.full((6, H, 128, K), float("nan"), device="cuda")
    idx = torch.tensor([4, 1, 3], dtype=torch.int32, device="cuda")
    flags = torch.zeros(3, dtype=torch.bool, device="cuda")
    d = whole.device()
    begin = whole.cu[:-1].tolist()
    rows = torch.cat([torch.arange(b, b + n) for b, n in zip(begin, lens)]).cuda()
    pos = torch.cat([torch.arange(n) for n in lens]).cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    rot = dict(inv_freq=inv, rotary_factor=factor)
    got = torch.full(whole.v.shape, float("nan"))
    out, _ = kda.linear_fwd(d["q"][rows], d["k"][rows], d["v"][rows], d["g"][rows], cu, state_cache=cache, state_indices=idx,
                            has_initial_state=flags, positions=pos, **rot)
    got[rows.cpu()] = out.float().cpu()
    for s in range(steps):
        row = torch.tensor([b + n + s for b, n in zip(begin, lens)], device="cuda")
        at = torch.tensor([n + s for n in lens], device="cuda")
        out = kda.linear_step(d["q"][row], d["k"][row], d["v"][row], d["g"][row], state_cache=cache, state_indices=idx,
                              positions=at, **rot)
        got[row.cpu()] = out.float().cpu()
    at = np.concatenate([np.arange(n + steps) for n in lens])
    q, k = (rotate(f64(x), at, inv.cpu().numpy(), factor=factor) for x in (whole.q, whole.k))
    o, S, oa, Sa = whole.oracle(q, k)
    # Prompts: q and k rounded once more each (u of a value each), beside the roundings of the walk.
    u = 2.0 ** -8
    close("out", got.double().numpy(), o, oa, 4 * u, 80, u)
    fin = f64(cache[idx.long()])
    close("state", fin, S, Sa, u, 80, 2.0 ** -24)


# ------------------------------------------------------------------------------ single tokens
STEPS = {
    "one": dict(lengths=[1]),
    "some": dict(lengths=[1] * 7, H=3),
    "many": dict(lengths=[1] * 130, H=2),
    "k64": dict(lengths=[1] * 5, K=64),
    "v64": dict(lengths=[1] * 5, V=64),
    "kv64_kfirst": dict(lengths=[1] * 5, K=64, V=64, k_first=True),
    "k64_kfirst": dict(lengths=[1] * 5, K=64, k_first=True),
    "v64_kfirst_f16": dict(lengths=[1] * 5, V=64, k_first=True, state_dtype="f16"),
    "kfirst": dict(lengths=[1] * 5, k_first=True, pad=64),
    "bf16": dict(lengths=[1] * 9, state_dtype="bf16", pad=8),
    "f16": dict(lengths=[1] * 9, state_dtype="f16"),
    "bf16_kfirst": dict(lengths=[1] * 9, state_dtype="bf16", k_first=True),
    "grouped": dict(lengths=[1] * 6, H=6, H_qk=2),
    "head_decay": dict(lengths=[1] * 6, decay="head"),
    "no_decay": dict(lengths=[1] * 6, decay="none"),
    "resets": dict(lengths=[1] * 64, decay="resets"),
    "bf16_decay": dict(lengths=[1] * 6, g_dtype="bf16"),
    "fused_rows": dict(lengths=[1] * 6, H=4, H_qk=2, fused=True),
}


def _step(case, d, **kw):
    return kda.linear_step(d["q"], d["k"], d["v"], d["g"], state_cache=d["cache"], state_indices=d["indices"],
                           has_initial_state=d["flags"], scale=case.scale, state_k_first=case.k_first, **kw)


def _check_step(case, d, out, q=None, k=None, rows=None):
    o, S, oa, Sa = case.oracle(q, k)
    rows = slice(None) if rows is None else rows
    # fp32 throughout: the result's rounding, and sums of K terms.
    close("out", f64(out)[rows], o[rows], oa[rows], 0.0, 1, HALF[torch.bfloat16], TINY[torch.bfloat16])
    sdt = case.store.dtype
    close("state", case.finals(d, None)[rows], S[rows], Sa[rows], 0.0, 1, HALF[sdt], TINY[sdt])


@pytest.mark.parametrize("name", sorted(STEPS))
def test_steps(name):
    case = Case(**STEPS[name], seed=len(name) + 40)
    _say(f"case step {name}")
    d = case.device()
    before = d["store"].clone()
    out = _step(case, d)
    torch.cuda.synchronize()
    _check_step(case, d, out)
    used, plane = set(case.indices.tolist()), case.H * case.K * case.V
    for s in range(case.slots):
        if s not in used:
            assert same_bits(d["store"][s], before[s])
        assert same_bits(d["store"][s, plane:], before[s, plane:])


@pytest.mark.parametrize("rot,interleaved,i64", [(128, False, True), (64, True, False), (2, True, True), (30, False, False)])
@pytest.mark.parametrize("k_first", [False, True])
def test_steps_with_rotary_positions(rot, interleaved, i64, k_first):
    case = Case([1] * 6, H=4, H_qk=2, k_first=k_first, seed=rot, flags="all")
    _say(f"case step rot={rot} interleaved={interleaved} k_first={k_first}")
    d = case.device()
    inv, _ = kda.rotary_frequencies(rot, device="cuda")
    pos = torch.tensor([0, 1, 77, 4096, 999_983, 1 << 22])
    out = _step(case, d, positions=(pos if i64 else pos.int()).cuda(), inv_freq=inv, interleaved=interleaved, rotary_factor=1.25)
    torch.cuda.synchronize()
    q, k = (rotate(f64(x), pos.numpy(), inv.cpu().numpy(), interleaved=interleaved, factor=1.25) for x in (case.q, case.k))
    # Rotation in fp32: four roundings and two functions within 2 2^-24, of terms as large as 1.25
    # (|a| + |b|); q and k pairs enter the sums of sizes through their absolute rotated values, so the
    # sizes are taken from the unrotated pairs' lengths instead.
    o, S, _, _ = case.oracle(q, k)
    size = [np.broadcast_to(1.25 * np.sqrt(2) * np.abs(f64(x)).max(axis=-1, keepdims=True), x.shape) for x in (case.q, case.k)]
    _, _, oa, Sa = case.oracle(*size)
    close("out", f64(out), o, oa, 16 * 2.0 ** -24, 1, HALF[torch.bfloat16])
    close("state", case.finals(d, None), S, Sa, 8 * 2.0 ** -24, 1, HALF[torch.float32])


def test_step_padding_rows_are_left_alone():
    case = Case([1] * 6, H=2, seed=50, flags="all")
    keep = [0, 2, 5]
    for n in (1, 3, 4):
        case.indices[n] = {1: -1, 3: case.slots, 4: -(1 << 30)}[n]
    d = case.device()
    before = d["store"].clone()
    out = torch.full_like(d["v"], 7.0)
    _step(case, d, out=out)
    torch.cuda.synchronize()
    _check_step(case, d, out, rows=keep)
    assert torch.all(out[[1, 3, 4]] == 7.0)
    used = {int(case.indices[n]) for n in keep}
    for s in range(case.slots):
        if s not in used:
            assert same_bits(d["store"][s], before[s])


def test_step_without_indices_takes_slot_n():
    case = Case([1] * 4, H=2, seed=51, flags="all", slots=6)
    case.indices = torch.arange(4, dtype=torch.int32)
    d = case.device()
    out = kda.linear_step(d["q"], d["k"], d["v"], d["g"], state_cache=d["cache"], scale=case.scale)
    torch.cuda.synchronize()
    _check_step(case, d, out)


def test_step_equals_prompt_of_one_token():
    """Both forms of one token agree to the prompt form's roundings."""
    case = Case([1] * 5, H=2, seed=52, flags="all")
    d, e = case.device(), case.device()
    a = _step(case, d)
    b, _ = case.forward(e)
    torch.cuda.synchronize()
    _check_step(case, d, a)
    check(case, b, e, None)


# ------------------------------------------------------------------------------ capture
def _capture(fn):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            r = fn()
    torch.cuda.current_stream().wait_stream(side)
    return g, r


def test_captured_prompts_replay_with_other_bounds():
    """The kernels read the bounds, so one captured call serves other bounds of as many sequences."""
    cases = [Case(lens, H=2, seed=60 + i, slots=8, extra_rows=300 - sum(lens))
             for i, lens in enumerate(([200, 0, 64], [3, 3, 290], [0, 300, 0], [100, 100, 100]))]
    d = cases[0].device()
    cases[0].forward(d, seg_len=64)  # eager first: code objects are loaded
    torch.cuda.synchronize()
    out = torch.empty_like(d["v"])
    g, _ = _capture(lambda: cases[0].forward(d, out=out, seg_len=64))
    for case in cases + cases[:1]:
        e = case.device()
        for n in ("q", "k", "v", "g", "cu", "store", "indices", "flags"):
            d[n].copy_(e[n])
        out.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        ref, _ = case.forward(e, out=torch.full_like(out, 7.0), seg_len=64)
        torch.cuda.synchronize()
        assert same_bits(out, ref) and same_bits(d["store"], e["store"])
        check(case, out, d, None)


def test_captured_steps_replay():
    case = Case([1] * 6, H=2, seed=70, flags="all")
    d, e = case.device(), case.device()
    inv, _ = kda.rotary_frequencies(128, device="cuda")
    pos = torch.arange(6, device="cuda")
    rot = dict(positions=pos, inv_freq=inv)
    _step(case, case.device(), **rot)
    torch.cuda.synchronize()
    out = torch.empty_like(d["v"])

    def one():
        _step(case, d, out=out, **rot)
        pos.add_(1)

    g, _ = _capture(one)
    at = torch.arange(6, device="cuda")
    pos.copy_(at)
    for r in range(4):
        g.replay()
        torch.cuda.synchronize()
        ref = _step(case, e, positions=at + r, inv_freq=inv)
        torch.cuda.synchronize()
        assert same_bits(out, ref) and same_bits(d["store"], e["store"]), f"replay {r}"


def test_two_captured_calls_share_a_workspace():
    """Graphs on one stream that use the same workspace in turn."""
    a, b = Case([200, 100], H=2, seed=80), Case([30, 270], H=2, seed=81)
    da, db = a.device(), b.device()
    ws = torch.empty(16 << 20, dtype=torch.uint8, device="cuda")
    stores = {n: x["store"].clone() for n, x in (("a", da), ("b", db))}
    a.forward(a.device(), seg_len=64), b.forward(b.device(), seg_len=64)
    torch.cuda.synchronize()
    ga, (oa, _) = _capture(lambda: a.forward(da, seg_len=64, workspace=ws))
    gb, (ob, _) = _capture(lambda: b.forward(db, seg_len=64, workspace=ws))
    for _ in range(3):
        da["store"].copy_(stores["a"]), db["store"].copy_(stores["b"])
        ga.replay(), gb.replay()
        torch.cuda.synchronize()
        check(a, oa, da, None)
        check(b, ob, db, None)


# ------------------------------------------------------------------------------ at the edges of the call
def test_offsets_past_32_bits():
    """Slots and rows whose element offsets pass 2^31: a pool with wide padding, rows far apart."""
    H, n = 2, 300
    case = Case([n - 80, 80], H=H, seed=90, flags="all", slots=4, state_dtype="bf16")
    case.indices = torch.tensor([3, 2], dtype=torch.int32)
    d = case.device()
    wide = 1 << 30  # elements between slots
    big = torch.empty(3 * wide + H * 128 * 128, dtype=torch.bfloat16, device="cuda")
    cache = big.as_strided((4, H, 128, 128), (wide, 128 * 128, 128, 1))
    cache.copy_(d["cache"])
    rows = torch.empty(n << 23, dtype=torch.bfloat16, device="cuda")  # 5 GB, 2^23 elements between tokens
    apart = rows.as_strided((n, H, 128), (1 << 23, 128, 1))
    apart.copy_(d["q"])
    d["cache"], d["q"] = cache, apart
    out, _ = case.forward(d, seg_len=64)
    torch.cuda.synchronize()
    d["store"].copy_(cache.reshape(4, -1))
    check(case, out, d, None)
    step = kda.linear_step(apart[:2], d["k"][:2], d["v"][:2], d["g"][:2], state_cache=cache, state_indices=d["indices"])
    ref = kda.linear_step(apart[:2].contiguous(), d["k"][:2], d["v"][:2], d["g"][:2], state_cache=case.planes(d["store"]),
                          state_indices=d["indices"])
    torch.cuda.synchronize()
    assert same_bits(step, ref) and same_bits(cache.reshape(4, -1), d["store"])


@pytest.mark.parametrize("bounds", [[0, 50, 20, 200], [0, -7, 90, 2 ** 31 - 1], [60, 60, 60, 60], [0, 0, -2 ** 31, 130]])
def test_bounds_that_break_the_rules_stay_inside(bounds):
    """Without host bounds nothing can refuse them; every access stays inside the rows and the slots."""
    case = Case([60, 40, 30], H=2, seed=91, flags="all", pad=64)
    d = case.device()
    d["cu"] = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    before = d["store"].clone()
    guard = torch.full((case.T + 128, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    case.forward(d, out=guard[64:-64], seg_len=64)
    torch.cuda.synchronize()
    assert torch.all(guard[:64] == 7.0) and torch.all(guard[-64:] == 7.0)
    used = set(case.indices.tolist())
    for s in range(case.slots):
        if s not in used:
            assert same_bits(d["store"][s], before[s])
        assert same_bits(d["store"][s, 2 * 128 * 128:], before[s, 2 * 128 * 128:])


def test_non_finite_rows_stay_in_their_head_and_sequence():
    case = Case([100, 70, 1], H=3, seed=92, state="dense")
    d = case.device()
    clean, final = case.forward(d, seg_len=64)
    d["v"][30, 1] = float("nan")
    d["k"][120, 2] = float("inf")
    d["g"][170, 0] = float("nan")
    out, bad = case.forward(d, seg_len=64)
    torch.cuda.synchronize()
    keep = torch.ones(171, 3, dtype=torch.bool, device="cuda")
    keep[:100, 1] = False
    keep[100:170, 2] = False
    keep[170, 0] = False
    assert same_bits(out[keep], clean[keep])
    ok = torch.ones(3, 3, dtype=torch.bool, device="cuda")
    ok[0, 1] = ok[1, 2] = ok[2, 0] = False
    assert same_bits(bad[ok], final[ok])
    assert torch.isnan(out[31:100, 1].float()).all() and torch.isnan(out[170, 0].float()).all()


def test_large_keys_do_not_reach_earlier_rows():
    """q . k of later tokens may overflow fp32: those pairs are left out, not multiplied by 0."""
    case = Case([60], H=1, seed=94, state="none")
    d = case.device()
    clean, _ = case.forward(d)
    d["k"][40:] = 3e38
    d["q"] = d["q"] * 1e3
    out, _ = case.forward(d)
    torch.cuda.synchronize()
    ref, _ = case.forward(dict(d, k=torch.where(torch.arange(60, device="cuda")[:, None, None] < 40, d["k"], 0)))
    torch.cuda.synchronize()
    assert torch.isfinite(out[:40]).all() and same_bits(out[:40], ref[:40])


def test_calls_from_two_threads_on_two_streams():
    import threading
    cases = [Case([150, 90], H=2, seed=93 + i) for i in range(2)]
    data = [c.device() for c in cases]
    outs, errors = [None, None], []
    torch.cuda.synchronize()

    def work(i):
        try:
            s = torch.cuda.Stream()
            store = data[i]["store"].clone()
            torch.cuda.synchronize()
            for _ in range(20):
                with torch.cuda.stream(s):
                    data[i]["store"].copy_(store)
                outs[i], _ = cases[i].forward(data[i], stream=s, seg_len=64)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    torch.cuda.synchronize()
    for c, d, o in zip(cases, data, outs):
        check(c, o, d, None)


def test_refused_calls_on_the_device():
    case = Case([20, 30], H=2, seed=95)
    d = case.device()
    with pytest.raises(ValueError):
        case.forward(d, workspace=torch.empty(8, dtype=torch.uint8))  # another device
    with pytest.raises(TypeError):
        case.forward(d, workspace=torch.empty(8, device="cuda"))
    with pytest.raises(kda.KDAError):
        case.forward(d, out=d["v"])
    with pytest.raises(kda.KDAError):
        case.forward(d, cu_seqlens_cpu=torch.tensor([0, 60, 50], dtype=torch.int32))
    with pytest.raises(kda.KDAError):
        case.forward(d, seg_len=100)
    with pytest.raises(ValueError):
        kda.linear_fwd(d["q"], d["k"], d["v"], d["g"], case.cu)  # bounds on the CPU


# ------------------------------------------------------------------------------ larger, random
@pytest.mark.parametrize("seed", range(12))
def test_random_calls(seed):
    r = np.random.default_rng(seed)
    lens = [int(x) for x in r.integers(0, 150, r.integers(1, 9))]
    if seed % 3 == 0:
        lens += [1] * int(r.integers(1, 40))
    H_qk = int(r.integers(1, 4))
    kw = dict(lengths=lens, H_qk=H_qk, H=H_qk * int(r.integers(1, 4)), K=int(r.choice([64, 128])), V=int(r.choice([64, 128])),
              decay=str(r.choice(["token", "head", "resets", "none"])), state=str(r.choice(["paged", "dense", "none"])),
              state_dtype=str(r.choice(["f32", "f16", "bf16"])), k_first=bool(r.integers(2)), fused=bool(r.integers(2)),
              pad=int(r.choice([0, 8, 4096])), extra_rows=int(r.choice([0, 3])), seed=seed)
    seg = int(r.choice([0, 64, 128, 256]))
    _say(f"case random {seed} seg_len={seg} {kw}")
    case = Case(**kw)
    d = case.device()
    out, final = case.forward(d, seg_len=seg)
    torch.cuda.synchronize()
    check(case, out, d, final)
