"""The gated delta rule's calls at the edges of what they allow: values that are not finite, sizes far from one, bad bounds and slots,
many sequences, streams, threads, captured calls, and the operators together as a model uses them."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import gated_delta_rule_pack_amd as kda
from gated_delta_rule_pack_amd import _lib
from oracle import delta_forward, qk_norm
from tests.delta_harness import DeltaCase, E1, check, close, f64, same_bits

pytestmark = pytest.mark.gpu

PATHS = pytest.mark.parametrize("path", ["walk", "scan"])
NAN, INF = float("nan"), float("inf")


def _say(s):
    print(s, flush=True)


# ------------------------------------------------------------------------------ values
BAD = {"k": NAN, "k inf": INF, "q": NAN, "q inf": -INF, "v": NAN, "v inf": INF, "beta": NAN, "beta inf": INF, "g": NAN, "g above 0": 0.5,
       "g inf": INF}


@PATHS
@pytest.mark.parametrize("state", ["dense", "none"])
@pytest.mark.parametrize("name", sorted(BAD))
def test_what_is_not_finite_reaches_no_earlier_token(name, state, path):
    """Sequence 1, head 1, tokens 40, 64 and 100 of 150: in the first chunk's middle, at the second's start, behind it."""
    lens, H = [70, 150, 1], 3
    for at in (0, 40, 64, 100):
        case = DeltaCase(lens, H, seed=21, state=state)
        d = case.device()
        clean, final = case.forward(d, path=path)
        _say(f"{name} at {at}, {state}, {path}")
        t, what = 70 + at, name.split()[0]
        d[what] = d[what].clone()
        if what in "qkv":
            d[what][t, 1, 5] = BAD[name]
        else:
            d[what][t, 1] = BAD[name]
        out, bad = case.forward(d, path=path)
        torch.cuda.synchronize()
        o, S, size = case.oracle()
        others = [0, 2]
        assert same_bits(out[:, others], clean[:, others]) and same_bits(out[:70], clean[:70]) and same_bits(out[220:], clean[220:])
        room = (2.0 ** -8 * np.abs(o) + 1.01 * case.scale * 8 * E1 * (1 + np.sqrt(150)) * size.max())[70:220, 1]
        got, want = f64(out)[70:220, 1], o[70:220, 1]
        hit = np.zeros(got.shape, bool)  # where a value may be lost
        if what == "q":
            hit[at] = True
        elif what == "v":
            hit[at:, 5] = True
        else:
            hit[at:] = True
        close("kept", np.where(hit, 0, got), np.where(hit, 0, want), np.where(hit, 1, room))
        assert not np.isfinite(got[hit]).any()
        if state == "dense":
            assert same_bits(bad[:, others], final[:, others]) and same_bits(bad[[0, 2]], final[[0, 2]])
            fin = np.isfinite(f64(bad)[1, 1])
            lost = np.zeros_like(fin) if what == "q" else np.ones_like(fin)
            if what == "v":
                lost[:] = False
                lost[5] = True
            assert np.array_equal(fin, ~lost)


@PATHS
@pytest.mark.parametrize("length", [1, 2, 15, 17, 33, 50, 63, 65, 70, 100, 127])
def test_rows_behind_a_sequence_are_not_read(length, path):
    """Every row behind the sequence's end is not finite: the next sequence's, and rows of the tensors behind the last bound."""
    case = DeltaCase([length, 80], 2, seed=37, state="dense", extra_rows=70)
    d = case.device()
    clean, final = case.forward(d, path=path)
    for x in ("q", "k", "v", "g", "beta"):
        d[x] = d[x].clone()
        d[x][length:] = NAN
    out, bad = case.forward(d, path=path)
    torch.cuda.synchronize()
    assert same_bits(out[:length], clean[:length]) and same_bits(bad[0], final[0])
    d = case.device()
    for x in ("q", "k", "v", "g", "beta"):
        d[x][length + 80:] = INF
    out, bad = case.forward(d, path=path)
    torch.cuda.synchronize()
    assert same_bits(out[:length + 80], clean[:length + 80]) and same_bits(bad, final)


@PATHS
def test_state_rows_that_are_not_finite_lose_their_channel(path):
    case = DeltaCase([130, 5], 2, seed=22, state="dense")
    d = case.device()
    clean, final = case.forward(d, path=path)
    d["initial"] = d["initial"].clone()
    d["initial"][0, 1, 7, 3] = NAN
    d["initial"][0, 1, 90, 3] = INF
    out, bad = case.forward(d, path=path)
    torch.cuda.synchronize()
    assert same_bits(out[:, 0], clean[:, 0]) and same_bits(out[130:], clean[130:]) and same_bits(bad[1], final[1])
    lost = [7, 90]
    rest = [c for c in range(128) if c not in lost]
    assert not torch.isfinite(out[:130, 1][:, lost]).any() and same_bits(out[:130, 1][:, rest], clean[:130, 1][:, rest])
    assert not torch.isfinite(bad[0, 1, lost]).any() and same_bits(bad[0, 1, rest], final[0, 1, rest])


@PATHS
@pytest.mark.parametrize("exponent", [-40, -14, 9, 30])
@pytest.mark.parametrize("K", [64, 128])
def test_raw_keys_far_from_unit_length(exponent, K, path):
    """Keys times s and step sizes over s^2 are the same rule of states over s, exactly."""
    case = DeltaCase([140, 1, 64], 2, seed=23, K=K, unit=True, state="dense")
    d = case.device()
    s = 2.0 ** exponent
    scaled = dict(d, k=(d["k"].float() * s).bfloat16(), beta=d["beta"] / s ** 2, initial=d["initial"] / s)
    out, final = case.forward(scaled, path=path)
    torch.cuda.synchronize()
    _say(f"keys of length 2^{exponent}, K={K}, {path}")
    check(case, (out.double() * s).cpu(), d, final.double() * s)


# Keys of different lengths in one chunk, step sizes b / |k|^2: a column of T holds its token's step size beside the chunk's
# largest, at least 2^-25 of that apart, so that what a key 2^a times as long as the shortest teaches is off by 2^(a - 24) of the
# largest state, or is lost, 2^-a: 2^-12 at worst, where two terms leave 2^-20.
@PATHS
@pytest.mark.parametrize("shortest,longest,worst", [(-2, 3, 8 * 2.0 ** -20), (0, 12, 2.0 ** -12)])
def test_raw_keys_of_different_lengths(shortest, longest, worst, path):
    """(-2, 3): |beta k| is up to 4 where the harness takes 1, and 2^(5 - 24) twice 2^-20: 8 times its bound."""
    lens = [140, 64, 3]
    case = DeltaCase(lens, 2, seed=29, unit=True, state="dense")
    gen = torch.Generator().manual_seed(3)
    size = 2.0 ** torch.randint(shortest, longest + 1, (case.T, case.H, 1), generator=gen).float()
    case.k = (case.k.float() * size).bfloat16()
    case.beta = case.beta / size[..., 0] ** 2
    d = case.device()
    out, final = case.forward(d, path=path)
    torch.cuda.synchronize()
    o, S, M = case.oracle()
    n = np.array(lens, np.float64)[:, None]
    state_off = 4 * worst * (1 + np.sqrt(n)) * M
    token_off = np.repeat(state_off + 4 * E1 * M, lens, axis=0)[:, :, None]
    close("out", f64(out), o, 2.0 ** -8 * np.abs(o) + 1.01 * case.scale * case.query_size() * token_off)
    close("state", f64(final), S, 2.0 ** -24 * np.abs(S) + 1.01 * state_off[:, :, None, None])


@PATHS
def test_raw_keys_too_far_apart_are_not_finite(path):
    """Lengths 2^20 apart with step sizes to match: their chunk and what follows of the head's sequence is not finite, all else as it was."""
    case = DeltaCase([200, 70], 2, seed=30, unit=True, state="dense")
    d = case.device()
    clean, final = case.forward(d, path=path)
    d["k"], d["beta"] = d["k"].clone(), d["beta"].clone()
    d["k"][80, 1] *= 2.0 ** 20
    d["beta"][80, 1] /= 2.0 ** 40
    out, bad = case.forward(d, path=path)
    torch.cuda.synchronize()
    assert same_bits(out[:64], clean[:64]) and same_bits(out[:, 0], clean[:, 0]) and same_bits(out[200:], clean[200:])
    assert not torch.isfinite(out[64:200, 1]).any() and not torch.isfinite(bad[0, 1]).any()
    assert same_bits(bad[0, 0], final[0, 0]) and same_bits(bad[1], final[1])


@PATHS
def test_tiny_steps_keep_their_digits(path):
    """Step sizes of 2^-60: what is learnt is far below the values, and keeps its own relative accuracy."""
    case = DeltaCase([200, 30], 2, seed=24, state="none", beta_max=2.0 ** -60)
    d = case.device()
    out, _ = case.forward(d, path=path)
    torch.cuda.synchronize()
    o, _, _ = case.oracle()
    # Bounds as the harness has them, with M the largest of what a step teaches: beta v.
    n = np.repeat([200, 30], [200, 30])[:, None, None]
    size = 2.0 ** -60 * abs(f64(case.v)).max()
    close("out", f64(out), o, 2.0 ** -8 * np.abs(o) + 1.01 * case.scale * 4 * E1 * (2 + np.sqrt(n)) * np.sqrt(n) * size)


@PATHS
def test_zero_rows_and_zero_steps(path):
    case = DeltaCase([150, 1, 1, 64], 2, seed=25, state="dense")
    case.k[3] = 0
    case.k[64:70] = 0
    case.q[10] = 0
    case.q[150] = 0
    case.k[151] = 0
    case.v[20:30] = 0
    case.beta[40:50] = 0
    case.beta[152:] = 0
    d = case.device()
    out, final = case.forward(d, path=path)
    torch.cuda.synchronize()
    check(case, out, d, final)
    assert torch.all(out[10] == 0) and torch.all(out[150] == 0)


@PATHS
@pytest.mark.parametrize("value", [-INF, float(torch.finfo(torch.float32).min), -119.0, 0.0])
def test_every_decay_the_same(value, path):
    case = DeltaCase([100, 64, 1], 2, seed=26, flags="all")
    case.g[:] = value
    d = case.device()
    out, _ = case.forward(d, path=path)
    torch.cuda.synchronize()
    check(case, out, d, None)


@PATHS
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_values_and_states_of_any_size(dtype, path):
    """Channels of v and of the state whose sizes differ by 2^40 (2^20 in fp16 tokens): each keeps its own accuracy."""
    case = DeltaCase([130, 3], 2, seed=27, state="dense", dtype=dtype)
    span = 20 if dtype == "bf16" else 6
    size = 2.0 ** torch.randint(-span, span + 1, (128,), generator=torch.Generator().manual_seed(1)).float()
    d = case.device()
    base, final = case.forward(d, path=path)
    grown = dict(d, v=(d["v"].float() * size.cuda()).to(case.dtype), initial=d["initial"] * size.cuda()[:, None])
    out, bad = case.forward(grown, path=path)
    torch.cuda.synchronize()
    check(case, base, d, final)
    check(case, (out.double() / size.cuda()).cpu(), d, bad.double() / size.cuda()[:, None])


# ------------------------------------------------------------------------------ calls
@pytest.mark.parametrize("N,H,long", [(512, 1, 90), (513, 1, 90), (300, 3, 130), (90, 4, 200)])
def test_many_sequences_of_all_lengths(N, H, long):
    """More workgroups than run at once, taken longest first while a workgroup can rank them."""
    r = np.random.default_rng(N)
    lens = np.where(r.random(N) < 0.6, r.integers(0, 3, N), np.exp(r.random(N) * np.log(long)).astype(int)).tolist()
    case = DeltaCase(lens, H, seed=28, K=64, V=64)
    stores = []
    for path in ("walk", "scan"):
        d = case.device()
        out, _ = case.forward(d, path=path, cu_seqlens_cpu=case.cu)
        torch.cuda.synchronize()
        _say(f"{N} sequences, {path}")
        check(case, out, d, None)
        stores.append(d["store"])


@PATHS
def test_calls_repeat_bit_for_bit(path):
    case = DeltaCase([300, 20, 1, 500], 3, seed=6)
    d = case.device()
    store = d["store"].clone()
    first = case.forward(d, path=path)[0].clone()
    after = d["store"].clone()
    for _ in range(3):
        d["store"].copy_(store)
        again, _ = case.forward(d, path=path)
        assert same_bits(again, first) and same_bits(d["store"], after)


@PATHS
def test_a_sequence_does_not_depend_on_its_batch(path):
    case = DeltaCase([77, 130, 1, 64], 2, seed=31, state="dense")
    d = case.device()
    out, final = case.forward(d, path=path)
    for n in range(4):
        a, b = int(case.cu[n]), int(case.cu[n + 1])
        one = {x: d[x][a:b].contiguous() for x in ("q", "k", "v", "g", "beta")}
        one.update(cu=torch.tensor([0, b - a], dtype=torch.int32, device="cuda"), initial=d["initial"][n:n + 1])
        o, f = case.forward(one, path=path)
        assert same_bits(o, out[a:b]) and same_bits(f[0], final[n])


@PATHS
@pytest.mark.parametrize("k_first", [False, True])
def test_dense_state_in_place(path, k_first):
    """initial_state and final_state may be the same memory."""
    case = DeltaCase([300, 0, 1, 40], H=2, state="dense", seed=7, k_first=k_first)
    d = case.device()
    state = d["initial"].clone()
    out = torch.empty_like(d["v"])
    a = kda.make_gated_delta_args(d["q"], d["k"], d["v"], d["g"], d["beta"], cu_seqlens=d["cu"], initial_state=state, final_state=state,
                                  out=out, state_k_first=k_first, normalize=True, path=path)
    lib = _lib.load()
    ws = torch.empty(lib.kda_gated_delta_fwd_workspace_bytes(ctypes.byref(a)) + 1, dtype=torch.uint8, device="cuda")
    rc = lib.kda_gated_delta_fwd(kda.get_context("cuda:0").ptr, ctypes.byref(a), ws.data_ptr(), ws.numel(),
                                 torch.cuda.current_stream().cuda_stream)
    assert rc == _lib.KDA_OK
    torch.cuda.synchronize()
    check(case, out, d, state)


@PATHS
def test_slots_outside_the_pool_are_no_slots(path):
    case = DeltaCase([80, 30, 0, 1, 1], H=2, seed=8, flags="all")
    case.indices[1], case.indices[2], case.indices[4] = -1, case.slots, 1 << 30
    d = case.device()
    before = d["store"].clone()
    out, _ = case.forward(d, path=path)
    torch.cuda.synchronize()
    check(case, out, d, None)
    used = {int(case.indices[0]), int(case.indices[3])}
    for s in range(case.slots):
        if s not in used:
            assert same_bits(d["store"][s], before[s])


@PATHS
def test_strided_output_and_padded_heads(path):
    case = DeltaCase([70, 1, 20], H=3, seed=9, V=64)
    d = case.device()
    wide = torch.full((case.T, 4, 80), 7.0, dtype=torch.bfloat16, device="cuda")
    out, _ = case.forward(d, out=wide[:, :3, :64], path=path)
    torch.cuda.synchronize()
    check(case, out, d, None)
    assert torch.all(wide[:, 3] == 7.0) and torch.all(wide[:, :, 64:] == 7.0)


@PATHS
def test_another_stream_and_given_workspace(path):
    case = DeltaCase([200, 90], H=2, seed=10)
    d = case.device()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, _ = case.forward(d, stream=side, path=path, workspace=torch.empty(64 << 20, dtype=torch.uint8, device="cuda"))
    side.synchronize()
    check(case, out, d, None)


@PATHS
def test_broadcast_rows(path):
    case = DeltaCase([100, 1], H=3, H_qk=1, seed=11)
    d = case.device()
    shared = dict(d, q=d["q"].expand(-1, 3, -1), k=d["k"].expand(-1, 3, -1))
    out, _ = case.forward(shared, path=path)
    torch.cuda.synchronize()
    check(case, out, d, None)


@PATHS
@pytest.mark.parametrize("bounds", [[0, 50, 20, 200], [0, -7, 90, 2 ** 31 - 1], [60, 60, 60, 60], [0, 0, -2 ** 31, 130], [130, 0, 130, 0]])
def test_bounds_that_break_the_rules_stay_inside(bounds, path):
    """Without host bounds nothing can refuse them; every access stays inside the rows and the slots."""
    case = DeltaCase([60, 40, 30], H=2, seed=91, flags="all", pad=64)
    d = case.device()
    d["cu"] = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    before = d["store"].clone()
    guard = torch.full((case.T + 128, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    _say(f"bounds {bounds} {path}")
    case.forward(d, out=guard[64:-64], path=path)
    torch.cuda.synchronize()
    assert torch.all(guard[:64] == 7.0) and torch.all(guard[-64:] == 7.0)
    used = set(case.indices.tolist())
    for s in range(case.slots):
        if s not in used:
            assert same_bits(d["store"][s], before[s])
        assert same_bits(d["store"][s, 2 * 128 * 128:], before[s, 2 * 128 * 128:])


@PATHS
def test_offsets_past_32_bits(path):
    """Slots and rows whose element offsets pass 2^31: a pool with wide padding, rows far apart."""
    H, n = 2, 300
    case = DeltaCase([n - 80, 79, 1], H=H, seed=90, flags="all", slots=5, state_dtype="bf16")
    case.indices = torch.tensor([3, 2, 4], dtype=torch.int32)
    d = case.device()
    wide = 1 << 30  # elements between slots
    big = torch.empty(4 * wide + H * 128 * 128, dtype=torch.bfloat16, device="cuda")
    cache = big.as_strided((5, H, 128, 128), (wide, 128 * 128, 128, 1))
    cache.copy_(d["cache"])
    rows = torch.empty(n << 23, dtype=torch.bfloat16, device="cuda")  # 5 GB, 2^23 elements between tokens
    apart = rows.as_strided((n, H, 128), (1 << 23, 128, 1))
    apart.copy_(d["q"])
    v = rows.as_strided((n, H, 128), (1 << 23, 128, 1), 1 << 12)
    v.copy_(d["v"])
    out = torch.empty(n << 23, dtype=torch.bfloat16, device="cuda").as_strided((n, H, 128), (1 << 23, 128, 1))
    d["cache"], d["q"], d["v"] = cache, apart, v
    case.forward(d, path=path, out=out)
    torch.cuda.synchronize()
    d["store"].copy_(cache.reshape(5, -1))
    check(case, out, d, None)
    small = dict(state_indices=d["indices"][:2], normalize=True)
    step = kda.gated_delta_step(apart[-2:], d["k"][:2], v[-2:], d["g"][:2], d["beta"][:2], state_cache=cache, **small)
    ref = kda.gated_delta_step(apart[-2:].contiguous(), d["k"][:2], v[-2:].contiguous(), d["g"][:2], d["beta"][:2],
                               state_cache=case.planes(d["store"]), **small)
    torch.cuda.synchronize()
    assert same_bits(step, ref) and same_bits(cache.reshape(5, -1), d["store"])


@PATHS
def test_calls_from_two_threads_on_two_streams(path):
    cases = [DeltaCase([150, 90], H=2, seed=93 + i) for i in range(2)]
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
                outs[i], _ = cases[i].forward(data[i], stream=s, path=path)
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


@PATHS
def test_captured_prompts_replay_with_other_bounds(path):
    cases = [DeltaCase(lens, H=2, seed=60 + i, slots=8, extra_rows=300 - sum(lens))
             for i, lens in enumerate(([200, 0, 64], [3, 1, 290], [0, 300, 0], [100, 100, 100], [1, 1, 1]))]
    d = cases[0].device()
    cases[0].forward(d, path=path)  # eager first: code objects are loaded
    torch.cuda.synchronize()
    out = torch.empty_like(d["v"])
    g, _ = _capture(lambda: cases[0].forward(d, out=out, path=path))
    for case in cases + cases[:1]:
        e = case.device()
        for n in ("q", "k", "v", "g", "beta", "cu", "store", "indices", "flags"):
            d[n].copy_(e[n])
        out.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        ref, _ = case.forward(e, out=torch.full_like(out, 7.0), path=path)
        torch.cuda.synchronize()
        assert same_bits(out, ref) and same_bits(d["store"], e["store"])
        check(case, out, d, None)


def test_captured_steps_replay():
    case = DeltaCase([1] * 6, H=2, seed=70, flags="all")
    d, e = case.device(), case.device()
    case.step(case.device())
    torch.cuda.synchronize()
    out = torch.empty_like(d["v"])
    g, _ = _capture(lambda: case.step(d, out=out))
    for r in range(4):
        g.replay()
        torch.cuda.synchronize()
        ref = case.step(e)
        torch.cuda.synchronize()
        assert same_bits(out, ref) and same_bits(d["store"], e["store"]), f"replay {r}"


def test_two_captured_calls_share_a_workspace():
    a, b = DeltaCase([200, 100], H=2, seed=80), DeltaCase([30, 270], H=2, seed=81)
    da, db = a.device(), b.device()
    ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    stores = {n: x["store"].clone() for n, x in (("a", da), ("b", db))}
    a.forward(a.device(), path="scan"), b.forward(b.device(), path="scan")
    torch.cuda.synchronize()
    ga, (oa, _) = _capture(lambda: a.forward(da, path="scan", workspace=ws))
    gb, (ob, _) = _capture(lambda: b.forward(db, path="scan", workspace=ws))
    for _ in range(3):
        da["store"].copy_(stores["a"]), db["store"].copy_(stores["b"])
        ga.replay(), gb.replay()
        torch.cuda.synchronize()
        check(a, oa, da, None)
        check(b, ob, db, None)


# ------------------------------------------------------------------------------ single tokens
def test_step_padding_rows_are_left_alone():
    case = DeltaCase([1] * 6, H=2, seed=50, flags="all")
    keep = [0, 2, 5]
    for n in (1, 3, 4):
        case.indices[n] = {1: -1, 3: case.slots, 4: -(1 << 30)}[n]
    d = case.device()
    before = d["store"].clone()
    out = torch.full_like(d["v"], 7.0)
    case.step(d, out=out)
    torch.cuda.synchronize()
    o, S, size = case.oracle()
    close("out", f64(out)[keep], o[keep], 2.0 ** -8 * np.abs(o[keep]) + 1.01 * case.scale * 2.0 ** -15 * size[keep][:, :, None])
    assert torch.all(out[[1, 3, 4]] == 7.0)
    used = {int(case.indices[n]) for n in keep}
    for s in range(case.slots):
        if s not in used:
            assert same_bits(d["store"][s], before[s])


def test_step_without_indices_takes_slot_n():
    case = DeltaCase([1] * 4, H=2, seed=51, flags="all", slots=6)
    case.indices = torch.arange(4, dtype=torch.int32)
    d = case.device()
    out = case.step(d, state_indices=None, has_initial_state=None)
    torch.cuda.synchronize()
    check(case, out, d, None, step=True)


@PATHS
@pytest.mark.parametrize("kw", [dict(), dict(k_first=True), dict(state_dtype="bf16"), dict(state_dtype="f16", k_first=True, V=64),
                                dict(K=64, dtype="f16")], ids=str)
def test_step_equals_prompt_of_one_token(kw, path):
    case = DeltaCase([1] * 5, H=2, seed=52, **kw)
    d, e = case.device(), case.device()
    a = case.step(d)
    b, _ = case.forward(e, path=path)
    torch.cuda.synchronize()
    check(case, a, d, None, step=True)
    check(case, b, e, None, step=True)


def test_what_is_not_finite_in_a_step():
    case = DeltaCase([1] * 6, H=2, seed=53, flags="all")
    d, e = case.device(), case.device()
    clean = case.step(e)
    d["q"][0, 0, 3], d["k"][1, 0, 3], d["v"][2, 0, 3] = NAN, INF, NAN
    d["g"][3, 0], d["beta"][4, 0] = 1e-3, NAN
    out = case.step(d)
    torch.cuda.synchronize()
    assert same_bits(out[:, 1], clean[:, 1]) and same_bits(out[5], clean[5])
    for n in (0, 1, 3, 4):
        assert not torch.isfinite(out[n, 0]).any()
    rest = [c for c in range(128) if c != 3]
    assert not torch.isfinite(out[2, 0, 3]) and same_bits(out[2, 0, rest], clean[2, 0, rest])
    got, ref = d["cache"][d["indices"].long()], e["cache"][e["indices"].long()]
    assert same_bits(got[:, 1], ref[:, 1]) and same_bits(got[0, 0], ref[0, 0]) and same_bits(got[2, 0, rest], ref[2, 0, rest])
    assert not torch.isfinite(got[[1, 3, 4], 0]).any() and not torch.isfinite(got[2, 0, 3]).any()


# ------------------------------------------------------------------------------ together
@PATHS
def test_norm_then_prompt_then_single_tokens(path):
    """As a model serves: q and k normed and turned, prompts fill the pool, then requests go on token by token; one
    sequence has no prompt."""
    steps, H, H_qk, K = 5, 4, 2, 128
    lens = [70, 0, 33, 1]
    whole = DeltaCase([n + steps for n in lens], H=H, H_qk=H_qk, seed=13, state="none")
    inv, _ = kda.rotary_frequencies(K, device="cuda")
    qw, kw = (1 + 0.1 * torch.randn(K, generator=torch.Generator().manual_seed(s)).bfloat16() for s in (1, 2))
    cache = torch.full((6, H, 128, K), NAN, device="cuda")
    idx = torch.tensor([4, 1, 3, 0], dtype=torch.int32, device="cuda")
    d = whole.device()
    begin = whole.cu[:-1].tolist()
    rows = torch.cat([torch.arange(b, b + n) for b, n in zip(begin, lens)]).cuda()
    pos = torch.cat([torch.arange(n) for n in lens]).cuda()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    weights = dict(q_weight=qw.cuda(), k_weight=kw.cuda())
    got = torch.full(whole.v.shape, NAN)
    taken = [torch.empty(x.shape, dtype=torch.bfloat16) for x in (whole.q, whole.k)]

    def normed(at, where):
        q, k = kda.qk_norm(d["q"][at], d["k"][at], **weights, positions=where, inv_freq=inv)
        taken[0][at.cpu()], taken[1][at.cpu()] = q.cpu(), k.cpu()
        return q, k

    q, k = normed(rows, pos)
    out, _ = kda.gated_delta_fwd(q, k, d["v"][rows], d["g"][rows], d["beta"][rows], cu, normalize=True, state_cache=cache, state_indices=idx,
                                 has_initial_state=torch.zeros(4, dtype=torch.bool, device="cuda"), path=path)
    got[rows.cpu()] = out.float().cpu()
    for s in range(steps):
        row = torch.tensor([b + n + s for b, n in zip(begin, lens)], device="cuda")
        q, k = normed(row, torch.tensor([n + s for n in lens], device="cuda"))
        out = kda.gated_delta_step(q, k, d["v"][row], d["g"][row], d["beta"][row], state_cache=cache, state_indices=idx, normalize=True)
        got[row.cpu()] = out.float().cpu()
    at = np.concatenate([np.arange(n + steps) for n in lens])
    for x, w, t in ((whole.q, qw, taken[0]), (whole.k, kw, taken[1])):
        want = qk_norm(f64(x), f64(w), at, inv.cpu().numpy())
        close("normed", f64(t), want, 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * np.abs(want).max(-1, keepdims=True))
    # The rule on what the norm stored.
    o, S, size = delta_forward(f64(taken[0]), f64(taken[1]), f64(whole.v), f64(whole.g), f64(whole.beta), whole.cu.tolist(), scale=K ** -0.5,
                               normalize=True)
    n = np.array([n + steps for n in lens], np.float64)[:, None]
    state_off = 4 * 2.0 ** -20 * (1 + np.sqrt(n)) * size
    token_off = np.repeat(state_off + 4 * E1 * size, [n + steps for n in lens], axis=0)
    close("out", got.double().numpy(), o, 2.0 ** -8 * np.abs(o) + 1.01 * K ** -0.5 * token_off[:, :, None])
    close("state", f64(cache[idx.long()]), S, 2.0 ** -24 * np.abs(S) + 1.01 * state_off[:, :, None, None])


def test_paths_agree():
    case = DeltaCase([1000, 1, 333, 64, 0, 2], H=4, H_qk=2, seed=95)
    d, e = case.device(), case.device()
    a, _ = case.forward(d, path="walk")
    b, _ = case.forward(e, path="scan", cu_seqlens_cpu=case.cu)
    torch.cuda.synchronize()
    check(case, a, d, None)
    check(case, b, e, None)


def test_refused_calls_on_the_device():
    case = DeltaCase([10], H=2, seed=96)
    d = case.device()
    with pytest.raises(kda.KDAError):
        case.forward(d, cu_seqlens_cpu=torch.tensor([0, 11], dtype=torch.int32))
    with pytest.raises(kda.KDAError):
        case.forward(d, out=d["v"])
    with pytest.raises(ValueError):
        kda.gated_delta_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], None)
    with pytest.raises((ValueError, TypeError)):
        case.forward(d, workspace=torch.empty(4, device="cuda"))
    with pytest.raises(ValueError):
        case.forward(dict(d, beta=d["beta"].cpu()))


def test_a_given_workspace_that_does_not_serve_is_refused():
    case = DeltaCase([200, 90], H=2, seed=97)
    d = case.device()
    before = d["store"].clone()
    out = torch.full_like(d["v"], 7.0)
    big = torch.empty(4 << 20, dtype=torch.uint8, device="cuda")
    for ws in (big[:0], big[:1000], big[128:], big[1:]):
        with pytest.raises(kda.KDAError, match="workspace"):
            case.forward(d, out=out, path="scan", workspace=ws)
    torch.cuda.synchronize()
    assert torch.all(out == 7.0) and same_bits(d["store"], before)
    case.forward(d, out=out, path="scan", workspace=big)
    torch.cuda.synchronize()
    check(case, out, d, None)
    e = case.device()
    case.forward(e, out=out, path="walk", workspace=big[1:3])  # which needs none
    torch.cuda.synchronize()
    check(case, out, e, None)
