"""How far the gated delta rule's prompts may be off, beyond the rounding of their own type.

What goes into the state enters every product in two fp16 terms (e2 = 2^-20 with the sums' own roundings, as in the harness), and so
do D and S on their way into outputs; P is within e_p = 2^-14 of itself. An output's independent roundings are then at most
(4 e2 + 4 e_p) M |q| and the state's own error, whatever the types of the tokens and of the pool.

Relative to all outputs, e_p is spread over the terms of an output and adds in quadrature to its own rounding, which averages
r = 2.1e-4 in fp16 and 1.66e-3 in bf16: sqrt(r^2 + e_p^2) is 1.042 r and 1.0007 r. One term anywhere (2^-11) is 1.28 r and more
than 1.01 r.
"""
import random

import numpy as np
import pytest
import torch

from tests.delta_harness import DeltaCase, E2, close, f64, HALF, TINY

pytestmark = pytest.mark.gpu

PATHS = pytest.mark.parametrize("path", ["walk", "scan"])
EP = 2.0 ** -14

CASES = {
    "f16 tokens": dict(dtype="f16"),
    "f16 tokens, unit, no state": dict(dtype="f16", unit=True, state="none"),
    "f16 tokens, bf16 pool": dict(dtype="f16", state_dtype="bf16", flags="all"),
    "bf16 tokens": dict(flags="all"),
    "bf16 tokens, no state": dict(state="none"),
    "bf16 tokens, bf16 pool": dict(state_dtype="bf16", flags="all"),
    "bf16 tokens, f16 pool": dict(state_dtype="f16", flags="all", K=64),
    "no decay": dict(decay="none", flags="all", dtype="f16", V=64),
}


@PATHS
@pytest.mark.parametrize("name", sorted(CASES))
def test_outputs_and_states_are_off_by_their_own_rounding(name, path):
    lens = [400, 130, 64, 37]
    case = DeltaCase(lens, H=3, seed=41, **CASES[name])
    d = case.device()
    out, final = case.forward(d, path=path)
    torch.cuda.synchronize()
    o, S, M = case.oracle()
    u = HALF[case.dtype]
    n = np.array(lens, np.float64)[:, None]
    state_off = 4 * E2 * (1 + np.sqrt(n)) * M
    token_off = np.repeat(state_off + 4 * (E2 + EP) * M, lens, axis=0)[:, :, None]
    rel = close("out", f64(out), o, u * np.abs(o) + (1 + u) * case.scale * case.query_size() * token_off + TINY[case.dtype])

    def own(x, dtype):
        return np.linalg.norm(f64(torch.from_numpy(x).to(dtype)) - x) / np.linalg.norm(x)

    ratio = rel / own(o, case.dtype)
    print(f"  out: {ratio:.4f} of its own rounding", flush=True)
    assert ratio < (1.05 if case.dtype == torch.float16 else 1.005)
    if case.state != "none":
        sdt = d["cache"].dtype if case.state == "paged" else final.dtype
        got = case.finals(d, final)
        rel = close("state", got, S, HALF[sdt] * np.abs(S) + (1 + HALF[sdt]) * state_off[:, :, None, None] + TINY[sdt])
        if sdt != torch.float32:
            ratio = rel / own(S, sdt)
            print(f"  state: {ratio:.4f} of its own rounding", flush=True)
            assert ratio < 1.005


@PATHS
@pytest.mark.parametrize("exponent", [6, 9, 12, 13, 14, 30])
@pytest.mark.parametrize("normalize", [False, True])
def test_zero_keys_among_long_ones(normalize, exponent, path):
    """A token with k = 0 only decays, whatever its step size; the other keys are s times a unit key's length, with step sizes over
    s^2: the same rule, of states over s, exactly. Normalised keys have no length, and their zero rows the largest steps."""
    case = DeltaCase([140, 3, 64], 2, seed=42, unit=not normalize, state="dense")
    gen = torch.Generator().manual_seed(5)
    zero = torch.rand(case.T, generator=gen) < 0.1
    zero[:2] = True  # the first tokens too
    case.k[zero] = 0
    case.beta[zero] = 0.5 if not normalize else 2.0
    d = case.device()
    s = 1.0 if normalize else 2.0 ** exponent
    steps = d["beta"] / s ** 2
    steps[zero.cuda()] = d["beta"][zero.cuda()]
    scaled = dict(d, k=(d["k"].float() * s).bfloat16(), beta=steps, initial=d["initial"] / s)
    out, final = case.forward(scaled, path=path)
    torch.cuda.synchronize()
    o, S, M = case.oracle()
    n = np.array(case.lengths, np.float64)[:, None]
    state_off = 4 * E2 * (1 + np.sqrt(n)) * M
    token_off = np.repeat(state_off + 4 * (E2 + EP) * M, case.lengths, axis=0)[:, :, None]
    close("out", f64(out) * s, o, 2.0 ** -8 * np.abs(o) + 1.01 * case.scale * case.query_size() * token_off)
    close("state", f64(final) * s, S, 2.0 ** -24 * np.abs(S) + 1.01 * state_off[:, :, None, None])


@PATHS
@pytest.mark.parametrize("size", [1.0, 2.0 ** 20, 2.0 ** 60])
@pytest.mark.parametrize("step", [2.0 ** -60, 2.0 ** -110, 2.0 ** -125, 2.0 ** -140])
def test_tiny_steps_beside_a_state(step, size, path):
    """Step sizes that do next to nothing beside a state: in all chunks, and in a last chunk of a single token."""
    for lens in ([200, 30], [65, 129]):
        case = DeltaCase(lens, 2, seed=43, state="dense")
        case.initial = case.initial * size
        some = torch.ones(case.T, dtype=torch.bool)
        if lens[0] == 65:
            some[:] = False
            some[[64, 193]] = True
        case.beta[some] *= step
        d = case.device()
        out, final = case.forward(d, path=path)
        torch.cuda.synchronize()
        o, S, M = case.oracle()
        n = np.array(case.lengths, np.float64)[:, None]
        state_off = 4 * E2 * (1 + np.sqrt(n)) * M
        token_off = np.repeat(state_off + 4 * (E2 + EP) * M, case.lengths, axis=0)[:, :, None]
        close("out", f64(out), o, 2.0 ** -8 * np.abs(o) + 1.01 * case.scale * token_off)
        close("state", f64(final), S, 2.0 ** -24 * np.abs(S) + 1.01 * state_off[:, :, None, None])


# ------------------------------------------------------------------------------ sizes far apart in one sequence
# L_t of a channel: the largest of what its token t is made of, each as far as it has decayed, max(e^{g_t} L_{t-1}, |beta_t v_t| |k_t|),
# from the largest element of its initial state on. The kernels keep every term within EL = 2^-16 of L_t, however large a value stands
# elsewhere in the chunk, so the harness's bounds hold with EL and L_t in place of e2 and M.
EL = 2.0 ** -16


def _check_reach(case, d, out, final, rows=slice(None)):
    o, S, _ = case.oracle()
    length = 1.0
    if not case.normalize:
        length = np.repeat(np.sqrt((f64(case.k) ** 2).sum(-1)), case.H // case.H_qk, axis=1)
    v = np.abs(f64(case.v)) * (np.abs(f64(case.beta)) * length)[:, :, None]
    decay = np.ones((case.T, case.H)) if case.g is None else np.exp(np.broadcast_to(f64(case.g), (case.T, case.H)))
    start = case.start()
    L, end, n = np.zeros_like(o), np.zeros((case.N, case.H, case.V)), np.zeros((case.T, 1, 1))
    for i in range(case.N):
        l = np.zeros((case.H, case.V)) if start is None else np.abs(start[i]).max(-1)
        for t in range(int(case.cu[i]), int(case.cu[i + 1])):
            l = np.maximum(decay[t][:, None] * l, v[t])
            L[t], n[t] = l, t - int(case.cu[i]) + 1
        end[i] = l
    u = HALF[case.dtype]
    room = u * np.abs(o) + (1 + u) * case.scale * case.query_size() * (4 * EL * (1 + np.sqrt(n)) + 4 * EP) * L + TINY[case.dtype]
    got = f64(out)
    close("out", got[rows], o[rows], room[rows])
    if case.state != "none":
        got = case.finals(d, final)
        sdt = d["cache"].dtype if case.state == "paged" else final.dtype
        m = np.array(case.lengths, np.float64)[:, None, None]
        close("state", got, S, HALF[sdt] * np.abs(S) + (1 + HALF[sdt]) * (4 * EL * (1 + np.sqrt(m)) * end)[..., None] + 1e-37)


@PATHS
@pytest.mark.parametrize("dtype,small,large", [("bf16", 0.1, 1e8), ("bf16", 1e-10, 1e10), ("bf16", 1.0, 1e4), ("f16", 1e-3, 6e4), ("f16", 1e-2, 6e4),
                                               ("f16", 1.0, 300.0)])
@pytest.mark.parametrize("where", [(1, None), (40, None), (40, 5), (63, 77), (70, None)])
@pytest.mark.parametrize("state", ["none", "dense"])
def test_a_large_value_behind_small_ones(state, where, dtype, small, large, path):
    """One token, of all channels or of one, far above those before it: they keep their own accuracy, and so does all else."""
    case = DeltaCase([150, 70], 2, seed=44, state=state, dtype=dtype, V=128 if where[1] is None else 64, K=64 if where[0] == 63 else 128)
    case.v = (case.v.float() * small / 4).clamp(-small, small).to(case.dtype)
    if state == "dense":
        case.initial *= small
    at, channel = where
    if channel is None:
        case.v[at] = (large * torch.sign(case.v[at].float())).to(case.dtype)
    else:
        case.v[at, :, channel % case.V] = large
    d = case.device()
    out, final = case.forward(d, path=path)
    torch.cuda.synchronize()
    _check_reach(case, d, out, final)


@PATHS
@pytest.mark.parametrize("size", [2.0 ** 8, 2.0 ** 20, 2.0 ** 60])
@pytest.mark.parametrize("at", [0, 1, 31, 63, 64, 100])
@pytest.mark.parametrize("reset", [-float("inf"), -90.0, -18.0])
def test_a_large_state_that_is_forgotten(reset, at, size, path):
    case = DeltaCase([150, 30, 64], 2, seed=45, state="dense", decay="none")
    case.initial *= size
    case.g = torch.full((case.T, 2), -0.01)
    case.g[[at, 150 + min(at, 29), 180 + min(at, 63)]] = reset
    d = case.device()
    out, final = case.forward(d, path=path)
    torch.cuda.synchronize()
    _check_reach(case, d, out, final)


@PATHS
@pytest.mark.parametrize("step", [2.0 ** -14, 2.0 ** -20, 2.0 ** -27, 2.0 ** -60])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("state", ["none", "dense"])
def test_small_steps_behind_a_reset(state, dtype, step, path):
    """Step sizes near 1, everything forgotten, then small ones alone: nothing larger is left to hide what they teach."""
    case = DeltaCase([150, 60, 64], 2, seed=46, state=state, dtype=dtype)
    for begin, at in ((0, 20), (0, 90), (150, 5), (210, 50)):
        case.g[begin + at] = -float("inf")
    for a, b in ((20, 64), (90, 150), (155, 210), (260, 274)):
        case.beta[a:b] *= step
    d = case.device()
    out, final = case.forward(d, path=path)
    torch.cuda.synchronize()
    _check_reach(case, d, out, final)


@PATHS
@pytest.mark.parametrize("decay", [-0.1, -1.0, -3.0, -8.0])
def test_large_values_that_decay_to_the_size_of_later_ones(decay, path):
    case = DeltaCase([200, 64, 3], 2, seed=47, state="dense", decay="none")
    case.g = torch.full((case.T, 2), decay)
    for t in (3, 70, 128, 210):
        case.v[t] *= 1e7
    d = case.device()
    out, final = case.forward(d, path=path)
    torch.cuda.synchronize()
    _check_reach(case, d, out, final)


@PATHS
def test_masked_tokens_keep_what_is_left(path):
    """Values and step sizes of zero for most of a sequence, while the state decays: what is left keeps its accuracy."""
    case = DeltaCase([200, 100, 40], 2, seed=48, state="dense", decay="none")
    case.g = torch.full((case.T, 2), -0.3)
    case.beta[10:150] = 0
    case.v[205:290] = 0
    case.v[300:] = 0
    d = case.device()
    out, final = case.forward(d, path=path)
    torch.cuda.synchronize()
    _check_reach(case, d, out, final)


@PATHS
@pytest.mark.parametrize("kw", [dict(), dict(decay="resets", flags="all"), dict(K=64, V=64, dtype="f16"), dict(unit=True, H=4, H_qk=2), dict(state="none")], ids=str)
def test_channels_of_all_sizes_and_times(kw, path):
    """Every value with a size of its own, from 2^-30 to 2^30 (2^-10 to 2^10 in fp16), in order and out of it."""
    kw = {**dict(H=2), **kw}
    case = DeltaCase([130, 64, 257, 1, 2], seed=49, **kw)
    gen = torch.Generator().manual_seed(8)
    span = 10 if case.dtype == torch.float16 else 30
    case.v = (case.v.float() * 2.0 ** torch.randint(-span, span + 1, case.v.shape, generator=gen).float()).to(case.dtype)
    d = case.device()
    out, final = case.forward(d, path=path)
    torch.cuda.synchronize()
    _check_reach(case, d, out, final)


@PATHS
@pytest.mark.parametrize("seed", range(24))
def test_random_batches(seed, path):
    """Types, head sizes, decays, sizes of values, steps and states, and lengths of raw keys, drawn by the seed."""
    rng = random.Random(seed)
    dtype, unit = rng.choice(["bf16", "bf16", "f16"]), rng.random() < 0.6
    lens = [rng.choice([1, 2, 40, 64, 65, 100, 150, 200]) for _ in range(rng.choice([1, 2, 3]))]
    case = DeltaCase(lens, H=rng.choice([1, 2, 3]), K=rng.choice([64, 128]), V=rng.choice([64, 128]), dtype=dtype, unit=unit,
                     state=rng.choice(["none", "dense"]), decay=rng.choice(["token", "none", "resets", "head"]), k_first=rng.random() < 0.3, seed=seed)
    gen = torch.Generator().manual_seed(seed)

    def powers(low, high, *shape):
        return 2.0 ** torch.randint(low, high + 1, shape, generator=gen).float()

    if case.g is not None and case.g.dim() == 2:
        # Beyond e^-60 what is left of a state falls below fp32's range, where nothing keeps its accuracy.
        case.g = torch.where(case.g > -20, (case.g * 10 ** rng.uniform(-2, 1)).clamp(min=-20), torch.full_like(case.g, -float("inf")))
    span = rng.choice([0, 3, 10, 30]) if dtype == "bf16" else rng.choice([0, 3, 8])
    shape = rng.choice([(case.T, case.H, case.V), (case.T, case.H, 1), (1, case.H, case.V)])
    case.v = (case.v.float() * powers(-span, span, *shape)).to(case.dtype)
    if case.state == "dense":
        case.initial *= 2.0 ** rng.choice([0, 0, -10, 10] + [-30, 30] * (dtype == "bf16"))
    case.beta = case.beta / powers(0, rng.choice([0, 0, 5, 30]), *case.beta.shape)
    case.beta[torch.rand(case.beta.shape, generator=gen) < rng.choice([0, 0, 0.2])] = 0
    if unit:
        low, high = rng.choice([(0, 0), (-4, 4), (-2, 3)] + [(-20, -18), (5, 9)] * (dtype == "bf16"))
        case.k = (case.k.float() * powers(low, high, case.T, case.H_qk, 1)).to(case.dtype)
        case.beta = case.beta / case.k.float().norm(dim=-1) ** 2
    d = case.device()
    out, final = case.forward(d, path=path)
    torch.cuda.synchronize()
    _check_reach(case, d, out, final)


# ------------------------------------------------------------------------------ rows at the end of bf16's range
LARGEST = torch.finfo(torch.bfloat16).max


@PATHS
@pytest.mark.parametrize("kw", [dict(), dict(K=64, V=64, decay="none", state="none")])
def test_parallel_rows_of_the_largest_elements(kw, path):
    """Normalised q and k in one direction, every element bf16's largest: the products of the rows as they are scaled have to fit fp16."""
    case = DeltaCase([70, 64], H=2, seed=61, **kw)
    signs = torch.randn(case.K, generator=torch.Generator().manual_seed(61)).sign()
    case.q, case.k = ((LARGEST * signs).expand_as(x).to(x.dtype).contiguous() for x in (case.q, case.k))
    d = case.device()
    out, final = case.forward(d, path=path)
    torch.cuda.synchronize()
    _check_reach(case, d, out, final)


@PATHS
@pytest.mark.parametrize("scale", [1.0, 4.0])
def test_raw_queries_of_the_largest_elements(scale, path):
    """Values are as small as bring the outputs back into range."""
    case = DeltaCase([70, 64], H=2, seed=62, unit=True, state="none")
    case.scale = scale
    case.q = (LARGEST * case.q.float().sign()).to(case.dtype)
    case.v = (case.v.float() * 2.0 ** -60).to(case.dtype)
    d = case.device()
    out, final = case.forward(d, path=path)
    torch.cuda.synchronize()
    _check_reach(case, d, out, final)
