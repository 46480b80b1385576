"""How far the gated delta rule's prompts may be off, beyond the rounding of their own type.

What goes into the state enters every product in two fp16 terms (e2 = 2^-20 with the sums' own roundings, as in the harness), and so
do D and S on their way into outputs; P is within e_p = 2^-14 of itself. An output's independent roundings are then at most
(4 e2 + 4 e_p) M |q| and the state's own error, whatever the types of the tokens and of the pool.

Relative to all outputs, e_p is spread over the terms of an output and adds in quadrature to its own rounding, which averages
r = 2.1e-4 in fp16 and 1.66e-3 in bf16: sqrt(r^2 + e_p^2) is 1.042 r and 1.0007 r. One term anywhere (2^-11) is 1.28 r and more
than 1.01 r.
"""
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
