"""GPU parity of the gated delta rule with the fp64 oracle: prompts and single tokens."""
import numpy as np
import pytest
import torch

import gated_delta_rule_pack_amd as kda
from tests.delta_harness import DeltaCase, check, f64, same_bits

pytestmark = pytest.mark.gpu

PROMPTS = {
    "one token": dict(lengths=[1]),
    "two tokens": dict(lengths=[2]),
    "a chunk": dict(lengths=[64]),
    "a chunk and one": dict(lengths=[65], flags="all"),
    "ragged": dict(lengths=[0, 1, 63, 0, 64, 130, 17, 1, 0], H=3),
    "no state": dict(lengths=[100, 5], state="none"),
    "dense": dict(lengths=[0, 200, 33], state="dense"),
    "dense k first": dict(lengths=[70, 1, 0], state="dense", k_first=True),
    "unit keys": dict(lengths=[190, 3], unit=True, flags="all"),
    "unit keys, no decay": dict(lengths=[300], unit=True, decay="none", flags="all"),
    "no decay": dict(lengths=[400], decay="none", flags="all"),
    "decay of the head": dict(lengths=[150, 40], decay="head"),
    "resets": dict(lengths=[200, 77], decay="resets", flags="all"),
    "bf16 decays and steps": dict(lengths=[90, 70], g_dtype="bf16", beta_dtype="bf16"),
    "steps up to 2": dict(lengths=[250], beta_max=2.0, flags="all"),
    "f16 tokens": dict(lengths=[100, 64, 1], dtype="f16"),
    "f16 tokens, unit": dict(lengths=[100, 64], dtype="f16", unit=True, K=64),
    "f16 pool": dict(lengths=[129, 1, 0], state_dtype="f16", flags="all"),
    "bf16 pool": dict(lengths=[129, 1, 0], state_dtype="bf16", flags="all"),
    "bf16 pool k first": dict(lengths=[65, 20], state_dtype="bf16", k_first=True),
    "f16 pool k first": dict(lengths=[65, 20], state_dtype="f16", k_first=True, K=64),
    "f32 pool k first": dict(lengths=[65, 20], k_first=True, V=64),
    "K 64": dict(lengths=[100, 31], K=64),
    "V 64": dict(lengths=[100, 31], V=64),
    "K 64 V 64": dict(lengths=[100, 31], K=64, V=64, state="dense"),
    "groups": dict(lengths=[80, 66], H=6, H_qk=2),
    "fused rows": dict(lengths=[80, 66], H=4, H_qk=2, fused=True),
    "fused rows f16": dict(lengths=[80, 66], H=4, H_qk=1, fused=True, dtype="f16", V=64),
    "rows behind": dict(lengths=[30, 40], extra_rows=50),
    "padded slots": dict(lengths=[30, 100], pad=64),
    "many": dict(lengths=[3, 70, 0, 9] * 20, H=4),
    "long": dict(lengths=[1500], H=1, flags="all"),
}


@pytest.mark.parametrize("path", ["walk", "scan"])
@pytest.mark.parametrize("name", sorted(PROMPTS))
def test_prompts(name, path):
    case = DeltaCase(**PROMPTS[name], seed=11)
    d = case.device()
    out = torch.full((case.T, case.H, case.V), 7.0, dtype=case.dtype, device="cuda")
    before = d["store"].clone() if "store" in d else None
    _, final = case.forward(d, out=out, path=path)
    check(case, out, d, final)
    rows = int(case.cu[-1])
    assert torch.all(out[rows:] == 7.0)
    if before is not None:  # slots of no sequence, and what lies between slots
        free = sorted(set(range(case.slots)) - set(case.indices.tolist()))
        assert same_bits(d["store"][free], before[free])
        plane = case.H * case.K * case.V
        assert same_bits(d["store"][:, plane:], before[:, plane:])


STEPS = {
    "one": dict(lengths=[1]),
    "some": dict(lengths=[1] * 5, H=3),
    "groups": dict(lengths=[1] * 7, H=4, H_qk=1),
    "unit": dict(lengths=[1] * 3, unit=True),
    "k first": dict(lengths=[1] * 4, k_first=True),
    "k first K 64": dict(lengths=[1] * 4, k_first=True, K=64, state_dtype="f16"),
    "k first V 64": dict(lengths=[1] * 4, k_first=True, V=64, state_dtype="bf16"),
    "K 64": dict(lengths=[1] * 4, K=64),
    "V 64": dict(lengths=[1] * 4, V=64),
    "K 64 V 64": dict(lengths=[1] * 4, K=64, V=64, state_dtype="f16"),
    "f16 tokens": dict(lengths=[1] * 4, dtype="f16"),
    "bf16 pool": dict(lengths=[1] * 9, state_dtype="bf16", beta_dtype="bf16", g_dtype="bf16"),
    "head decay": dict(lengths=[1] * 4, decay="head"),
    "no decay": dict(lengths=[1] * 4, decay="none", beta_max=2.0),
    "resets": dict(lengths=[1] * 40, decay="resets"),
    "fused": dict(lengths=[1] * 6, fused=True, H=4, H_qk=2),
    "padded": dict(lengths=[1] * 6, pad=16),
}


@pytest.mark.parametrize("name", sorted(STEPS))
def test_steps(name):
    case = DeltaCase(**STEPS[name], seed=5)
    d = case.device()
    out = case.step(d)
    check(case, out, d, None, step=True)
