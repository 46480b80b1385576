"""CPU tests of the strides that the binding passes for a single token."""
import ctypes

import pytest
import torch

import gated_delta_rule_pack_amd as kda
from gated_delta_rule_pack_amd import _lib

BF = torch.bfloat16


@pytest.mark.parametrize("entry", ["prompt", "step"])
def test_one_token_of_heads_that_lie_far_apart(entry):
    """One token of a buffer with the heads outside the tokens: its head stride is the buffer's length, and its token
    stride, which nothing reads, must not put the call past the limit of token strides."""
    H, S = 32, 5000
    one = torch.empty(H, S, 128, dtype=BF).transpose(0, 1)[:1]
    state = dict(state_cache=torch.zeros(1, H, 128, 128), out=torch.zeros(1, H, 128, dtype=BF), state_indices=torch.zeros(1, dtype=torch.int32))
    if entry == "prompt":
        state.update(cu_seqlens=torch.tensor([0, 1], dtype=torch.int32), has_initial_state=torch.zeros(1, dtype=torch.bool))
    else:
        state.update(N=1)
    lib = _lib.load()
    validate = lib.kda_linear_fwd_validate if entry == "prompt" else lib.kda_linear_step_validate
    dense = torch.zeros(1, H, 128, dtype=BF)
    for name in ("q", "k", "v"):
        t = dict(q=dense.clone(), k=dense.clone(), v=dense.clone())
        t[name] = one
        a = kda.make_linear_args(t["q"], t["k"], t["v"], None, **state)
        assert getattr(a, f"{name}_stride_h") == S * 128
        for n in ("q", "k", "v", "out"):  # far from each other; nothing is read
            setattr(a, n, (1 + "q k v out".split().index(n)) << 42)
        assert validate(ctypes.byref(a)) == _lib.KDA_OK, name
