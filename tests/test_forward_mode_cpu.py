"""CPU tests: the calls compute no forward-mode gradient, and refuse inputs that carry a tangent, whose results would lose it."""
import pytest
import torch
from torch.autograd import forward_ad

import gated_delta_rule_pack_amd as kda

BF = torch.bfloat16


def _linear():
    return dict(q=torch.zeros(20, 2, 128, dtype=BF), k=torch.zeros(20, 2, 128, dtype=BF), v=torch.zeros(20, 4, 64, dtype=BF),
                g=torch.zeros(20, 4), cu_seqlens=torch.tensor([0, 7, 20], dtype=torch.int32), out=torch.zeros(20, 4, 64, dtype=BF))


def _pool():
    return dict(state_cache=torch.zeros(3, 4, 64, 128), state_indices=torch.zeros(2, dtype=torch.int32),
                has_initial_state=torch.zeros(2, dtype=torch.bool))


def _rows():
    return dict(q=torch.zeros(5, 2, 8), k=torch.zeros(5, 2, 8), positions=torch.arange(5), inv_freq=torch.ones(4, dtype=torch.float64),
                out_q=torch.zeros(5, 2, 8), out_k=torch.zeros(5, 2, 8))


CALLS = {
    "linear": (kda.make_linear_args, _linear, ["q", "k", "v", "g", "out"]),
    "linear, pool": (kda.make_linear_args, lambda: {**_linear(), **_pool()}, ["state_cache"]),
    "linear, dense": (kda.make_linear_args, lambda: {**_linear(), "initial_state": torch.zeros(2, 4, 64, 128)}, ["initial_state"]),
    "delta": (kda.make_gated_delta_args, lambda: {**_linear(), "beta": torch.zeros(20, 4)}, ["q", "k", "v", "g", "beta", "out"]),
    "delta, pool": (kda.make_gated_delta_args, lambda: {**_linear(), **_pool(), "beta": torch.zeros(20, 4)}, ["state_cache"]),
    "rotary": (kda.make_rotary_args, _rows, ["q", "k", "out_q", "out_k"]),
    "norm": (kda.make_qk_norm_args, lambda: {**_rows(), "q_weight": torch.ones(8), "k_weight": torch.ones(8)},
             ["q", "k", "q_weight", "k_weight", "out_q", "out_k"]),
    "norm, back": (kda.make_qk_norm_args, lambda: {**_rows(), "q_weight": None, "k_weight": None, "grad_q": torch.zeros(5, 2, 8),
                                                   "grad_k": torch.zeros(5, 2, 8)}, ["grad_q", "grad_k"]),
}


@pytest.mark.parametrize("call,name", [(c, n) for c in sorted(CALLS) for n in CALLS[c][2]])
def test_tangents_are_refused(call, name):
    make, inputs, _ = CALLS[call]
    kw = inputs()
    with forward_ad.dual_level():
        make(**kw)  # none carries one
        kw[name] = forward_ad.make_dual(kw[name], torch.ones_like(kw[name]))
        with pytest.raises(ValueError, match="tangent"):
            make(**kw)
        with torch.no_grad(), pytest.raises(ValueError, match="tangent"):  # which leaves forward mode in force
            make(**kw)
        make(**{**kw, name: kw[name].detach()})
    make(**inputs())
