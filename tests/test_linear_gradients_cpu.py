"""CPU tests: the linear and rotary calls record no gradient, and refuse inputs that ask for one."""
import pytest
import torch

import gated_delta_rule_pack_amd as kda

BF = torch.bfloat16


def _linear():
    return dict(q=torch.zeros(20, 2, 128, dtype=BF), k=torch.zeros(20, 2, 128, dtype=BF), v=torch.zeros(20, 4, 64, dtype=BF),
                g=torch.zeros(20, 4), cu_seqlens=torch.tensor([0, 7, 20], dtype=torch.int32), out=torch.zeros(20, 4, 64, dtype=BF))


def _rotary():
    return dict(q=torch.zeros(5, 2, 8), k=torch.zeros(5, 2, 8), positions=torch.arange(5), inv_freq=torch.ones(4, dtype=torch.float64),
                out_q=torch.zeros(5, 2, 8), out_k=torch.zeros(5, 2, 8))


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "out", "initial_state", "state_cache"])
def test_linear(name):
    kw = _linear()
    if name == "initial_state":
        kw[name] = torch.zeros(2, 4, 64, 128)
    elif name == "state_cache":
        kw.update(state_cache=torch.zeros(3, 4, 64, 128), state_indices=torch.zeros(2, dtype=torch.int32),
                  has_initial_state=torch.zeros(2, dtype=torch.bool))
    kw[name].requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        kda.make_linear_args(**kw)
    with torch.no_grad():
        assert kda.make_linear_args(**kw).T == 20
    kw[name] = kw[name].detach()
    assert kda.make_linear_args(**kw).T == 20


@pytest.mark.parametrize("name", ["q", "k", "out_q", "out_k"])
def test_rotary(name):
    kw = _rotary()
    kw[name].requires_grad_()
    with pytest.raises(ValueError, match="inverse=True"):
        kda.make_rotary_args(**kw)
    with torch.no_grad():
        assert kda.make_rotary_args(**kw).T == 5


def test_in_an_autograd_function():
    """Its halves run with gradients off, where the calls are made."""
    class Turn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q):
            kw = _rotary()
            kw["q"] = q
            assert kda.make_rotary_args(**kw).inverse == 0
            return q.clone()

        @staticmethod
        def backward(ctx, dq):
            kw = _rotary()
            kw["q"] = dq.contiguous()
            assert kda.make_rotary_args(**kw, inverse=True).inverse == 1
            return dq.clone()

    q = torch.ones(5, 2, 8, requires_grad=True)
    Turn.apply(q).sum().backward()
    assert torch.equal(q.grad, torch.ones(5, 2, 8))
