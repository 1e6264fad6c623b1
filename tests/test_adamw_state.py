"""What adamw_state makes of a parameter that requires a gradient: plain tensors, no part of a graph."""

import copy

import pytest
import torch

import verify_spec_draft_gb300 as vsd


def params(device):
    p = torch.nn.Parameter(torch.linspace(-1, 1, 300, device=device).to(torch.bfloat16))
    return [p, torch.nn.Parameter(torch.ones(4, 5, device=device)), (p * 2).view(30, 10)]


@pytest.mark.parametrize("bits", [32, 8])
def test_state_of_a_parameter(bits):
    for p in params("cpu"):
        s = vsd.adamw_state(p, bits)
        for k, t in s.items():
            assert t.is_leaf and not t.requires_grad and t.grad_fn is None, k
        t = copy.deepcopy(s)
        assert set(t) == set(s) and all(torch.equal(t[k].float(), s[k].float()) for k in s)
        if p.dtype == torch.bfloat16:
            assert torch.equal(s["master"], p.detach().float()) and s["master"].numpy().shape == p.shape
        given = torch.zeros(p.shape)
        if p.dtype == torch.bfloat16:
            assert vsd.adamw_state(p, bits, master=given)["master"] is given


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_over_parameters(spec, bits):
    """The same step as over plain tensors, by the gradients that a backward pass left."""
    step = lambda: torch.zeros(1, dtype=torch.int32, device="cuda")
    ps = params("cuda")[:2]
    sum((p.float() ** 3).sum() for p in ps).backward()
    plain = [p.detach().clone() for p in ps]
    states, others = ([vsd.adamw_state(p, bits) for p in x] for x in (ps, plain))
    vsd.adamw(vsd.adamw_table(ps, [p.grad for p in ps], states), step(), lr=1e-2)
    vsd.adamw(vsd.adamw_table(plain, [p.grad.clone() for p in ps], others), step(), lr=1e-2)
    for p, q, s, t in zip(ps, plain, states, others):
        assert p.requires_grad and p.is_leaf and torch.equal(p.detach(), q)
        assert all(torch.equal(s[k].float(), t[k].float()) for k in t)
        assert not any(s[k].requires_grad for k in s)
        assert not torch.equal(p.detach(), torch.ones_like(p))
