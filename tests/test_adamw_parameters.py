"""AdamW steps over parameters of an autograd graph: gradients that are no longer theirs,
and backward passes through parameters that have changed (one GB300)."""

import pytest
import torch

import verify_spec_draft_gb300 as vsd

pytestmark = pytest.mark.gpu


def table():
    ps = [torch.nn.Parameter(torch.ones(n, device="cuda", dtype=t)) for n, t in ((300, torch.float32), (64, torch.bfloat16))]
    sum((p.float() ** 2).sum() for p in ps).backward()
    return ps, vsd.adamw_table(ps, [p.grad for p in ps], [vsd.adamw_state(p) for p in ps]), \
        torch.zeros(1, dtype=torch.int32, device="cuda")


def test_a_gradient_that_is_not_the_tables(spec):
    ps, t, step = table()
    vsd.adamw(t, step, lr=1e-2)
    for p in ps:                                   # kept and zeroed, and added to by the next pass
        p.grad.zero_()
    sum((p.float() ** 2).sum() for p in ps).backward()
    vsd.adamw(t, step, lr=1e-2)
    ps[0].grad = ps[0].grad.detach()               # another tensor object over the same memory
    vsd.adamw(t, step, lr=1e-2)
    before = [p.detach().clone() for p in ps]
    ps[1].grad = None
    with pytest.raises(ValueError, match="parameter 1"):
        vsd.adamw(t, step, lr=1e-2)
    (ps[1].float() ** 2).sum().backward()          # a new tensor
    with pytest.raises(ValueError, match="parameter 1"):
        vsd.adamw(t, step, lr=1e-2)
    assert all(torch.equal(p.detach(), q) for p, q in zip(ps, before)) and int(step) == 3
    states = t.states
    vsd.adamw(vsd.adamw_table(ps, [p.grad for p in ps], states), step, lr=1e-2)
    assert int(step) == 4


def test_gradients_of_the_callers_own(spec):
    """A table over other tensors than p.grad steps by them, whatever p.grad is."""
    ps, _, step = table()
    grads = [torch.ones_like(p) for p in ps]
    t = vsd.adamw_table(ps, grads, [vsd.adamw_state(p) for p in ps])
    for p in ps:
        p.grad = None
    vsd.adamw(t, step, lr=0.5, weight_decay=0.0)
    # m / (sqrt(v) + eps) is 1 but for eps and some roundings of 2^-24, and the parameter's own half step
    assert all((p.detach().float() - 0.5).abs().max() < 1e-6 + 0.5 * 2.0 ** -8 * (p.dtype == torch.bfloat16) for p in ps)


def test_a_backward_pass_through_what_a_step_has_changed_is_refused(spec):
    ps, t, step = table()
    loss = sum((p.float() * p.float()).sum() for p in ps[:1]) + (ps[1] * ps[1]).float().sum()
    vsd.adamw(t, step, lr=1e-2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    loss = sum((p * p).float().sum() for p in ps)
    loss.backward()                                # of the parameters as they are now
    vsd.adamw(t, step, lr=1e-2)
    assert int(step) == 2
