"""Refusals of process_logits, top_logits and distill that need CUDA tensors to get as far."""

import pytest
import torch

import verify_spec_draft_gb300 as vsd

pytestmark = pytest.mark.gpu


def test_outputs_left_out(spec):
    """An output that the call has to write and the caller's dict lacks."""
    z = torch.randn((6, 1000), generator=torch.Generator().manual_seed(1)).cuda()
    top = vsd.top_logits(z, 20)
    with pytest.raises(ValueError):
        vsd.process_logits(z.view(1, 6, 1000), out=dict())
    with pytest.raises(ValueError):
        vsd.process_logits(z.view(1, 6, 1000), out=dict(logits=None))
    with pytest.raises(ValueError):
        vsd.top_logits(z, 20, out=dict(values=top["values"], ids=top["ids"]))
    loss = dict(loss=torch.empty(6, device="cuda"))
    with pytest.raises(ValueError):
        vsd.distill(z, top["values"], top["ids"], grad=True, out=loss)
    with pytest.raises(ValueError):
        vsd.distill(z, top["values"], top["ids"], grad=True, out=dict(loss, grad=None))
    assert torch.isfinite(vsd.distill(z, top["values"], top["ids"], out=loss)["loss"]).all()
