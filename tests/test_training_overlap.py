"""Outputs of policy_loss and markov_grad that share memory with an input or one another are refused,
whatever their offset; rows that lie between another tensor's rows do not.  (Without a GPU the addresses are made up:
every call is refused before its first CUDA call.)"""

import pytest
import torch

import verify_spec_draft_gb300 as vsd
from verify_spec_draft_gb300 import build

INVALID = 1
F32, BF16 = torch.float32, torch.bfloat16
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")


@pytest.fixture(scope="module")
def lib():
    if build.needs_build():
        build.build()
    return vsd.load()


@no_gpu
@pytest.mark.parametrize("change", [
    dict(logp=0x700000), dict(logp=0x700000 + 12), dict(logp=0x700000 - 12),
    dict(loss=0x200000), dict(logp=0x300000 + 12), dict(loss=0x400000 - 12), dict(logp=0x500000), dict(loss=0x600000),
    dict(grad=0x100000 + 16), dict(grad=0x100000 + 3 * 208), dict(grad=0x100000 + 3 * 208 + 192),
    dict(grad=0x200000), dict(grad=0x300000 - 3 * 208 - 192), dict(grad=0x500000 - 208), dict(grad=0x600000 - 16), dict(grad=0x700000),
    dict(grad=0x800000 - 2 * 208), dict(loss=0x100000 + 208), dict(logp=0x100000 + 3 * 208 + 196),
    dict(logits=0x900000 + 16, grad=0x900000), dict(logits=0x700000, grad=0),
])
def test_policy_loss(lib, change):
    a = dict(logits=0x100000, tok=0x200000, old=0x300000, adv=0x400000, ref=0x500000, w=0x600000, loss=0x700000,
             logp=0x800000, grad=0x900000)
    a.update(change)
    # 4 rows of 100 bf16 entries, 104 apart
    assert lib.spec_policy_loss(a["logits"], vsd.BF16, 4, 100, 104, a["tok"], a["old"], a["adv"], a["ref"], a["w"], 1.0,
                                0.2, 0.2, 0.1, a["loss"], a["logp"], a["grad"], 0xA00000, 1 << 20, None) == INVALID


@no_gpu
@pytest.mark.parametrize("change", [
    dict(dU=0x700000 + 16), dict(dU=0x700000 - 32), dict(dU=0x200000 + 1584), dict(dW=0x200000 - 3184), dict(dU=0x300000 + 16),
    dict(dW=0x300000 - 16), dict(dU=0x100000 + 7 * 208 + 192), dict(dW=0x100000 - 3184), dict(dU=0x400000), dict(dW=0x500000 - 3184),
])
def test_markov_grad(lib, change):
    a = dict(dU=0x600000, dW=0x700000)
    a.update(change)
    # 2 x 4 rows of 100 bf16 entries, 104 apart; weights of rank 8 in bf16 (1600 bytes), outputs in float32 (3200)
    assert lib.spec_markov_grad(0x100000, vsd.BF16, 2, 4, 100, 104, 0x400000, 0x500000, 0x200000, 0x300000, vsd.BF16, 8,
                                a["dU"], a["dW"], vsd.F32, 0x800000, 1 << 30, None) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,V", [(BF16, 4096), (F32, 1004)])
def test_policy_loss_on_the_gpu(spec, dtype, V):
    R = 6
    g = torch.Generator().manual_seed(V)
    both = torch.full((R, 2 * V), 7.0, dtype=dtype, device="cuda")
    both[:, :V] = torch.randn((R, V), generator=g).to(dtype).cuda()
    z = both[:, :V]
    ids = (torch.randint(0, V, (R,), generator=g, dtype=torch.int32).cuda(), torch.full((R,), -7.0, device="cuda"),
           torch.randn(R, generator=g).cuda())
    good = vsd.policy_loss(z, *ids, grad=True)
    new = lambda: torch.empty(R, device="cuda")
    # the gradient's rows between the logits'
    got = vsd.policy_loss(z, *ids, grad=True, out=dict(loss=new(), logp=new(), grad=both[:, V:]))
    assert all(torch.equal(got[k], good[k]) for k in ("loss", "logp", "grad")) and torch.equal(both[:, V:], good["grad"])
    one, keep = new(), z.clone()
    flat = both.view(-1)
    off = 16 // dtype.itemsize
    shifted = flat[off:off + (R - 1) * 2 * V + V].as_strided((R, V), (2 * V, 1))
    for out in (dict(loss=one, logp=one, grad=good["grad"]), dict(loss=new(), logp=new(), grad=shifted),
                dict(loss=ids[1], logp=new(), grad=good["grad"]), dict(loss=new(), logp=ids[2], grad=good["grad"])):
        with pytest.raises(vsd.SpecError, match="INVALID_ARG"):
            vsd.policy_loss(z, *ids, grad=True, out=out)
    torch.cuda.synchronize()
    assert torch.equal(z, keep)


@pytest.mark.gpu
def test_markov_grad_on_the_gpu(spec):
    V, r = 1000, 16
    buf = torch.randn(5 * V * r, device="cuda")
    part = lambda at: buf[at:at + V * r].view(V, r)
    U, Wt = part(0), part(V * r)
    grad = torch.randn((3, 2, V), device="cuda")
    ids = torch.arange(6, dtype=torch.int32, device="cuda").view(3, 2)
    args = (grad, ids[:, 0].contiguous(), ids, U, Wt)
    good = vsd.markov_grad(*args)
    got = vsd.markov_grad(*args, out=dict(U=part(2 * V * r), Wt=part(3 * V * r)))
    assert torch.equal(got["U"], good["U"]) and torch.equal(got["Wt"], good["Wt"])
    for at in ((2 * V * r - 4, 3 * V * r), (2 * V * r, 3 * V * r - 4), (2 * V * r, 4), (V * r - 4, 3 * V * r)):
        with pytest.raises(vsd.SpecError, match="INVALID_ARG"):
            vsd.markov_grad(*args, out=dict(U=part(at[0]), Wt=part(at[1])))
