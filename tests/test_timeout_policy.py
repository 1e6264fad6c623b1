"""Waits of policy_loss that run out.

The CTAs that share a row wait for one another's pairs.  Two words of the workspace, which are 0
otherwise, have the first CTA keep one of its pairs to itself and shorten the waits, so that those of its
cluster run out: the call has to end by itself, set SPEC_DEV_TIMEOUT, and leave NaN, not numbers, in
what it could not compute, that cluster's later rows included.  Nothing here faults the GPU or
waits without a limit.
"""

import pytest
import torch

import verify_spec_draft_gb300 as vsd

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
# behind the header's status, last-CTA counters and barriers: patience (us), withheld
PATIENCE = 4 * (32 + 32 + 64 * 64)
WITHHELD = PATIENCE + 4


def poke(ws, at, value):
    ws[at:at + 4] = torch.tensor(list(value.to_bytes(4, "little")), dtype=torch.uint8, device=ws.device)


def inputs(R, V, dtype):
    g = torch.Generator().manual_seed(R + V)
    z = (torch.randn((8, V), generator=g) * 3).to(dtype).cuda().repeat(R // 8 + 1, 1)[:R].contiguous()
    z[:, :2000] += torch.randint(-3, 4, (R, 2000), generator=g).to(dtype).cuda()
    weight = torch.rand(R, generator=g).cuda()
    weight[3::7] = 0.0
    args = dict(ref_logp=torch.randn(R, generator=g).cuda() - 9, kl=0.05, weight=weight)
    return z, (torch.randint(0, V, (R,), generator=g, dtype=torch.int32).cuda(), torch.full((R,), -9.0).cuda(),
               torch.randn(R, generator=g).cuda()), args


# rows kept in turn by clusters, a row a cluster, rows too long to be kept, and the loss alone
@pytest.mark.parametrize("R,V,dtype,grad,in_place", [
    (700, 60001, BF16, True, False), (700, 60001, BF16, True, True), (1000, 60000, BF16, True, False),
    (400, 60001, F32, True, True), (40, 60001, F32, True, False), (7, 32000, F32, True, True),
    (2, 1 << 20, F32, True, False), (2, (1 << 20) - 3, F32, True, True),
    (40, 60001, F32, False, False), (7, 248320, BF16, False, False)])
@pytest.mark.parametrize("withheld", [1, 2, 3])
def test_pair_kept_back(spec, R, V, dtype, grad, in_place, withheld):
    z, ids, args = inputs(R, V, dtype)
    good = vsd.policy_loss(z, *ids, grad=grad, **args)
    keep = z.clone()
    names = ("loss", "logp") + (("grad",) if grad else ())
    torch.cuda.synchronize()

    ws = vsd.workspace(vsd.OP_POLICY_LOSS, R, 1, V)
    poke(ws, PATIENCE, 2000)
    poke(ws, WITHHELD, withheld)
    out = {k: torch.full_like(good[k], 7.0) for k in names}
    if in_place:
        out["grad"] = z
    vsd.policy_loss(z, *ids, grad=grad, ws=ws, out=out, **args)
    flags = vsd.device_status(ws)
    lost = torch.isnan(out["loss"])
    assert torch.equal(torch.isnan(out["logp"]), lost)
    for k in names:
        assert torch.equal(out[k][~lost], good[k][~lost]), k
    if grad:
        assert torch.isnan(out["grad"][lost]).all()
    assert not lost[args["weight"] == 0].any()
    rows = lost.nonzero().flatten().tolist()
    if flags & vsd.DEV_TIMEOUT:
        # the first cluster's rows from the withheld pair's on; those between are of others, and whole
        assert rows and (rows[0] == 0) == (withheld == 1)
        assert all(b - a > 16 for a, b in zip(rows, rows[1:]))
    else:
        assert withheld > 1 and not rows and flags == 0
    assert flags or withheld > 1
    # the workspace and the context go on
    ws.zero_()
    again = vsd.policy_loss(keep, *ids, grad=grad, ws=ws, **args)
    assert vsd.device_status(ws) == 0
    for k in names:
        assert torch.equal(again[k], good[k])
