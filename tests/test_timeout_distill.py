"""Waits of distill's gradient kernel that run out.

A row's CTAs wait for one another's records.  Two words of the workspace, which are 0 otherwise, have
the first CTA keep back the record of one exchange and shorten the waits, so that those of its group
run out: the call has to end by itself, set SPEC_DEV_TIMEOUT, and leave NaN, not numbers, in what it
could not compute.  Nothing here faults the GPU or waits without a limit.
"""

import pytest
import torch

import verify_spec_draft_gb300 as vsd

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
# the gradient kernel's words stand behind the 32 KiB header: epoch, exits, patience (us), withheld
PATIENCE, WITHHELD = 32768 + 8, 32768 + 12


def poke(ws, at, value):
    ws[at:at + 4] = torch.tensor(list(value.to_bytes(4, "little")), dtype=torch.uint8, device=ws.device)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("R,V,K,dtype", [(40, 60001, 20, F32), (200, 151936, 33, BF16), (3, 20000, 128, BF16),
                                         (700, 40003, 12, BF16)])
@pytest.mark.parametrize("withheld", [1, 2, 5])
def test_record_kept_back(spec, R, V, K, dtype, withheld, in_place):
    g = torch.Generator().manual_seed(R + V)
    z = (torch.randn((8, V), generator=g) * 3).to(dtype).cuda().repeat(R // 8 + 1, 1)[:R].contiguous()
    z[:, :2000] += torch.randint(-3, 4, (R, 2000), generator=g).to(dtype).cuda()
    top = vsd.top_logits(z + torch.randn((R, 1), generator=g).to(dtype).cuda(), K)
    weight = torch.rand(R, generator=g).cuda()
    weight[::7] = 0.0
    weight[0] = 0.5
    args = dict(tail=top["tail"], weight=weight, grad=True)
    good = vsd.distill(z, top["values"], top["ids"], **args)
    keep = z.clone()
    torch.cuda.synchronize()

    ws = vsd.workspace(vsd.OP_DISTILL, R, K, V)
    poke(ws, PATIENCE, 2000)
    poke(ws, WITHHELD, withheld)
    out = {k: torch.full_like(good[k], 7.0) for k in ("loss", "lse", "grad")}
    if in_place:
        out["grad"] = z
    vsd.distill(z, top["values"], top["ids"], ws=ws, out=out, **args)
    flags = vsd.device_status(ws)
    for k in ("loss", "lse", "grad"):
        got, want = out[k], good[k]
        lost = torch.isnan(got)
        assert torch.equal(got[~lost], want[~lost]), k
    rows = torch.isnan(out["grad"]).any(1)
    if flags:                                  # the first group got as far as that exchange
        assert flags & vsd.DEV_TIMEOUT
        assert rows[0] if withheld == 1 else rows.any()
        # another group's rows are whole
        if R >= 40:
            assert not rows[1]
    else:
        assert withheld > 1 and not rows.any()
    if withheld == 1:
        assert flags
    # the context goes on, and so does the workspace once it is zeroed
    ws.zero_()
    again = vsd.distill(keep, top["values"], top["ids"], ws=ws, **args)
    assert vsd.device_status(ws) == 0
    for k in ("loss", "lse", "grad"):
        assert torch.equal(again[k], good[k])
