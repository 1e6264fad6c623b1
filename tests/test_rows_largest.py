"""distill's gradient at the largest vocabularies: every entry, the unnamed ones above all, whose gradients
are about 1 / V, against the formula in float64."""

import pytest
import torch

import verify_spec_draft_gb300 as vsd

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("R,V", [(2, 1 << 20), (3, (1 << 20) - 1), (5, 700001)])
@pytest.mark.parametrize("with_tail", [True, False])
def test_every_entry(spec, dtype, R, V, with_tail):
    """A probability is off by e = 2^-24 (4 max|z| + 100) and as much for the teacher's values, relative;
    an unnamed entry's gradient w (q_v - p_T q_v / q_T) by 2 e of both parts, a named one's
    w (q_v - p_k) likewise, and by the rounding to its type."""
    K = 128
    g = torch.Generator().manual_seed(V)
    z = (torch.randn((R, V), generator=g) * 2).to(dtype).cuda()
    at = torch.stack([torch.randperm(V - 2, generator=g)[:K] + 1 for _ in range(R)])
    at[0, 0], at[0, 1] = 0, V - 1                    # the ends are named in row 0 only
    ids = at.to(torch.int32).cuda()
    values = torch.randn((R, K), generator=g).cuda()
    tail = torch.full((R,), 6.0, device="cuda") if with_tail else None
    weight = torch.tensor([1.0, 3.0, -0.5, 2.0, 0.25][:R], device="cuda")
    out = vsd.distill(z, values, ids, tail=tail, weight=weight, grad=True)
    assert vsd.device_status(out["ws"]) == 0

    q = torch.softmax(z.double(), 1)
    b = values.double()
    if with_tail:
        b = torch.cat([b, tail.double()[:, None]], 1)
    p = torch.softmax(b, 1)
    named = torch.zeros((R, V), dtype=torch.bool, device="cuda").scatter_(1, ids.long(), True)
    share = q.masked_fill(named, 0.0)
    share /= share.sum(1, keepdim=True)
    minus = (p[:, K:] * share if with_tail else torch.zeros_like(q)).scatter(1, ids.long(), p[:, :K])
    w = weight.double()[:, None]
    e = 2.0 ** -24 * (4 * z.abs().max().item() + 100) + 2.0 ** -24 * (4 * 6 + 100)
    bar = w.abs() * 2 * e * (q + minus) + (2.0 ** -8 if dtype == BF16 else 2.0 ** -23) * (w * (q - minus)).abs() + 1e-37
    got = out["grad"].double()
    assert ((got - w * (q - minus)).abs() <= bar).all()
    # the bar tells the rest's part from nothing, and a gradient from none, at all but a few entries
    if with_tail:
        assert ((w * minus).abs() > 4 * bar).double().mean() > 0.999
    assert ((w * (q - minus)).abs() > 4 * bar).double().mean() > 0.999
