"""markov_grad where rows without a token hold NaN and infinities, at sizes where the second pass over dWt goes
round its ring of stages, changes accumulators, takes several tiles a pair, reads marks of more than 32
steps, and runs through the parts of float32 weights (one GB300).

Such rows count for nothing, so both gradients equal, bit for bit, those of the same inputs with 0 in
these rows: the sums are the same ones in the same order.
"""

import pytest
import torch

import verify_spec_draft_gb300 as vsd

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("B,gamma,V,r,wdtype,odtype", [
    (100, 7, 40000, 64, BF16, BF16),     # 11 steps a tile, two or three tiles a pair
    (100, 7, 40000, 256, BF16, F32),
    (357, 7, 2048, 128, BF16, F32),      # 40 steps
    (100, 7, 40000, 64, F32, F32),       # the same with three products a step
    (357, 7, 2048, 200, F32, BF16),
    (30, 64, 20008, 50, BF16, F32),      # a rank that is staged, 30 steps
    (700, 7, 4104, 32, BF16, BF16),      # rows ordered by sorted blocks, 77 steps
    (2, 7, 40000, 96, BF16, BF16)])      # one step a tile
def test_rows_without_a_token_hold_anything(spec, B, gamma, V, r, wdtype, odtype):
    g = torch.Generator(device="cuda").manual_seed(B * V + r)
    dz = (torch.randn((B, gamma, V), generator=g, device="cuda") * 1e-3).to(BF16)
    U, Wt = ((torch.randn((V, r), generator=g, device="cuda") * 0.02).to(wdtype) for _ in range(2))
    x = torch.randint(0, V, (B, gamma + 1), generator=g, device="cuda", dtype=torch.int32)
    x[torch.rand((B, gamma + 1), generator=g, device="cuda") < 0.3] = -1
    x[0, 0] = x[-1, gamma - 1] = -1           # the first row and the last
    if B * gamma > 300:
        x[100 // gamma:200 // gamma] = -1     # a whole step of rows
    anchor, tokens = x[:, 0].contiguous(), x[:, 1:].contiguous()
    none = x[:, :gamma] < 0
    kw = dict(dtype=odtype)
    zeroed = dz.clone()
    zeroed[none] = 0
    want = vsd.markov_grad(zeroed, anchor, tokens, U, Wt, **kw)
    assert torch.isfinite(want["U"]).all() and torch.isfinite(want["Wt"]).all() and (want["Wt"] != 0).any()
    ws = vsd.workspace(vsd.OP_MARKOV_GRAD, B, gamma, V, r)
    rows = none.nonzero()
    for kind in ("all", "one", "none", "last"):
        d = dz.clone()
        if kind == "all":
            d[none] = float("nan")
            d[none & (torch.rand(none.shape, generator=g, device="cuda") < 0.5)] = float("-inf")
        elif kind == "one":
            b, j = rows[len(rows) // 2].tolist()
            d[b, j, 3 * V // 4] = float("inf")
        elif kind == "last":
            d[-1, gamma - 1, V - 1] = float("nan")
        got = vsd.markov_grad(d, anchor, tokens, U, Wt, ws=ws, **kw)
        assert torch.equal(got["U"], want["U"]) and torch.equal(got["Wt"], want["Wt"]), kind
    assert vsd.device_status(ws) == 0
