"""What 8-bit AdamW states come to over many steps, beside 32-bit ones over the same gradients (one GB300).

Rounding at random keeps the mean of what it rounds: m's mean is that of 32-bit states.  It is sqrt(v)
that is rounded, so the mean of v gains the rounding's variance at every step.  A step moves a
code R by d = R (1 - beta2) / 2 * |g^2 / v - 1|, and the variance of rounding R + d between codes s apart is
d (s - d).  What a step adds is forgotten at a rate of 1 - beta2, so v settles above by |g^2 / v - 1| / 2 * s / R
of itself, whatever beta2 is.  The mean of |g^2 - 1| is 0.968 for normal gradients and s / R lies between 1/16 and
1/8, which makes 3 to 6.4 % (of the larger v); 4 standard errors of a mean over 65,536 entries are
0.5 %.
"""

import pytest
import torch

import verify_spec_draft_gb300 as vsd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("beta2,steps", [(0.999, 6000), (0.99, 1500)])
def test_states_settle(spec, beta2, steps):
    n = 65536
    g = torch.Generator(device="cuda").manual_seed(steps)
    grad = torch.empty(n, device="cuda")
    runs = []
    for bits in (8, 32):
        p = torch.zeros(n, device="cuda")
        s = vsd.adamw_state(p, bits)
        runs.append((vsd.adamw_table([p], [grad], [s]), torch.zeros(1, dtype=torch.int32, device="cuda"), s))
    ws = vsd.workspace(vsd.OP_ADAMW, 1, 1, 1)
    for _ in range(steps):
        grad.normal_(generator=g)
        for table, step, _ in runs:
            vsd.adamw(table, step, lr=1e-3, betas=(0.9, beta2), seed=7, ws=ws)
    assert vsd.device_status(ws) == 0
    (_, _, s8), (_, _, s32) = runs
    value = lambda k: (s8[k].double().view(-1, vsd.ADAMW_BLOCK) * s8[k + "_scale"].double()[:, None]).view(-1)
    v8, v32, m8, m32 = value("v") ** 2, s32["v"].double(), value("m"), s32["m"].double()
    assert 1.025 < float(v8.mean() / v32.mean()) < 1.07
    # m8's error has no mean: 4 standard errors of one of a tenth of m32 are 0.16 %
    assert abs(float((m8 * m32).mean() / (m32 * m32).mean()) - 1.0) < 0.005
    assert (v8 > 0).all()
