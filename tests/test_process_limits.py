"""process_logits with temperatures and repetition penalties at the ends of their range."""

import pytest
import torch

import verify_spec_draft_gb300 as vsd

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def run(dtype, temperature, repetition, V=100):
    x = torch.tensor([0.0, 0.0, -torch.inf, -torch.inf, 1.0, 1.0, -1.0, -1.0]).repeat(V // 8 + 1)[:V]
    hist = torch.arange(0, V, 2, dtype=torch.int32)          # every other one is seen
    r = vsd.process_logits(x.to(dtype).view(1, 1, V).cuda(), history=hist[None].cuda(),
                           temperature=torch.tensor([temperature]).cuda(),
                           repetition=torch.tensor([repetition]).cuda())
    return x, hist.long(), r["logits"][0, 0].float().cpu(), vsd.device_status(r["ws"])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [100, 104, 5001])
@pytest.mark.parametrize("temperature,repetition", [
    (2.0 ** -126, 1.0), (1e-30, 1.0), (1e-30, 1e7), (1e-30, 1e-7), (8e37, 1.0), (1e30, 1e-7), (1.0, 1e37), (1.0, 1e-37)])
def test_ends(spec, dtype, V, temperature, repetition):
    """0 stays 0 and -inf stays -inf; the others by the formula in float64, rounded to float32's range:
    three roundings of the factors and the product, and bf16's."""
    x, hist, y, flags = run(dtype, temperature, repetition, V)
    t, rho = float(torch.tensor(temperature)), float(torch.tensor(repetition))
    want = x.double()
    want[hist] = torch.where(want[hist] > 0, want[hist] / rho, want[hist] * rho)
    want = want / t
    assert flags == 0
    big = want.to(F32).to(dtype).double()
    fin = torch.isfinite(big)
    assert torch.equal(y.double()[~fin], big[~fin])
    bar = (4 * 2.0 ** -24 + (2.0 ** -8 if dtype == BF16 else 0.0)) * want[fin].abs()
    assert ((y.double()[fin] - want[fin]).abs() <= bar).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("temperature,repetition", [
    (1e-39, 1.0), (1e-45, 1.0), (3e38, 1.0), (1e-30, 1e30), (1e-30, 1e-30), (1e30, 1e30), (1.0, 1e-39), (1.0, 3e38)])
def test_beyond_the_ends(spec, dtype, temperature, repetition):
    """Where a factor is no normal number the request is reported, not answered in part."""
    _, _, y, flags = run(dtype, temperature, repetition)
    assert flags == vsd.DEV_NONFINITE and torch.isnan(y).all()
