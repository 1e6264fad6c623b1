"""Rows whose finite logits are far from zero: masks of -1e10, -1e30 and the type's lowest value that
leave nothing else in a row or in its rest, masks of another type's lowest value, the same divided
by a temperature, and large values.

Bars.  A weight 2^((z - m) log2e / t) matters down to 2^-40 of the largest.  Its exponent is off by
2^-24 of itself in the scale and as much in the product or the difference, 4 * 2^-24 * 40 with room,
the exponential by 2^-22, and a sum adds at most about 40 roundings on any path, so its relative
error is at most
    EPS = 2^-24 (4 * 40 + 100).
A logarithm of a sum adds the roundings of m / t, of its scale, of the change of base and of the
result, 2^-21 of its size.  None of this grows with the logits' distance from zero.
"""

import numpy as np
import pytest
import torch

import verify_spec_draft_gb300 as vsd
from oracle import teacher as ot

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
EPS = 2.0 ** -24 * (4 * 40 + 100)
LOW = torch.finfo(F32).min
FAR = [-5e7, -1e10, -1e30, -1e38, LOW / 1.3, float(torch.finfo(BF16).min)]


def f64(t):
    return t.double().cpu().numpy()


def far_rows(kind, R, V, far, dtype, t):
    g = torch.Generator().manual_seed(R + V)
    z = torch.full((R, V), far)
    if kind == "rest":                         # a dozen entries are allowed
        for r in range(R):
            at = torch.randperm(V, generator=g)[:12]
            z[r, at] = torch.randn(min(12, V), generator=g) * 3
    elif kind == "levels":                     # two masks over one another, one entry allowed
        z[torch.rand((R, V), generator=g) < 0.5] = far * (1 - 2.0 ** -6)
        z[:, V // 3] = 2.5
    elif kind == "two":                        # the same without one
        z[torch.rand((R, V), generator=g) < 0.5] = far * (1 - 2.0 ** -6)
    elif kind == "high":
        z = -z
    elif kind == "border":                     # units in the last place around |z| log2e / t = 2^26
        m = torch.tensor(-2.0 ** 26 * np.log(2.0) * t, dtype=F32)
        ulp = 2.0 ** (np.floor(np.log2(abs(float(m)))) - 23)
        z = m + ulp * torch.randint(-6, 7, (R, V), generator=g)
    return z.to(dtype).cuda()


def check_log(got, want):
    with np.errstate(over="ignore"):
        want32 = want.astype(np.float32)
    fin = np.isfinite(want32)
    np.testing.assert_array_equal(got[~fin], want32[~fin])
    assert (np.abs(got[fin] - want[fin]) <= EPS + 2.0 ** -21 * np.abs(want[fin])).all(), (got, want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["rest", "whole", "levels", "two", "high"])
@pytest.mark.parametrize("R,V,K", [(3, 9000, 20), (2, 33001, 100), (40, 4100, 20), (2, 50, 64)])
def test_top(spec, dtype, kind, R, V, K):
    for far in FAR:
        for t in (1.0, 0.25, 3.0):
            z = far_rows(kind, R, V, far, dtype, t)
            out = vsd.top_logits(z, K, temperature=t)
            ref = ot.top_logits(f64(z), K, t)
            np.testing.assert_array_equal(out["ids"].cpu().numpy(), ref["ids"])
            np.testing.assert_array_equal(f64(out["values"]), ref["values"])
            for k in ("tail", "lse"):
                check_log(f64(out[k]), ref[k])
            assert vsd.device_status(out["ws"]) == 0


@pytest.mark.parametrize("t", [1.0, 0.3, 7.0])
@pytest.mark.parametrize("V,K", [(9000, 20), (33001, 100)])
def test_top_border(spec, V, K, t):
    z = far_rows("border", 4, V, 0.0, F32, t)
    out = vsd.top_logits(z, K, temperature=t)
    ref = ot.top_logits(f64(z), K, t)
    np.testing.assert_array_equal(out["ids"].cpu().numpy(), ref["ids"])
    for k in ("tail", "lse"):
        check_log(f64(out[k]), ref[k])
