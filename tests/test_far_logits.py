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


# ---------------------------------------------------------------------------------
def check_distill(z, values, ids, tail, t, out, largest=None):
    """A probability is off by E = 2 EPS + the teacher's 2^-24 (4 max|a / t| + 100), relative; a loss, sum
    p (ln p - ln q), by 2 E (1 + sum p |ln p - ln q|), a gradient by 2 E / t of the terms it is made of,
    and by the rounding to its type.  Loss and gradient do not depend on what is added to a row, so
    the row's maximum is taken off first, and q_v / q_T is formed against the rest's own maximum: next to
    1e30 float64 has no room for a ln n.  `largest`: the teacher's |a / t| that
    counts, where only differences do."""
    z, values, ids = f64(z), f64(values), ids.cpu().numpy()
    check_log(f64(out["lse"]), np.array([ot.lse(row / t) for row in z]))
    z = z - z.max(1, keepdims=True)
    with np.errstate(all="ignore"):   # (the oracle's own q_v / q_T, which is not used)
        ref = ot.distill(z, values, ids, None if tail is None else f64(tail), None, t)
    a = np.abs(values[ids >= 0]).max() / t if largest is None else largest
    if tail is not None:
        a = max(a, np.abs(f64(tail)).max())
    e = 2 * EPS + 2.0 ** -24 * (4 * a + 100)
    step = 0.0
    if "grad" in out:
        step = 2.0 ** -8 if out["grad"].dtype == BF16 else 2.0 ** -23
    for r in range(z.shape[0]):
        p, q = ref["p"][r], ref["q"][r]
        lq = z[r] / t - ref["lse"][r]
        rest = np.ones(z.shape[1], bool)
        rest[ids[r][ids[r] >= 0]] = False
        lqt = ot.lse(lq[rest])
        share = np.zeros(z.shape[1])
        if rest.any():
            share[rest] = np.exp((z[r][rest] - z[r][rest].max()) / t)
            share /= share.sum()
        lqb = np.append(np.where(ids[r] >= 0, lq[np.maximum(ids[r], 0)], 0.0), lqt)
        on = p > 0
        size = (p[on] * np.abs(np.log(p[on]) - lqb[on])).sum()
        with np.errstate(over="ignore"):
            want = float(np.float32(ref["loss"][r]))
        got = float(out["loss"][r])
        if np.isinf(want):
            assert got == want, (r, got)
        else:
            assert abs(got - want) <= 2 * e * (1 + size), (r, got, want)
        if "grad" not in out:
            continue
        parts = q + p[-1] * share
        for k, v in enumerate(ids[r]):
            if v >= 0:
                parts[v] += p[k]
        g = ref["grad"][r]
        g[rest] = (q - p[-1] * share)[rest] / t
        bad = np.abs(f64(out["grad"][r]) - g) > 2 * e / t * parts + step * np.abs(g) + 1e-37
        assert not bad.any(), (r, np.nonzero(bad)[0][:5], f64(out["grad"][r])[bad][:5], g[bad][:5])


def named_in(z, kind, K, seed):
    """K ids a row, among them every entry that the mask of `kind` allows."""
    g = torch.Generator().manual_seed(seed)
    R, V = z.shape
    ids = torch.full((R, K), -1, dtype=torch.int32)
    for r in range(R):
        pick = torch.randperm(V, generator=g)
        if kind in ("rest", "levels"):
            allowed = (z[r].float().cpu().abs() < 1e6).nonzero()[:, 0]
            pick = torch.cat([allowed, pick[~torch.isin(pick, allowed)]])
        n = min(K, V)
        ids[r, :n] = pick[:n].to(torch.int32)
    return ids.cuda()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["rest", "whole", "levels", "two", "high"])
@pytest.mark.parametrize("R,V,K", [(3, 9000, 12), (2, 33001, 16), (170, 1100, 20), (2, 50, 12)])
def test_distill(spec, dtype, kind, R, V, K):
    for far in FAR:
        for t in (1.0, 0.25, 3.0):
            z = far_rows(kind, R, V, far, dtype, t)
            ids = named_in(z, kind, K, seed=V)
            values = torch.randn(ids.shape, generator=torch.Generator().manual_seed(K)).cuda()
            for tail in (None, torch.full((R,), -0.5, device="cuda")):
                for grad in (False, True):
                    out = vsd.distill(z, values, ids, tail=tail, temperature=t, grad=grad)
                    check_distill(z, values, ids, tail, t, out)
                    assert vsd.device_status(out["ws"]) == 0


@pytest.mark.parametrize("t", [1.0, 0.3, 7.0])
@pytest.mark.parametrize("V,K", [(9000, 20), (33001, 100)])
def test_distill_border(spec, V, K, t):
    z = far_rows("border", 4, V, 0.0, F32, t)
    ids = named_in(z, "border", K, seed=V)
    values = torch.randn(ids.shape, generator=torch.Generator().manual_seed(K)).cuda()
    for tail in (None, torch.full((4,), 1.5, device="cuda")):
        for grad in (False, True):
            out = vsd.distill(z, values, ids, tail=tail, temperature=t, grad=grad)
            check_distill(z, values, ids, tail, t, out)
            assert vsd.device_status(out["ws"]) == 0


def test_processed_rows_are_learned_from(spec):
    """Rows masked with the type's lowest value, over a temperature by process_logits, whose grammar
    allows fewer tokens than the teacher has entries."""
    V, K = 5003, 16
    x = far_rows("rest", 6, V, LOW, F32, 1.0)
    y = vsd.process_logits(x[None], temperature=torch.tensor([1.3]).cuda())["logits"][0]
    ids = named_in(y, "rest", K, seed=1)
    values = torch.randn(ids.shape, generator=torch.Generator().manual_seed(2)).cuda()
    out = vsd.distill(y, values, ids, grad=True)
    check_distill(y, values, ids, None, 1.0, out)
    assert vsd.device_status(out["ws"]) == 0


# ---------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("R,V,K", [(3, 9000, 12), (170, 1100, 20), (2, 50, 50)])
def test_teacher_far_from_zero(spec, dtype, R, V, K):
    """A teacher without a rest is renormalised, so only the differences of its values count: they
    are exact, and the probabilities off by EPS, whatever is added to them."""
    g = torch.Generator().manual_seed(V)
    z = (torch.randn((R, V), generator=g) * 3).to(dtype).cuda()
    ids = named_in(z, "whole", K, seed=K)
    steps = torch.randint(0, 9, (R, K), generator=g)
    for at, ulp in ((3e5, 0.25), (-1e7, 1.0), (-1e10, 0.0), (-1e30, 0.0), (LOW, 0.0), (3e38, 0.0), (-3e38, 2.0 ** 104)):
        for t in (1.0, 0.3, 3.0):
            values = (at - ulp * steps if at > LOW else torch.full((R, K), at)).float()
            values[:, 0] = at
            values[R - 1, 1:] = -torch.inf                 # one entry has all of it
            ref = torch.where(values > -torch.inf, values - values.max(1, keepdim=True).values, values)
            for grad in (False, True):
                out = vsd.distill(z, values.cuda(), ids, temperature=t, grad=grad)
                check_distill(z, ref.clamp(min=-1e6).cuda(), ids, None, t, out, largest=40.0)
                assert vsd.device_status(out["ws"]) == 0


def test_teacher_far_from_zero_with_a_rest(spec):
    """Whichever of the buckets has the mass, what there is adds up: the gradient's rows sum to 0."""
    g = torch.Generator().manual_seed(3)
    z = (torch.randn((4, 3001), generator=g) * 3).cuda()
    ids = named_in(z, "whole", 12, seed=4)
    for at in (-1e10, -1e30, LOW, 3e38):
        for t in (1.0, 0.3, 3.0):
            values = torch.full((4, 12), at, device="cuda")
            tail = torch.tensor([min(max(at / t, LOW), -LOW), 0.0, LOW, -LOW], device="cuda")
            out = vsd.distill(z, values, ids, tail=tail, temperature=t, grad=True)
            assert vsd.device_status(out["ws"]) == 0
            assert torch.isfinite(out["grad"]).all() and not torch.isnan(out["loss"]).any()
            # 3001 entries of at most 1 / t, each off by 2 EPS of itself
            assert (out["grad"].double().sum(1).abs() <= 4 * EPS / t).all()


def test_own_far_teacher(spec):
    """A masked row and its own top logits, at the type's lowest value over a temperature."""
    x = far_rows("rest", 4, 5003, LOW, F32, 1.0)
    x[1] = LOW
    y = vsd.process_logits(x[None], temperature=torch.tensor([1.3]).cuda())["logits"][0]
    top = vsd.top_logits(y, 16)
    out = vsd.distill(y, top["values"], top["ids"], grad=True)
    ref = (top["values"] - top["values"].max(1, keepdim=True).values).clamp(min=-1e6)
    check_distill(y, ref, top["ids"], None, 1.0, out, largest=40.0)
    assert vsd.device_status(out["ws"]) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("t", [2.0 ** -126, 1e-30, 1e-10, 1e10, 1e30, 3e38])
def test_temperatures(spec, dtype, t):
    """From the smallest normal number to the largest."""
    t = float(np.float32(t))
    g = torch.Generator().manual_seed(6)
    z = (torch.randn((3, 9001), generator=g) * 3).to(dtype).cuda()
    out = vsd.top_logits(z, 20, temperature=t)
    ref = ot.top_logits(f64(z), 20, t)
    np.testing.assert_array_equal(out["ids"].cpu().numpy(), ref["ids"])
    for k in ("tail", "lse"):
        check_log(f64(out[k]), ref[k])
    ids = named_in(z, "whole", 20, seed=7)
    values = torch.randn(ids.shape, generator=g).cuda()
    for grad in (False, True):
        d = vsd.distill(z, values, ids, temperature=t, grad=grad)
        check_distill(z, values - values.max(1, keepdim=True).values, ids, None, t, d, largest=40.0)
        assert vsd.device_status(d["ws"]) == 0
    assert vsd.device_status(out["ws"]) == 0
