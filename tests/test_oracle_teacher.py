"""Pins of oracle.teacher: worked values, limits, finite differences."""

import numpy as np
import pytest

from oracle import teacher as ot


def test_top_worked_example():
    z = np.log([4.0, 1.0, 4.0, 2.0, 0.0 + 1e-300])
    z[4] = -np.inf
    v, i, tail, lse = ot.top_row(z, 2)
    assert i.tolist() == [0, 2]                      # the tie goes to the lowest index
    assert tail == pytest.approx(np.log(3.0)) and lse == pytest.approx(np.log(11.0))
    v, i, tail, _ = ot.top_row(z, 6)
    assert i.tolist() == [0, 2, 3, 1, -1, -1] and (v[4:] == -np.inf).all() and tail == -np.inf
    # at t = 2 the weights are the square roots
    _, _, tail, lse = ot.top_row(z, 2, 2.0)
    assert tail == pytest.approx(np.log(1 + np.sqrt(2))) and lse == pytest.approx(np.log(5 + np.sqrt(2)))


def test_a_tiny_rest_keeps_its_logarithm():
    z = np.array([30.0, 2.0, 1.0])
    _, _, tail, lse = ot.top_row(z, 1)
    assert tail == pytest.approx(np.log(np.exp(2.0) + np.exp(1.0)), rel=1e-14) and lse == pytest.approx(30.0)


def test_invalid_rows():
    for bad in (np.nan, np.inf):
        v, i, tail, lse = ot.top_row(np.array([0.0, bad]), 1)
        assert np.isnan(v).all() and (i == -1).all() and np.isnan(tail) and np.isnan(lse)
    v, i, tail, lse = ot.top_row(np.full(3, -np.inf), 2)
    assert (i == -1).all() and tail == -np.inf and lse == -np.inf


def test_full_kl_and_cross_entropy():
    rng = np.random.default_rng(0)
    z, a = rng.normal(size=9) * 2, rng.normal(size=9) * 2
    perm = rng.permutation(9)
    r = ot.distill_row(z, a[perm], perm, t=1.5)
    p, q = np.exp(a / 1.5), np.exp(z / 1.5)
    p, q = p / p.sum(), q / q.sum()
    assert r["loss"] == pytest.approx((p * np.log(p / q)).sum(), rel=1e-12)
    np.testing.assert_allclose(r["grad"], (q - p) / 1.5, rtol=1e-12)
    r = ot.distill_row(z, np.zeros(1), np.array([4]))
    q = np.exp(z) / np.exp(z).sum()
    assert r["loss"] == pytest.approx(-np.log(q[4]), rel=1e-12)


def test_own_row_is_the_minimum():
    rng = np.random.default_rng(1)
    for t in (0.7, 1.0, 2.0):
        z = rng.normal(size=50) * 3
        v, i, tail, _ = ot.top_row(z, 6, t)
        r = ot.distill_row(z, v, i, tail, t=t)
        assert abs(r["loss"]) < 1e-14 and np.abs(r["grad"]).max() < 1e-15
        assert ot.distill_row(rng.normal(size=50), v, i, tail, t=t)["loss"] > 0


@pytest.mark.parametrize("with_tail", [True, False])
@pytest.mark.parametrize("t", [0.5, 1.0, 2.0])
def test_gradient_finite_differences(with_tail, t):
    rng = np.random.default_rng(7)
    V, K = 23, 5
    z = rng.normal(size=V) * 2
    v, i, tail, _ = ot.top_row(rng.normal(size=V) * 2, K, t)
    v[3], i[3] = -np.inf, -1                        # an empty slot
    tail = tail if with_tail else -np.inf
    r = ot.distill_row(z, v, i, tail, weight=0.3, t=t)
    h = 1e-6
    for u in range(V):
        zp, zm = z.copy(), z.copy()
        zp[u] += h
        zm[u] -= h
        num = 0.3 * (ot.distill_row(zp, v, i, tail, t=t)["loss"] - ot.distill_row(zm, v, i, tail, t=t)["loss"]) / (2 * h)
        assert r["grad"][u] == pytest.approx(num, abs=1e-9)
    assert abs(r["grad"].sum()) < 1e-14


def test_rows_without_a_teacher_or_weight():
    z = np.array([1.0, 2.0, 3.0])
    r = ot.distill_row(z, np.array([5.0]), np.array([-1]))
    assert r["loss"] == 0.0 and (r["grad"] == 0).all() and r["lse"] == pytest.approx(ot.lse(z))
    r = ot.distill_row(np.full(3, np.nan), np.array([5.0]), np.array([1]), weight=0.0)
    assert r["loss"] == 0.0 and (r["grad"] == 0).all()
    # a rest and no named entry: both sides are one bucket
    r = ot.distill_row(z, np.array([5.0]), np.array([-1]), tail=2.0)
    assert r["loss"] == pytest.approx(0.0, abs=1e-15) and np.abs(r["grad"]).max() < 1e-15
    # mass on what the student rules out
    r = ot.distill_row(np.array([0.0, -np.inf]), np.zeros(2), np.array([0, 1]))
    assert r["loss"] == np.inf and r["grad"].tolist() == [0.5, -0.5]
    for ids in ([0, 0], [3, 1], [-2, 1]):
        assert np.isnan(ot.distill_row(z, np.zeros(2), np.array(ids))["loss"])
