"""Pins of oracle.policy, oracle.markov and oracle.adamw: worked values, limits, finite differences."""

import numpy as np
import pytest

from oracle import adamw as oa, draft as od, markov as om, policy as op


# ------------------------------------------------------------------------------ policy
@pytest.mark.parametrize("u,A,want,flows", [
    (1.0, 2.0, -2.0, True), (1.1, 2.0, -2.2, True), (1.5, 2.0, -2.4, False), (0.5, 2.0, -1.0, True),
    (0.9, -2.0, 1.8, True), (0.5, -2.0, 1.6, False), (1.5, -2.0, 3.0, True), (1.5, 0.0, 0.0, False)])
def test_policy_worked_rows(u, A, want, flows):
    z = np.log([4.0, 1.0, 3.0])
    r = op.row(z, 2, np.log(0.375 / u), A)
    assert r["logp"] == pytest.approx(np.log(0.375)) and r["loss"] == pytest.approx(want)
    slope = -u * A if flows else 0.0
    np.testing.assert_allclose(r["grad"], slope * (np.array([0, 0, 1]) - np.array([4, 1, 3]) / 8), rtol=1e-12, atol=1e-300)


@pytest.mark.parametrize("t", [0.5, 1.0, 2.0])
def test_policy_gradient_finite_differences(t):
    rng = np.random.default_rng(3)
    V = 17
    for A, ref in ((1.3, -2.0), (-0.7, -3.5), (0.4, None)):
        z = rng.normal(size=V) * 2
        x = int(rng.integers(V))
        kw = dict(t=t, kl=0.3 if ref is not None else 0.0, low=0.3, high=0.4)
        old = op.row(z, x, 0.0, A)["logp"] - 0.1 if t == 1.0 else op.row(z, x, 0.0, A, t=t)["logp"] - 0.1
        r = op.row(z, x, old, A, ref, weight=0.3, **kw)
        for v in range(V):
            h = np.zeros(V)
            h[v] = 1e-6
            num = 0.3 * (op.row(z + h, x, old, A, ref, **kw)["loss"] - op.row(z - h, x, old, A, ref, **kw)["loss"]) / 2e-6
            # the two losses carry some 4 roundings of 2^-53 each (1e-15 of the loss together), over 2e-6:
            # 5e-10 of it; what central differences leave out is h^2 = 1e-12 of third derivatives
            assert r["grad"][v] == pytest.approx(num, abs=1e-8 + 1e-9 * abs(r["loss"]))
        assert abs(r["grad"].sum()) < 1e-14 * (1 + abs(r["slope"]))


def test_policy_kl_term():
    z = np.log([4.0, 1.0, 3.0])
    lp = np.log(0.5)
    at = op.row(z, 0, lp, 0.0, ref=lp, kl=1.0)
    assert abs(at["loss"]) < 1e-15 and np.abs(at["grad"]).max() < 1e-15
    for ref in (-3.0, -0.1, -0.7):
        assert op.row(z, 0, lp, 0.0, ref=ref, kl=1.0)["loss"] == pytest.approx(np.exp(ref - lp) - (ref - lp) - 1)
    # a token of probability 0: no ratio, and with a KL term nothing finite
    z[1] = -np.inf
    r = op.row(z, 1, -1.0, -2.0)
    assert r["logp"] == -np.inf and r["loss"] == pytest.approx(1.6) and (r["grad"] == 0).all()
    r = op.row(z, 1, -1.0, -2.0, ref=-1.0, kl=0.1)
    assert r["loss"] == np.inf and np.isnan(r["grad"]).all()


def test_policy_invalid_rows():
    z = np.zeros(3)
    for bad in (dict(x=3), dict(x=-1), dict(old=np.nan), dict(A=np.inf), dict(weight=np.nan), dict(ref=np.inf, kl=1.0)):
        r = op.row(z, **{**dict(x=0, old=0.0, A=1.0), **bad})
        assert np.isnan(r["loss"]) and np.isnan(r["grad"]).all()
    assert np.isnan(op.row(np.full(3, -np.inf), 0, 0.0, 1.0)["loss"])
    r = op.row(np.full(3, np.nan), -5, np.nan, np.nan, weight=0.0)
    assert r["loss"] == 0 and (r["grad"] == 0).all()


# ------------------------------------------------------------------------------ markov
def test_markov_gradient_against_the_drafts_rows():
    """d(sum of c z) with z the rows that the draft returns, its tokens held."""
    rng = np.random.default_rng(5)
    B, G, V, r = 2, 4, 11, 3
    logits, U, Wt = rng.normal(size=(B, G, V)) * 3, rng.normal(size=(V, r)) * 0.1, rng.normal(size=(V, r)) * 0.1
    anchor = np.array([3, 3])
    c = rng.normal(size=(B, G, V))

    def rows(U, Wt):
        d = od.draft_block(logits, anchor, U, Wt, 0, None, return_z=True)
        return d["z"], d["tokens"]
    z, tok = rows(U, Wt)
    g = om.markov_grad(c, anchor, tok, U, Wt)
    for name, M in (("U", U), ("Wt", Wt)):
        for at in [(3, 0), (3, 2), (int(tok[0, 0]), 1), (7, 1), (0, 2)]:
            h = np.zeros_like(M)
            h[at] = 1e-6
            up, t1 = rows(U + h, Wt) if name == "U" else rows(U, Wt + h)
            dn, t2 = rows(U - h, Wt) if name == "U" else rows(U, Wt - h)
            assert (t1 == tok).all() and (t2 == tok).all()
            assert g[name][at] == pytest.approx((c * (up - dn)).sum() / 2e-6, abs=1e-7)


def test_markov_tokens_that_come_back_and_blocks_that_end():
    rng = np.random.default_rng(6)
    V, r = 6, 2
    U, Wt = rng.normal(size=(V, r)), rng.normal(size=(V, r))
    dz = rng.normal(size=(2, 3, V))
    tokens = np.array([[4, 4, 0], [-1, -1, -1]])
    dz[1, 1:] = np.nan
    g = om.markov_grad(dz, np.array([4, 1]), tokens, U, Wt)
    np.testing.assert_allclose(g["U"][4], dz[0].sum(0) @ Wt)
    np.testing.assert_allclose(g["U"][1], dz[1, 0] @ Wt)
    assert (g["U"][[0, 2, 3, 5]] == 0).all() and np.isfinite(g["Wt"]).all()


# ------------------------------------------------------------------------------- adamw
def test_adamw_worked_steps():
    # the first step moves by lr against the gradient's sign, whatever its size
    for g in (1e-3, 5.0, -2.0):
        p, m, v = oa.step(1.0, g, 0.0, 0.0, 1, lr=0.1, eps=1e-300, wd=0.0)
        assert p == pytest.approx(1.0 - 0.1 * np.sign(g)) and m == pytest.approx(0.1 * g) and v == pytest.approx(1e-3 * g * g)
    assert oa.step(2.0, 0.0, 0.0, 0.0, 1, lr=0.1, wd=0.5)[0] == pytest.approx(1.9)
    p, m, v = 1.0, 0.0, 0.0
    for T in range(1, 50):
        q, m, v = oa.step(p, 3.0, m, v, T, lr=0.01, eps=1e-300, wd=0.0)
        assert q == pytest.approx(p - 0.01)
        p = q


def test_philox4x32_published_answers():
    """The known answers that the generator's authors publish (kat_vectors of Random123)."""
    for key, counter, want in (
            ((0, 0), (0, 0, 0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((0xFFFFFFFF,) * 2, (0xFFFFFFFF,) * 4, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0xA4093822, 0x299F31D0), (0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        assert tuple(int(w) for w in oa.philox4x32(key, counter)) == want


def test_codes():
    torch = pytest.importorskip("torch")
    codes = np.array([c for c in range(256) if c & 127 != 127])
    want = torch.tensor(codes, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert (oa.code_value(codes) == want).all()
    # what is a code's value stays one, whatever the random number
    x = np.append(want[np.abs(want) < 256], 255.0)   # the block's largest in [128, 256)
    for random in (0, 1, 65535):
        code, s, _ = oa.encode(x[-128:], np.full(128, random))
        assert s[0] == 1.0 and (oa.code_value(code)[:-1] == x[-128:-1]).all()


def test_random_rounding_has_the_value_as_its_mean():
    rng = np.random.default_rng(8)
    x = rng.normal(size=256) * np.exp(rng.normal(size=256) * 3)
    total, n = np.zeros(256), 64
    for k in range(n):                              # stratified: every 1024th random number
        code, s, _ = oa.encode(x, np.full(256, k * 1024))
        total += oa.code_value(code) * np.repeat(s, 128)
    assert (np.abs(x).reshape(2, 128).max(1) / s >= 128).all() and (np.abs(x).reshape(2, 128).max(1) / s < 256).all()
    # a code's spacing is at most 1/8 of the value, 2^-9 of the scale; the strata miss by 1/64 of it
    assert (np.abs(total / n - x) <= (np.abs(x) / 8 + np.repeat(s, 128) * 2.0 ** -9) / n).all()
    code, s, _ = oa.encode(np.array([1e-9, 1.0, 0.0]), np.zeros(3), root=True)
    assert code[0] == 1 and code[2] == 0
    a, b = oa.random16(12345, 1000, 7, 3)
    assert abs(a.mean() / 65536 - 0.5) < 0.05 and abs(b.mean() / 65536 - 0.5) < 0.05 and a.max() < 65536 and b.max() < 65536
