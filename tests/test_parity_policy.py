"""policy_loss against the float64 oracle (one GB300)."""

import numpy as np
import pytest
import torch

import verify_spec_draft_gb300 as vsd
from oracle import policy as op

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def inputs(R, V, dtype, seed, t=1.0, low=0.2, high=0.28, scale=3.0, offset=0.0):
    rng = np.random.default_rng(seed)
    z = torch.from_numpy((rng.normal(size=(R, V)) * scale + offset).astype(np.float32)).to(dtype)
    x = np.where(rng.random(R) < 0.5, z.double().numpy().argmax(1), rng.integers(0, V, R)).astype(np.int32)
    lp = np.array([op.row(z[i].double().numpy(), int(x[i]), 0.0, 0.0, t=t)["logp"] for i in range(R)])
    moved = rng.normal(size=R) * 0.25
    for border in (np.log(1 - low) if low < 1 else -50.0, np.log(1 + high)):   # no row on a border
        moved = np.where(np.abs(moved - border) < 1e-3, moved + 4e-3, moved)
    old = (lp - moved).astype(np.float32)
    return dict(z=z, x=torch.from_numpy(x), old=torch.from_numpy(old),
                A=torch.from_numpy(rng.normal(size=R).astype(np.float32)),
                ref=torch.from_numpy((lp + 0.5 * rng.normal(size=R)).astype(np.float32)),
                w=torch.from_numpy((rng.random(R) * (rng.random(R) > 0.2)).astype(np.float32)))


def call(d, grad=True, kl=0.05, t=1.0, low=0.2, high=0.28, ref=True, weight=True, **kw):
    c = {k: v.cuda() for k, v in d.items() if k != "z"}
    z = d["z"] if d["z"].is_cuda else d["z"].cuda()
    return vsd.policy_loss(z, c["x"], c["old"], c["A"], ref_logp=c["ref"] if ref else None,
                           weight=c["w"] if weight else None, temperature=t, clip=(low, high), kl=kl, grad=grad, **kw)


def oracle(d, kl=0.05, t=1.0, low=0.2, high=0.28, ref=True, weight=True):
    return op.policy_loss(d["z"].cpu().double().numpy(), d["x"].numpy(), d["old"].double().numpy(),
                          d["A"].double().numpy(), d["ref"].double().numpy() if ref else None,
                          d["w"].double().numpy() if weight else None, t, float(np.float32(low)), float(np.float32(high)),
                          float(np.float32(kl)))


def check(d, got, want, t, kl, grad=True):
    """Tolerances, in roundings e = 2^-24.  ln Z: a weight 2^x is off by the rounding of its argument (|x| e; the
    weights that matter have |x| < 24), by 2^-22 of the instruction's own, and a thread's sum of V / 256
    entries at most (two accumulators), the merges' some 30 more: zt = (24 + 4 + V / 512 + 30) e, at most.
    lp adds the roundings of (z - M) / t (two of its size), of ln Z and of the difference."""
    e = 2.0 ** -24
    z, x, w = d["z"].cpu().double().numpy(), d["x"].numpy(), d["w"].double().numpy()
    R, V = z.shape
    np.seterr(invalid="ignore")   # rows without an answer are left out of the comparisons
    zt = (58 + V / 512) * e
    on = np.isfinite(want["loss"])
    gap = np.abs(z.max(1) - z[np.arange(R), np.clip(x, 0, V - 1)]) / t
    lp_bar = np.where(np.isfinite(gap), 3 * gap, 0) * e + zt + 3 * np.abs(np.where(on, want["logp"], 0)) * e
    got_lp, got_loss = got["logp"].double().cpu().numpy(), got["loss"].double().cpu().numpy()
    fin = on & np.isfinite(want["logp"])
    assert (np.isnan(got_loss) == np.isnan(want["loss"])).all() and (got_loss[np.isinf(want["loss"])] == np.inf).all()
    assert (np.abs(got_lp - want["logp"])[fin] <= lp_bar[fin]).all()
    # u and e^d are off by lp's error and a few roundings of their own (4, for expf, expm1f and the products)
    lp = np.where(fin, want["logp"], 0.0)
    u = np.where(fin, np.exp(np.minimum(lp - d["old"].double().numpy(), 80)), 0)
    ed = np.exp(np.minimum(d["ref"].double().numpy() - lp, 80)) if kl else 0 * u
    A = np.abs(d["A"].double().numpy())
    rel = lp_bar + 8 * e
    slope_bar = (u * A + kl * (ed + 1)) * rel
    loss_bar = slope_bar + (2 * A + kl * (ed + np.abs(d["ref"].double().numpy() - lp) + 1)) * 8 * e
    assert (np.abs(got_loss - want["loss"])[on] <= loss_bar[on]).all()
    if not grad:
        return
    g = got["grad"].double().cpu().numpy()
    bad = np.isnan(want["grad"])
    assert (np.isnan(g) == bad).all()
    ok = ~bad.any(1)
    ind = np.abs(np.where(np.arange(V)[None] == x[:, None], 1 - want["q"], want["q"]))   # |[v = x] - q|
    k = np.abs(w) / t
    half = 2.0 ** -8 if d["z"].dtype == BF16 else e
    # an entry's weight: its argument's rounding (|x| e, x = log2 q at most), as much as Z's error again
    arg = np.abs(np.log2(np.maximum(ind, 1e-38)))
    bar = k[:, None] * (slope_bar[:, None] * ind + np.abs(want["slope"])[:, None] * ind * (2 * zt + (2 * arg + 8) * e))
    bar = bar * 1.02 + half * np.abs(want["grad"]) + 1e-38
    if d["z"].dtype == BF16:
        bar = bar + 2.0 ** -134    # half the spacing of bf16's smallest numbers
    assert (np.abs(g - want["grad"])[ok] <= bar[ok]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("R,V", [(1, 1), (3, 2), (5, 7), (4, 33), (9, 1000), (2, 4099), (7, 32000), (3, 50257), (2, 131073)])
def test_sizes(spec, R, V, dtype):
    d = inputs(R, V, dtype, seed=V)
    got, want = call(d), oracle(d)
    check(d, got, want, 1.0, 0.05)
    assert vsd.device_status(got["ws"]) == 0
    alone = call(d, grad=False)
    check(d, alone, want, 1.0, 0.05, grad=False)


@pytest.mark.parametrize("t,kl,low,high", [(0.5, 0.0, 0.2, 0.2), (2.0, 0.3, 0.0, 0.0), (1.0, 0.0, 1.0, 5.0), (0.7, 1.0, 0.1, 0.3)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_settings(spec, t, kl, low, high, dtype):
    d = inputs(40, 3001, dtype, seed=3, t=t, low=low, high=high)
    kw = dict(t=t, kl=kl, low=low, high=high, ref=kl > 0)
    check(d, call(d, **kw), oracle(d, **kw), t, kl)


@pytest.mark.parametrize("dtype,V,ld", [(F32, 5001, 5004), (F32, 5001, 5003), (BF16, 5001, 5008), (BF16, 5001, 5005),
                                        (BF16, 8192, 8193)])
def test_row_strides_and_neighbours(spec, dtype, V, ld):
    """Rows that lie further apart, at any offset: what lies between them stays."""
    d = inputs(6, V, dtype, seed=11)
    room = torch.full((6, ld), 7.0, dtype=dtype, device="cuda")
    room[:, :V] = d["z"].cuda()
    out = torch.full((6, ld), 9.0, dtype=dtype, device="cuda")
    got = call(dict(d, z=room[:, :V]), out=dict(loss=torch.empty(6, device="cuda"), logp=torch.empty(6, device="cuda"),
                                                 grad=out[:, :V]))
    check(d, got, oracle(d), 1.0, 0.05)
    assert (out[:, V:] == 9.0).all() and (room[:, V:] == 7.0).all()
    # in place
    got2 = call(dict(d, z=room[:, :V]), out=dict(loss=got["loss"].clone(), logp=got["logp"].clone(), grad=room[:, :V]))
    assert torch.equal(got2["grad"], got["grad"]) and torch.equal(got2["loss"], got["loss"]) and (room[:, V:] == 7.0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_masked_entries(spec, dtype):
    """Entries of -inf have no probability and no gradient; the type's lowest value and -1e30 neither."""
    d = inputs(8, 2000, dtype, seed=5)
    z = d["z"]
    z[0, :] = -torch.inf
    z[0, int(d["x"][0])] = 1.0                        # the token alone: lp = 0, gradient 0
    z[1, 100:] = -torch.inf
    d["x"][1] = 50
    z[2, 100:] = torch.finfo(dtype).min
    d["x"][2] = 50
    z[3, 100:] = -1e30
    d["x"][3] = 7
    z[4] = (z[4].float() * 1e-3 - 1e10).to(dtype)      # a whole row far from zero
    z[5] = (z[5].float() + 3e5).to(dtype)
    d["old"] = torch.zeros(8) - 1.0
    d["ref"] = torch.zeros(8) - 1.2
    d["A"] = torch.linspace(0.5, 1.5, 8)
    d["w"] = torch.full((8,), 0.25)
    for i in range(8):                                  # u = 1.1: away from the borders
        d["old"][i] = op.row(z[i].double().numpy(), int(d["x"][i]), 0.0, 0.0)["logp"] - 0.095
        d["ref"][i] = d["old"][i] - 0.3
    got, want = call(d), oracle(d)
    check(d, got, want, 1.0, 0.05)
    assert (got["grad"][1, 100:] == 0).all() and (got["grad"][2, 100:] == 0).all() and got["logp"][0] == 0
    assert vsd.device_status(got["ws"]) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_without_an_answer(spec, dtype):
    d = inputs(14, 1500, dtype, seed=6)
    d["w"] = torch.full((14,), 0.5)
    z = d["z"]
    z[0, 3] = torch.nan
    z[1, 1499] = torch.inf
    z[2] = -torch.inf
    d["old"][3] = torch.nan
    d["A"][4] = torch.inf
    d["ref"][5] = -torch.inf
    d["w"][6] = torch.nan
    d["w"][7] = 0.0
    z[7] = torch.nan                                    # not read
    d["x"][7] = -9
    z[8, int(d["x"][8])] = -torch.inf                   # a token of probability 0: loss inf, no gradient
    d["old"][9], d["A"][9] = -1000.0, -1.0              # u beyond float32's range
    d["A"][10] = 0.0
    got, want = call(d), oracle(d)
    check(d, got, want, 1.0, 0.05)
    assert got["loss"][8] == torch.inf and got["logp"][8] == -torch.inf and got["loss"][9] == torch.inf
    assert got["loss"][7] == 0 and got["logp"][7] == 0 and (got["grad"][7] == 0).all()
    assert vsd.device_status(got["ws"]) == vsd.DEV_NONFINITE
    for x in (-1, 1500):
        e = inputs(3, 1500, dtype, seed=7)
        e["x"][1], e["w"][1] = x, 1.0
        r = call(e)
        assert torch.isnan(r["loss"][1]) and torch.isnan(r["logp"][1]) and torch.isnan(r["grad"][1]).all()
        assert torch.isfinite(r["grad"][[0, 2]]).all() and vsd.device_status(r["ws"]) == vsd.DEV_TOKEN


@pytest.mark.parametrize("dtype,V", [(F32, 1 << 20), (BF16, 1 << 20), (F32, 600011), (BF16, 248320)])
def test_largest_rows(spec, dtype, V):
    """Rows over many CTAs, the largest read twice; aliased as well."""
    d = inputs(3, V, dtype, seed=8)
    got, want = call(d), oracle(d)
    check(d, got, want, 1.0, 0.05)
    z = d["z"].cuda()
    again = call(dict(d, z=z), out=dict(loss=torch.empty(3, device="cuda"), logp=torch.empty(3, device="cuda"), grad=z))
    assert torch.equal(again["grad"], got["grad"]) and torch.equal(again["loss"], got["loss"])


# more rows than the device holds at once, of one CTA each and of several; words that are not whole
@pytest.mark.parametrize("R,V,dtype", [(2000, 301, BF16), (400, 40000, F32), (700, 12001, F32), (420, 70001, BF16)])
def test_many_rows(spec, R, V, dtype):
    d = inputs(R, V, dtype, seed=9)
    d["w"][:3] = 0.0
    d["w"][-1] = 0.0
    check(d, call(d), oracle(d), 1.0, 0.05)
    check(d, call(d, grad=False, weight=False), oracle(d, weight=False), 1.0, 0.05, grad=False)


def test_rows_past_32_bits(spec):
    """2.2e9 entries: the last rows against the same rows alone."""
    R, V = 8700, 248320
    z = torch.zeros((R, V), dtype=BF16, device="cuda")
    d = inputs(4, V, BF16, seed=13)
    z[-4:] = d["z"].cuda()
    x = torch.zeros(R, dtype=torch.int32, device="cuda")
    x[-4:] = d["x"].cuda()
    old, adv, w = (torch.zeros(R, device="cuda") for _ in range(3))
    old[-4:], adv[-4:], w[-4:] = d["old"].cuda(), d["A"].cuda(), 0.25
    w[0] = 0.25
    got = vsd.policy_loss(z, x, old, adv, weight=w, grad=True)
    alone = vsd.policy_loss(z[-4:], x[-4:].contiguous(), old[-4:].contiguous(), adv[-4:].contiguous(),
                            weight=w[-4:].contiguous(), grad=True)
    assert (got["grad"][1:-4] == 0).all() and got["logp"][1:-4].abs().sum() == 0
    # the rows alone may be split among other CTAs: their sums' order differs, each within its bar
    bar = 2 * (58 + V / 512) * 2.0 ** -24
    assert (got["logp"][-4:] - alone["logp"]).abs().max() <= bar * 2
    assert ((got["grad"][-4:].float() - alone["grad"].float()).abs() <= (2 * 2.0 ** -8 + 4 * bar) * alone["grad"].float().abs() + 1e-30).all()


def test_gradient_against_differences(spec):
    """The loss's own differences, in the direction of each of a few entries."""
    d = inputs(6, 40, F32, seed=12)
    d["w"] = torch.ones(6)
    g = call(d)["grad"].double().cpu().numpy()
    h = 2.0 ** -6
    for v in (0, 13, 39):
        up, dn = d["z"].clone(), d["z"].clone()
        up[:, v] += h
        dn[:, v] -= h
        num = (call(dict(d, z=up))["loss"] - call(dict(d, z=dn))["loss"]).double().cpu().numpy() / (2 * h)
        want = oracle(d)
        exact = (oracle(dict(d, z=up))["loss"] - oracle(dict(d, z=dn))["loss"]) / (2 * h)
        # what the difference leaves out is the oracle's own; each loss is off by some 60 roundings of 10
        assert (np.abs((num - exact)) <= 2 * 60 * 2.0 ** -24 * 10 / (2 * h)).all()
        assert (np.abs(g[:, v] - want["grad"][:, v]) <= 1e-4 * (1 + np.abs(want["grad"][:, v]))).all()


def test_refusals(spec):
    d = {k: v.cuda() for k, v in inputs(4, 100, F32, seed=1).items()}
    args = (d["z"], d["x"], d["old"], d["A"])
    with pytest.raises(ValueError, match="ref_logp"):
        vsd.policy_loss(*args, kl=0.1)
    with pytest.raises(ValueError):
        vsd.policy_loss(d["z"], d["x"].long(), d["old"], d["A"])
    with pytest.raises(ValueError):
        vsd.policy_loss(d["z"], d["x"][:3], d["old"], d["A"])
    with pytest.raises(ValueError):
        vsd.policy_loss(d["z"], None, d["old"], d["A"])
    with pytest.raises(TypeError):
        vsd.policy_loss(d["z"].half(), d["x"], d["old"], d["A"])
    for bad in (dict(temperature=0.0), dict(clip=(1.5, 0.2)), dict(clip=(0.2, -1.0)), dict(kl=-0.1)):
        with pytest.raises(vsd.SpecError):
            vsd.policy_loss(*args, **bad)
    with pytest.raises(ValueError):
        vsd.policy_loss(*args, out=dict(loss=torch.empty(4, device="cuda")))
    with pytest.raises(ValueError):
        vsd.policy_loss(*args, grad=True, out=dict(loss=torch.empty(4, device="cuda"), logp=torch.empty(4, device="cuda")))
    with pytest.raises(vsd.SpecError):
        vsd.policy_loss(*args, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
