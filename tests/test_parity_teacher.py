"""spec_top_logits and spec_distill on the GPU against the float64 oracle.

ids and values are exact.  Bars of the float32 sums: a weight 2^((z - m) log2e / t) is off by
2^-24 of its exponent (the scale's and the difference's rounding) plus 2^-22 (the exponential),
and weights matter down to 2^-20 of the largest; a sum adds at most about 40 roundings on any
path; the maximum / t adds one rounding of its own size.  So a logarithm of a sum is off by at
most
    EPS(z) = 2^-24 (4 max|z / t| + 100),
and a probability by that relative amount.  The loss, sum p (ln p - ln q), then by
2 (EPS(z) + EPS(a)) (1 + sum p |ln p - ln q|), and a gradient entry by
(weight / t) 2 (EPS(z) + EPS(a)) (p + q (1 + p_T / q_T)); a bf16 gradient rounds once more, by at
most 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

import verify_spec_draft_gb300 as vsd
from oracle import teacher as ot

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def f64(t):
    return t.double().cpu().numpy()


def eps(z, t):
    z = f64(z) if torch.is_tensor(z) else np.asarray(z)
    z = np.abs(z[np.isfinite(z)])
    return 2.0 ** -24 * (4 * (z.max() if z.size else 0) / t + 100)


def rows_of(R, V, dtype, seed, kind="gaussian", ld=None):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((R, V), generator=g) * 3
    if kind == "coarse":                       # many equal values
        z = (z * 2).round() / 2
    elif kind == "grammar":                    # a handful of entries is allowed
        z[torch.rand((R, V), generator=g) > 12.0 / V] = -torch.inf
        z[:, V // 2] = 1.0
    elif kind == "constant":
        z[:] = 1.25
    elif kind == "ascending":
        z = z.sort(1).values
    elif kind == "descending":
        z = z.sort(1, descending=True).values
    elif kind == "lowest":                     # masked with the type's lowest value
        z[torch.rand((R, V), generator=g) > 0.05] = torch.finfo(dtype).min
    elif kind == "peak":                       # the rest is e^-60 of the row
        z[torch.arange(R), torch.randint(0, V, (R,), generator=g)] = 75.0
    elif kind == "striped":                    # the large entries 2048 apart
        z[:, ::2048] += 40.0
    elif kind == "zeros":                      # both signs of zero
        z = torch.where(z > 2, z, torch.where(z > 0, 0.0, -0.0))
    out = torch.zeros((R, ld or V), dtype=dtype, device="cuda")[:, :V]
    out.copy_(z)
    return out


def check_top(z, K, t, out):
    ref = ot.top_logits(f64(z), K, t)
    np.testing.assert_array_equal(out["ids"].cpu().numpy(), ref["ids"])
    np.testing.assert_array_equal(f64(out["values"]), ref["values"])
    for k in ("tail", "lse"):
        got, want = f64(out[k]), ref[k]
        fin = np.isfinite(want)
        np.testing.assert_array_equal(got[~fin], want[~fin])
        for r in np.nonzero(fin)[0]:
            row = f64(z[r])
            big = row[np.isfinite(row) & (row > -1e30)]
            bar = eps(big, t) + 2.0 ** -23 * abs(want[r])
            assert abs(got[r] - want[r]) <= bar, (k, r, got[r], want[r])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("R,V,K,t", [
    (1, 1, 1, 1.0), (3, 1, 4, 1.0), (2, 5, 8, 0.7), (2, 127, 20, 1.0), (3, 128, 128, 2.0), (5, 257, 1, 1.0),
    (2, 1000, 64, 1.5), (7, 4099, 100, 1.0), (2, 16384, 20, 1.0), (3, 20001, 128, 0.5), (1, 65537, 33, 1.0)])
def test_top_sizes(spec, dtype, R, V, K, t):
    z = rows_of(R, V, dtype, seed=R + V + K)
    out = vsd.top_logits(z, K, temperature=t)
    check_top(z, K, t, out)
    assert vsd.device_status(out["ws"]) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["coarse", "grammar", "constant", "ascending", "descending", "lowest", "peak",
                                  "striped", "zeros"])
@pytest.mark.parametrize("V,K", [(9000, 20), (33001, 128)])
def test_top_distributions(spec, dtype, kind, V, K):
    z = rows_of(3, V, dtype, seed=11, kind=kind)
    check_top(z, K, 1.0, vsd.top_logits(z, K))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("R,V,K", [(40, 151936, 128), (33, 151937, 128), (160, 33024, 100), (700, 4000, 20)])
def test_top_many_rows(spec, dtype, R, V, K):
    """Rows enough for picks of their own launch, chosen blocks enough for several looks."""
    z = rows_of(R, V, dtype, seed=V + K, kind="coarse" if R == 33 else "gaussian")
    out = vsd.top_logits(z, K)
    check_top(z, K, 1.0, out)
    assert vsd.device_status(out["ws"]) == 0


@pytest.mark.parametrize("dtype,V,ld", [(F32, 1001, 1003), (BF16, 1001, 1009), (BF16, 5000, 5008)])
def test_top_row_stride(spec, dtype, V, ld):
    z = rows_of(6, V, dtype, seed=2, ld=ld)
    assert z.stride(0) == ld
    check_top(z, 20, 1.0, vsd.top_logits(z, 20))


def test_top_shapes_and_workspace(spec):
    z = rows_of(6, 3001, BF16, seed=3)
    ws = vsd.workspace(vsd.OP_TOP_LOGITS, 6, 9, 3001)
    a = vsd.top_logits(z.view(2, 3, 3001), 9, ws=ws)
    assert a["values"].shape == (2, 3, 9) and a["tail"].shape == (2, 3)
    first = {k: a[k].clone() for k in ("values", "ids", "tail", "lse")}
    b = vsd.top_logits(z.view(2, 3, 3001), 9, ws=ws)
    for k in first:
        assert torch.equal(first[k], b[k])
    check_top(z, 9, 1.0, {k: first[k].view(6, *first[k].shape[2:]) for k in first})


def test_top_invalid_rows(spec):
    for dtype in (F32, BF16):
        z = rows_of(5, 3001, dtype, seed=4)
        z[1, 77], z[2, 3000] = float("nan"), float("inf")
        z[3] = -torch.inf
        out = vsd.top_logits(z, 10)
        check_top(z, 10, 1.0, out)
        assert vsd.device_status(out["ws"]) == vsd.DEV_NONFINITE


def test_top_refusals(spec):
    z = rows_of(2, 100, F32, seed=1)
    for k in (0, 129):
        with pytest.raises(vsd.SpecError):
            vsd.top_logits(z, k)
    with pytest.raises(vsd.SpecError):
        vsd.top_logits(z, 3, temperature=0.0)
    with pytest.raises(TypeError):
        vsd.top_logits(z.half(), 3)
    with pytest.raises(ValueError):
        vsd.top_logits(z.t(), 3)


# ---------------------------------------------------------------------------------
def teacher_of(z, K, t, with_tail, seed, values_dtype=F32):
    """A teacher row per student row: the top of a noisy copy, as tensors on the GPU."""
    g = torch.Generator().manual_seed(seed)
    noisy = z.float().cpu()
    noisy = noisy + torch.randn(noisy.shape, generator=g)
    noisy[noisy < -1e30] = -torch.inf
    top = ot.top_logits(noisy.to(z.dtype).double().numpy(), K, t)
    values = torch.from_numpy(top["values"]).to(values_dtype).cuda()
    ids = torch.from_numpy(top["ids"]).to(torch.int32).cuda()
    tail = torch.from_numpy(top["tail"]).float().cuda() if with_tail else None
    return values, ids, tail


def check_distill(z, values, ids, tail, weight, t, out, grad=True):
    ref = ot.distill(f64(z), f64(values), ids.cpu().numpy(), None if tail is None else f64(tail),
                     None if weight is None else f64(weight), t)
    R, V = z.shape
    for r in range(R):
        row, a = f64(z[r]), f64(values[r])
        e = eps(row[np.abs(row) < 1e30], t) + eps(a[np.abs(a) < 1e30], t)
        if tail is not None:
            e += eps(f64(tail[r:r + 1]), 1.0)
        want, got = ref["loss"][r], float(out["loss"][r])
        assert np.isnan(want) == np.isnan(got), (r, want, got)
        if np.isnan(want):
            if grad:
                assert torch.isnan(out["grad"][r]).all()
            continue
        assert abs(float(out["lse"][r]) - ref["lse"][r]) <= e + 2.0 ** -23 * abs(ref["lse"][r])
        p, q, qt = ref["p"][r], ref["q"][r], ref["qt"][r]
        if np.isinf(want):
            assert got == want
        else:
            on = p > 0
            lq = np.append([np.log(max(q[i], 1e-300)) if i >= 0 else 0.0 for i in ids[r].cpu().numpy()],
                           np.log(max(qt, 1e-300)))
            size = (p[on] * np.abs(np.log(p[on]) - lq[on])).sum()
            assert abs(got - want) <= 2 * e * (1 + size), (r, got, want)
        if grad:
            w = 1.0 if weight is None else abs(float(weight[r]))
            ratio = p[-1] / qt if qt > 0 else 0.0
            pv = np.zeros(V)
            named = ids[r].cpu().numpy()
            pv[named[named >= 0]] = p[:-1][named >= 0]
            bar = w / t * 2 * e * (pv + q * (1 + ratio)) + 1e-37
            g = ref["grad"][r]
            if z.dtype == BF16:
                bar = bar + 2.0 ** -8 * np.abs(g)
            bad = np.abs(f64(out["grad"][r]) - g) > bar
            assert not bad.any(), (r, np.nonzero(bad)[0][:5], f64(out["grad"][r])[bad][:5], g[bad][:5])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("R,V,K,t,tail", [
    (1, 1, 1, 1.0, False), (2, 1, 2, 1.0, True), (3, 5, 8, 0.7, True), (2, 127, 20, 1.0, True),
    (3, 128, 128, 2.0, False), (5, 257, 1, 1.0, True), (2, 1000, 64, 1.5, True), (7, 4099, 100, 1.0, False),
    (2, 16384, 20, 1.0, True), (3, 20001, 128, 0.5, True), (1, 65537, 33, 1.0, True), (40, 3001, 20, 1.0, True),
    (400, 130, 5, 1.0, True), (2, 131072, 64, 1.0, True)])
def test_distill_sizes(spec, dtype, R, V, K, t, tail):
    z = rows_of(R, V, dtype, seed=R + V + K)
    values, ids, tl = teacher_of(z, K, t, tail, seed=V)
    weight = torch.randn(R, generator=torch.Generator().manual_seed(V)).cuda()
    if R > 2:
        weight[1] = 0.0
    out = vsd.distill(z, values, ids, tail=tl, weight=weight, temperature=t, grad=True)
    check_distill(z, values, ids, tl, weight, t, out)
    assert vsd.device_status(out["ws"]) == 0
    alone = vsd.distill(z, values, ids, tail=tl, weight=weight, temperature=t)
    assert "grad" not in alone
    check_distill(z, values, ids, tl, weight, t, alone, grad=False)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", ["coarse", "grammar", "constant", "lowest", "peak", "striped"])
@pytest.mark.parametrize("V,K", [(9000, 20), (33001, 100)])
def test_distill_distributions(spec, dtype, kind, V, K):
    z = rows_of(3, V, dtype, seed=13, kind=kind)
    values, ids, tl = teacher_of(z, K, 1.0, True, seed=V)
    out = vsd.distill(z, values, ids, tail=tl, grad=True)
    check_distill(z, values, ids, tl, None, 1.0, out)


def test_distill_own_row(spec):
    z = rows_of(4, 20001, F32, seed=5)
    top = vsd.top_logits(z, 50, temperature=1.3)
    out = vsd.distill(z, top["values"], top["ids"], tail=top["tail"], temperature=1.3, grad=True)
    check_distill(z, top["values"], top["ids"], top["tail"], None, 1.3, out)
    assert out["loss"].abs().max() < 1e-5 and out["grad"].abs().max() < 1e-6
    assert torch.allclose(out["lse"], top["lse"], rtol=0, atol=2e-5)


def test_distill_differences(spec):
    """The gradient against central differences of the call's own loss, in float32: a step of
    0.25 leaves a truncation of h^2 / 6 times a third derivative below 1, 0.0105, and the
    loss's rounding of 1e-5 over 2 h."""
    z = rows_of(1, 40, F32, seed=8)
    values, ids, tl = teacher_of(z, 6, 1.0, True, seed=9)
    g = vsd.distill(z, values, ids, tail=tl, grad=True)["grad"][0]
    step = 0.25 * torch.eye(40, device="cuda")
    rep = lambda x: None if x is None else x.expand(40, *x.shape[1:]).contiguous()    # noqa: E731
    up = vsd.distill((z + step).contiguous(), rep(values), rep(ids), tail=rep(tl))["loss"]
    dn = vsd.distill((z - step).contiguous(), rep(values), rep(ids), tail=rep(tl))["loss"]
    assert ((up - dn) / 0.5 - g).abs().max() <= 0.0105 + 2e-5 / 0.5


def test_distill_hard_label_is_cross_entropy(spec):
    z = rows_of(5, 3001, F32, seed=6)
    label = torch.tensor([[0], [3000], [17], [512], [2047]], dtype=torch.int32, device="cuda")
    out = vsd.distill(z, torch.zeros((5, 1), device="cuda"), label, grad=True)
    ref = torch.log_softmax(z.double(), 1)
    want = -ref.gather(1, label.long())[:, 0]
    bar = 2 * (eps(z, 1.0) + 100 * 2.0 ** -24)
    assert (out["loss"].double() - want).abs().max() <= bar * (1 + want.max())
    g = ref.exp().scatter_add(1, label.long(), -torch.ones((5, 1), dtype=torch.float64, device="cuda"))
    assert (out["grad"].double() - g).abs().max() <= bar


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,K,named", [(5000, 3, 1e-3), (60001, 5, 1e-4), (131072, 2, 3e-5)])
def test_distill_little_named_mass(spec, dtype, V, K, named):
    """The rests hold nearly all of both rows, so the loss is far below 1 and its own digits
    count.  With p_N, q_N the named masses, a weight's relative error e moves the loss by e of
    its own mass (through the sums) and by e |ln p - ln q| of it (through the terms), the
    rest's weight by e |p_N - q_N|; a rest's gradient, q / q_T (p_N - q_N), by e (p_N + q_N) and
    e of itself.  Two roundings of the result are added."""
    z = rows_of(4, V, dtype, seed=V) / 3
    ids = torch.randint(0, V // K, (4, K), dtype=torch.int32, generator=torch.Generator().manual_seed(V)).cuda()
    ids += torch.arange(K, dtype=torch.int32, device="cuda") * (V // K)
    values = (torch.arange(K) + 1.0).div(K).mul(named).log().expand(4, K).contiguous().cuda()
    tl = torch.zeros(4, device="cuda")
    ref = ot.distill(f64(z), f64(values), ids.cpu().numpy(), f64(tl), None, 1.0)
    for grad in (False, True):
        out = vsd.distill(z, values, ids, tail=tl, grad=grad)
        for r in range(4):
            e = eps(z[r], 1.0) + eps(values[r], 1.0)
            p, q, qt = ref["p"][r][:-1], ref["q"][r], ref["qt"][r]
            qn = q[ids[r].cpu().numpy()]
            far = np.abs(np.log(p) - np.log(qn)).max()
            both = p.sum() + qn.sum()
            want = ref["loss"][r]
            bar = e * both * (2 + far) + 2.0 ** -23 * want
            assert want < 0.01
            assert abs(float(out["loss"][r]) - want) <= bar, (r, float(out["loss"][r]), want, bar)
            if grad:
                rest = np.ones(V, bool)
                rest[ids[r].cpu().numpy()] = False
                g = ref["grad"][r][rest]
                step = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
                bar = q[rest] / qt * 2 * e * both + (2 * e + 2 * step) * np.abs(g) + 1e-37
                assert (np.abs(f64(out["grad"][r])[rest] - g) <= bar).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_distill_bf16_values_and_empty_slots(spec, dtype):
    z = rows_of(4, 5000, dtype, seed=21)
    values, ids, tl = teacher_of(z, 30, 1.0, True, seed=22, values_dtype=BF16)
    ids[1, 3:20] = -1
    values[1, 3:20] = float("nan")           # what an empty slot holds is not looked at
    ids[2] = -1                              # the rest is all there is
    out = vsd.distill(z, values, ids, tail=tl, grad=True)
    check_distill(z, values, ids, tl, None, 1.0, out)
    none = vsd.distill(z, values, ids, grad=True)
    assert none["loss"][2] == 0 and (none["grad"][2] == 0).all()
    tl[3] = -torch.inf
    check_distill(z, values, ids, tl, None, 1.0, vsd.distill(z, values, ids, tail=tl, grad=True))


@pytest.mark.parametrize("dtype,V,ld", [(F32, 1001, 1003), (BF16, 1001, 1009), (BF16, 5000, 5008), (F32, 64, 100)])
def test_distill_row_stride_and_in_place(spec, dtype, V, ld):
    z = rows_of(6, V, dtype, seed=2, ld=ld)
    values, ids, tl = teacher_of(z, 20, 1.0, True, seed=3)
    buf = torch.full((6, ld), 7.0, dtype=dtype, device="cuda")
    out = dict(loss=torch.empty(6, device="cuda"), lse=torch.empty(6, device="cuda"), grad=buf[:, :V])
    vsd.distill(z, values, ids, tail=tl, grad=True, out=out)
    check_distill(z, values, ids, tl, None, 1.0, out)
    assert (buf[:, V:] == 7.0).all()
    own = vsd.distill(z, values, ids, tail=tl, grad=True,
                      out=dict(loss=torch.empty(6, device="cuda"), lse=None, grad=z))
    assert own["grad"] is z
    assert torch.equal(out["grad"], z) and torch.equal(out["loss"], own["loss"])


def test_distill_bad_rows(spec):
    for dtype in (F32, BF16):
        z = rows_of(12, 3001, dtype, seed=31)
        values, ids, tl = teacher_of(z, 10, 1.0, True, seed=32)
        z[0, 5], z[1, int(ids[1, 0])], z[2, 9] = float("nan"), float("nan"), float("inf")
        z[3] = -torch.inf
        values[4, 2], tl[5] = float("nan"), float("inf")
        out = vsd.distill(z, values, ids, tail=tl, grad=True)
        check_distill(z, values, ids, tl, None, 1.0, out)
        assert vsd.device_status(out["ws"]) == vsd.DEV_NONFINITE
        ids[6, 9] = ids[6, 0]
        ids[7, 4], ids[8, 4] = 3001, -2
        z[9, int(ids[9, 0])] = -torch.inf    # mass on what the student rules out: the loss is +inf
        weight = torch.ones(12, device="cuda")
        weight[0] = 0.0                      # a NaN row that does not count
        out = vsd.distill(z, values, ids, tail=tl, weight=weight, grad=True)
        check_distill(z, values, ids, tl, weight, 1.0, out)
        assert float(out["loss"][9]) == float("inf")
        assert vsd.device_status(out["ws"]) == vsd.DEV_NONFINITE | vsd.DEV_TOKEN


def test_distill_all_rows_skipped(spec):
    z = torch.full((9, 2000), float("nan"), device="cuda")
    ids = torch.zeros((9, 3), dtype=torch.int32, device="cuda")
    out = vsd.distill(z, torch.zeros((9, 3), device="cuda"), ids, weight=torch.zeros(9, device="cuda"), grad=True)
    assert (out["grad"] == 0).all() and (out["loss"] == 0).all() and (out["lse"] == 0).all()
    assert vsd.device_status(out["ws"]) == 0


def test_distill_workspace_reuse(spec):
    z = rows_of(33, 9001, BF16, seed=41)
    values, ids, tl = teacher_of(z, 20, 1.0, True, seed=42)
    ws = vsd.workspace(vsd.OP_DISTILL, 33, 20, 9001)
    first = vsd.distill(z, values, ids, tail=tl, grad=True, ws=ws)
    for _ in range(5):
        again = vsd.distill(z, values, ids, tail=tl, grad=True, ws=ws)
        for k in ("loss", "lse", "grad"):
            assert torch.equal(first[k], again[k])
    check_distill(z, values, ids, tl, None, 1.0, first)


@pytest.mark.parametrize("R,V,K,dtype", [(1700, 1003, 12, BF16), (1100, 17005, 20, F32), (1000, 30001, 128, BF16),
                                         (230, 60000, 64, F32), (200, 151937, 33, BF16)])
def test_distill_many_rows_per_group(spec, R, V, K, dtype):
    """Rows behind one another in the same CTAs, some of them skipped: every 37th row and the
    last ones against the oracle, twice the same bits."""
    z = rows_of(8, V, dtype, seed=V).repeat(R // 8 + 1, 1)[:R].contiguous()
    z += torch.randint(-3, 4, (R, 1), generator=torch.Generator().manual_seed(R)).cuda()   # (small whole numbers)
    top = vsd.top_logits(z + torch.tensor(0.5, dtype=dtype, device="cuda"), K)
    ids = top["ids"].clone()
    ids[::3] = (ids[::3] + 1) % V
    ids = torch.where((ids.sort(1).values.diff(dim=1) == 0).any(1, keepdim=True), top["ids"], ids)
    weight = torch.randn(R, generator=torch.Generator().manual_seed(V)).cuda()
    weight[torch.rand(R, generator=torch.Generator().manual_seed(K)) < 0.2] = 0.0
    args = dict(tail=top["tail"], weight=weight, grad=True)
    out = vsd.distill(z, top["values"], ids, **args)
    assert vsd.device_status(out["ws"]) == 0
    at = torch.cat([torch.arange(0, R, 37), torch.arange(R - 4, R)]).cuda()
    check_distill(z[at], top["values"][at], ids[at], top["tail"][at], weight[at], 1.0,
                  {k: out[k][at] for k in ("loss", "lse", "grad")})
    first = {k: out[k].clone() for k in ("loss", "lse", "grad")}
    again = vsd.distill(z, top["values"], ids, ws=out["ws"], out=out, **args)
    for k in first:
        assert torch.equal(first[k], again[k])


def test_distill_refusals(spec):
    z = rows_of(2, 100, F32, seed=1)
    values, ids = torch.zeros((2, 3), device="cuda"), torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    with pytest.raises(ValueError):
        vsd.distill(z, values[:1], ids)
    with pytest.raises(ValueError):
        vsd.distill(z, values, ids.long())
    with pytest.raises(ValueError):
        vsd.distill(z, values, ids, tail=torch.zeros(3, device="cuda"))
    with pytest.raises(TypeError):
        vsd.distill(z, values.half(), ids)
    with pytest.raises(vsd.SpecError):
        vsd.distill(z, values, ids, temperature=-1.0)
    with pytest.raises(ValueError):
        vsd.distill(z, values, ids, grad=True, out=dict(loss=torch.empty(2, device="cuda"), lse=None, grad=z.bfloat16()))


def test_offsets_past_32_bits(spec):
    R, V, K = 8700, 248320, 4                # 2.16e9 entries
    z = torch.zeros((R, V), dtype=BF16, device="cuda")
    at = torch.arange(R, device="cuda") * 28
    z[torch.arange(R, device="cuda"), at] = 8.0
    top = vsd.top_logits(z, K)
    assert torch.equal(top["ids"][:, 0].long(), at) and (top["values"][:, 0] == 8).all()
    assert (top["values"][:, 1:] == 0).all() and (top["ids"][2:, 1] == 0).all()
    ids = torch.stack([at, at + 1], 1).to(torch.int32)
    out = vsd.distill(z, torch.zeros((R, 2), device="cuda"), ids, grad=True,
                      out=dict(loss=torch.empty(R, device="cuda"), lse=torch.empty(R, device="cuda"), grad=z))
    Z = np.exp(8.0) + V - 1
    loss = 0.5 * (np.log(0.5 / (np.exp(8.0) / Z)) + np.log(0.5 * Z))
    assert (out["loss"] - loss).abs().max() < 1e-4
    g = torch.stack([z[torch.arange(R, device="cuda"), at], z[torch.arange(R, device="cuda"), at + 1]], 1).double()
    want = torch.tensor([np.exp(8.0) / Z - 0.5, 1 / Z - 0.5], dtype=torch.float64, device="cuda")
    assert (g - want).abs().max() <= 2.0 ** -8 * 0.5
    assert (z[-1].double().sum() - 0.0).abs() < 0.01


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_streams_and_graphs(spec, dtype):
    """The three calls on a side stream and replayed from a graph give what they give alone."""
    z = rows_of(6, 5001, dtype, seed=51).view(2, 3, 5001)
    hist = torch.randint(0, 5001, (2, 50), dtype=torch.int32, device="cuda")
    freq = torch.full((2,), 0.5, device="cuda")
    plain = vsd.process_logits(z, history=hist, frequency=freq)["logits"]
    top = vsd.top_logits(plain, 16)
    alone = vsd.distill(z, top["values"], top["ids"], tail=top["tail"], grad=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a = vsd.process_logits(z, history=hist, frequency=freq, stream=s)
    b = vsd.top_logits(a["logits"], 16, stream=s)
    c = vsd.distill(z, b["values"], b["ids"], tail=b["tail"], grad=True, stream=s)
    s.synchronize()
    assert torch.equal(a["logits"], plain)
    for k in ("loss", "lse", "grad"):
        assert torch.equal(c[k], alone[k])
    x = z.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        vsd.process_logits(x, history=hist, frequency=freq, ws=a["ws"], out=a)
        vsd.top_logits(a["logits"], 16, ws=b["ws"], out=b)
        vsd.distill(x, b["values"], b["ids"], tail=b["tail"], grad=True, ws=c["ws"], out=c)
    x.copy_(rows_of(6, 5001, dtype, seed=52).view(2, 3, 5001))
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    p2 = vsd.process_logits(x, history=hist, frequency=freq)["logits"]
    t2 = vsd.top_logits(p2, 16)
    d2 = vsd.distill(x, t2["values"], t2["ids"], tail=t2["tail"], grad=True)
    assert torch.equal(a["logits"], p2) and torch.equal(b["ids"], t2["ids"])
    for k in ("loss", "lse", "grad"):
        assert torch.equal(c[k], d2[k])
