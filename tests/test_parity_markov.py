"""markov_grad against the float64 oracle (one GB300)."""

import numpy as np
import pytest
import torch

import verify_spec_draft_gb300 as vsd
from oracle import markov as om

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def inputs(B, G, V, r, gdt, wdt, seed=0, pad=0, same=False):
    rng = np.random.default_rng(seed)
    dz = torch.from_numpy((rng.normal(size=(B, G, V)) * np.exp(rng.normal(size=(B, G, V)))).astype(np.float32)).to(gdt)
    if pad:
        room = torch.full((B, G, V + pad), 3.0, dtype=gdt)
        room[..., :V] = dz
        dz = room[..., :V]
    U, Wt = (torch.from_numpy(rng.normal(size=(V, r)).astype(np.float32)).to(wdt) for _ in range(2))
    x = np.minimum((V ** rng.random((B, G + 1))).astype(np.int32) - 1, V - 1)
    if same:
        x[:] = V // 2
    ends = rng.integers(1, 3 * G + 2, (B, 1))
    ends[0] = G + 1
    x = np.where(np.arange(G + 1)[None] < ends, x, -1).astype(np.int32)
    return dz, torch.from_numpy(x[:, 0].copy()), torch.from_numpy(x[:, 1:].copy()), U, Wt


def on_gpu(dz, *rest):
    """dz with its row stride kept"""
    if dz.is_contiguous():
        return (dz.cuda(), *(t.cuda() for t in rest))
    B, G, V = dz.shape
    ld = dz.stride(-2)
    room = torch.full((B, G, ld), float("nan"), dtype=dz.dtype, device="cuda")
    room[..., :V] = dz.cuda()
    return (room[..., :V], *(t.cuda() for t in rest))


def check(got, want, n, V, out):
    """Bars in roundings e = 2^-24 of the sums of magnitudes.  dWt sums n products: n + 16 at most, the 16
    for what a tensor core drops within a step.  dU sums V products in parts and then the rows: with 8 parts
    or steps of 16 that lose two roundings each, V / 8 + 64 at most.  The output's rounding is half a step."""
    e = 2.0 ** -24
    half = 2.0 ** -8 if out == BF16 else e
    tiny = 2.0 ** -134 if out == BF16 else 0.0
    for k, terms in (("Wt", n + 16), ("U", V / 8 + 64 + n / 8)):
        g, w = got[k].double().cpu().numpy(), want[k]
        assert g.shape == w.shape
        bar = terms * e * want[k + "_abs"] * (1 + half) + half * np.abs(w) + tiny
        assert (np.abs(g - w) <= bar).all(), (k, np.abs(g - w).max(), (np.abs(g - w) / np.maximum(bar, 1e-300)).max())


@pytest.mark.parametrize("gdt,wdt,out", [(F32, F32, F32), (BF16, BF16, BF16), (BF16, BF16, F32), (F32, BF16, BF16),
                                         (BF16, F32, F32)])
@pytest.mark.parametrize("B,G,V,r", [(1, 1, 1, 1), (1, 1, 5, 3), (2, 3, 130, 8), (3, 7, 1000, 64), (1, 7, 2048, 256),
                                     (20, 7, 515, 128), (5, 64, 333, 17), (40, 5, 1024, 192)])
def test_sizes_and_types(spec, B, G, V, r, gdt, wdt, out):
    a = inputs(B, G, V, r, gdt, wdt, seed=B * 100 + r)
    got = vsd.markov_grad(*on_gpu(*a), dtype=out)
    want = om.markov_grad(*(t.double().numpy() if t.is_floating_point() else t.numpy() for t in a))
    check(got, want, B * G, V, out)
    assert got["U"].dtype == out and vsd.device_status(got["ws"]) == 0
    untouched = torch.ones(V, dtype=torch.bool)
    prev = torch.cat([a[1][:, None], a[2][:, :-1]], 1).reshape(-1).long()
    untouched[prev[prev >= 0]] = False
    assert (got["U"].cpu()[untouched] == 0).all()
    # the same call again, with outputs and workspace given, bit for bit
    again = vsd.markov_grad(*on_gpu(*a), ws=got["ws"], out={k: torch.full_like(got[k], 5.0) for k in ("U", "Wt")})
    assert torch.equal(again["U"], got["U"]) and torch.equal(again["Wt"], got["Wt"])


@pytest.mark.parametrize("V,pad,r", [(1000, 8, 64), (1000, 1, 64), (1001, 0, 128), (1001, 7, 64), (50257, 0, 64),
                                     (4096, 3, 256)])
def test_row_strides(spec, V, pad, r):
    """Rows at any offset; what lies between them (NaN here) is not read into anything."""
    a = inputs(4, 7, V, r, BF16, BF16, seed=V + pad, pad=pad)
    got = vsd.markov_grad(*on_gpu(*a), dtype=F32)
    want = om.markov_grad(*(t.double().numpy() if t.is_floating_point() else t.numpy() for t in a))
    check(got, want, 28, V, F32)


@pytest.mark.parametrize("dt,r", [(F32, 20), (BF16, 64)])
def test_one_token_everywhere(spec, dt, r):
    a = inputs(30, 9, 700, r, dt, dt, seed=4, same=True)
    got = vsd.markov_grad(*on_gpu(*a), dtype=F32)
    want = om.markov_grad(*(t.double().numpy() if t.is_floating_point() else t.numpy() for t in a))
    check(got, want, 270, 700, F32)


@pytest.mark.parametrize("dt,r,V", [(F32, 20, 900), (BF16, 64, 900), (BF16, 128, 900), (BF16, 64, 904), (BF16, 192, 904),
                                    (F32, 100, 904)])
def test_rows_without_a_token(spec, dt, r, V):
    """Their dz may hold anything; tokens out of range are reported."""
    a = list(inputs(6, 5, V, r, dt, dt, seed=5))
    a[1][2] = -1
    a[2][2] = -1
    prev = torch.cat([a[1][:, None], a[2][:, :-1]], 1)
    assert (prev < 0).sum() >= 5
    a[0][prev < 0] = torch.nan
    got = vsd.markov_grad(*on_gpu(*a), dtype=F32)
    want = om.markov_grad(*(t.double().numpy() if t.is_floating_point() else t.numpy() for t in a))
    check(got, want, 30, V, F32)
    assert vsd.device_status(got["ws"]) == 0
    # the next call with this workspace, on rows that are all finite
    clean = [t.clone() for t in a]
    clean[0][prev < 0] = 1.0
    again = vsd.markov_grad(*on_gpu(*clean), dtype=F32, ws=got["ws"])
    assert torch.equal(again["U"], got["U"]) and torch.equal(again["Wt"], got["Wt"])
    a[2][0, 0] = V
    a[1][1] = -7
    a[0][0, 1] = torch.inf
    a[0][1, 0] = torch.nan
    got = vsd.markov_grad(*on_gpu(*a), dtype=F32)
    want = om.markov_grad(*(t.double().numpy() if t.is_floating_point() else t.numpy() for t in a))
    check(got, want, 30, V, F32)
    assert vsd.device_status(got["ws"]) == vsd.DEV_TOKEN


@pytest.mark.parametrize("V,r", [(1, 1), (2, 7), (7, 65), (63, 8), (64, 256), (65, 130)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_tiny_vocabularies(spec, V, r, dt):
    """Smaller than a box of the copies, with more rows than one pass takes."""
    a = inputs(4, 5, V, r, dt, dt, seed=V)
    got = vsd.markov_grad(*on_gpu(*a), dtype=F32)
    want = om.markov_grad(*(t.double().numpy() if t.is_floating_point() else t.numpy() for t in a))
    check(got, want, 20, V, F32)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_nothing_counts(spec, dt):
    a = list(inputs(3, 4, 300, 64, dt, dt, seed=6))
    a[1][:], a[2][:] = -1, -1
    got = vsd.markov_grad(*on_gpu(*a))
    assert (got["U"] == 0).all() and (got["Wt"] == 0).all() and vsd.device_status(got["ws"]) == 0


def test_gamma_one_needs_no_tokens(spec):
    a = inputs(9, 1, 600, 64, BF16, BF16, seed=7)
    g = on_gpu(*a)
    one, two = vsd.markov_grad(*g), vsd.markov_grad(g[0], g[1], None, g[3], g[4])
    assert torch.equal(one["U"], two["U"]) and torch.equal(one["Wt"], two["Wt"])


# the training batch's width; odd rows in one slice and in several; float32 in several slices; one block; many
# tiles of rows over few entries, in one round and in four
@pytest.mark.parametrize("B,G,V,r,dt", [
    (256, 7, 20000, 256, BF16), (61, 15, 31111, 192, BF16), (256, 7, 30001, 256, BF16), (100, 5, 40001, 64, F32),
    (1, 7, 248320, 256, BF16), (1300, 7, 1500, 64, BF16), (1024, 64, 300, 8, BF16)])
def test_larger(spec, B, G, V, r, dt):
    """Against float64 products on the GPU."""
    a = inputs(B, G, V, r, dt, dt, seed=8)
    g = on_gpu(*a)
    got = vsd.markov_grad(*g, dtype=F32)
    prev = torch.cat([g[1][:, None], g[2][:, :-1]], 1).reshape(-1).long()
    on = prev >= 0
    d, u, w = g[0].reshape(-1, V)[on].double(), g[3][prev[on]].double(), g[4].double()
    want = {}
    for k, f in (("", lambda t: t), ("_abs", torch.abs)):
        want["Wt" + k] = (f(d).t() @ f(u)).cpu().numpy()
        z = torch.zeros((V, r), dtype=torch.float64, device="cuda")
        want["U" + k] = z.index_add_(0, prev[on], f(d) @ f(w)).cpu().numpy()
    check(got, want, B * G, V, F32)
    assert vsd.device_status(got["ws"]) == 0


def test_rows_past_32_bits(spec):
    """2.2e9 entries of dz: the last rows, the last entries."""
    B, G, V, r = 1250, 7, 248320, 64
    dz = torch.zeros((B, G, V), dtype=BF16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    dz[B - 1] = torch.randn((G, V), generator=gen, device="cuda")
    dz[:, :, V - 3:] = 0.5
    U, Wt = (torch.randn((V, r), generator=gen, device="cuda").to(BF16) for _ in range(2))
    anchor = torch.arange(B, dtype=torch.int32, device="cuda")
    tokens = torch.full((B, G), V - 1, dtype=torch.int32, device="cuda")
    got = vsd.markov_grad(dz, anchor, tokens, U, Wt, dtype=F32)
    x = dz[B - 1, 0].double() @ Wt.double()
    bar = (V / 8 + 64) * 2.0 ** -24 * (dz[B - 1, 0].double().abs() @ Wt.double().abs())
    assert ((got["U"][B - 1].double() - x).abs() <= bar).all()
    last = dz[:, :, V - 1].double().reshape(-1)
    rows = U[torch.cat([anchor[:, None], tokens[:, :-1]], 1).reshape(-1).long()].double()
    bar = (B * G + 16) * 2.0 ** -24 * (last.abs() @ rows.abs())
    assert ((got["Wt"][V - 1].double() - last @ rows).abs() <= bar).all()
    assert vsd.device_status(got["ws"]) == 0


def test_refusals(spec):
    dz, anchor, tokens, U, Wt = on_gpu(*inputs(3, 4, 100, 8, F32, F32))
    for bad in ((dz[0], anchor, tokens, U, Wt), (dz, anchor, None, U, Wt), (dz, anchor, tokens[:, :3], U, Wt),
                (dz, anchor.long(), tokens, U, Wt), (dz, anchor, tokens, U[:99], Wt[:99]), (dz, anchor, tokens, U, Wt[:, :4]),
                (dz, anchor, tokens, U, Wt.to(BF16)), (dz, anchor, tokens, U, None), (dz, anchor.cpu(), tokens, U, Wt)):
        with pytest.raises(ValueError):
            vsd.markov_grad(*bad)
    with pytest.raises(TypeError):
        vsd.markov_grad(dz, anchor, tokens, U.half(), Wt.half())
    with pytest.raises(TypeError):
        vsd.markov_grad(dz, anchor, tokens, U, Wt, dtype=torch.float16)
    with pytest.raises(ValueError):
        vsd.markov_grad(dz, anchor, tokens, U, Wt, out=dict(U=torch.empty_like(U)))
    with pytest.raises(ValueError):
        vsd.markov_grad(dz, anchor, tokens, U, Wt, out=dict(U=torch.empty_like(U), Wt=torch.empty_like(Wt).to(BF16)))
    with pytest.raises(vsd.SpecError):
        need = vsd.workspace_bytes(vsd.OP_MARKOV_GRAD, 3, 4, 100, 8)
        vsd.markov_grad(dz, anchor, tokens, U, Wt, ws=torch.zeros(need - 1, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("gdt,wdt,out", [(F32, F32, F32), (BF16, BF16, BF16), (BF16, F32, F32)])
@pytest.mark.parametrize("V,r", [(40000, 32), (39041, 31), (5003, 256), (20011, 250), (78000, 12), (45000, 28), (39000, 16),
                                 (40001, 2)])
def test_a_few_rows_many_turns(spec, V, r, gdt, wdt, out):
    """Every CTA takes more than one turn, of 1 to 4 entries a thread; one row's dz is not finite and does not
    count.  A thread adds V / 608 terms at most, a CTA 128 threads' and the join 304 CTAs' sums: fewer than the
    roundings that check counts."""
    a = list(inputs(2, 4, V, r, gdt, wdt, seed=V))
    a[2][1, 1] = -1
    a[0][1, 2] = torch.nan
    got = vsd.markov_grad(*on_gpu(*a), dtype=out)
    want = om.markov_grad(*(t.double().numpy() if t.is_floating_point() else t.numpy() for t in a))
    check(got, want, 8, V, out)
    assert vsd.device_status(got["ws"]) == 0


@pytest.mark.parametrize("B,G,V,r,dt", [(140, 64, 500, 8, BF16), (9001, 1, 90, 40, F32), (163, 63, 2000, 130, BF16)])
def test_many_rows(spec, B, G, V, r, dt):
    """More rows than are ordered by counting: tokens that come back in many blocks, rows without one and
    tokens out of range."""
    a = list(inputs(B, G, V, r, dt, dt, seed=B))
    a[1][3], a[1][7] = -1, V
    a[1][B // 2:B // 2 + 50] = 17
    got = vsd.markov_grad(*on_gpu(*a), dtype=F32)
    want = om.markov_grad(*(t.double().numpy() if t.is_floating_point() else t.numpy() for t in a))
    check(got, want, B * G, V, F32)
    assert vsd.device_status(got["ws"]) == vsd.DEV_TOKEN
    again = vsd.markov_grad(*on_gpu(*a), dtype=F32)
    assert torch.equal(again["U"], got["U"]) and torch.equal(again["Wt"], got["Wt"])
