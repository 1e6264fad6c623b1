"""adamw against the float64 oracle (one GB300)."""

import numpy as np
import pytest
import torch

import verify_spec_draft_gb300 as vsd
from oracle import adamw as oa

pytestmark = pytest.mark.gpu
F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
E = 2.0 ** -24
HYPER = dict(lr=2e-3, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1)


def make(n, pdt, gdt, bits, seed, offset=0):
    """Parameter, gradient and state of n entries, `offset` entries into their buffers."""
    rng = np.random.default_rng(seed)

    def t(x, dt, scale=False):
        x = np.asarray(x, dtype=np.float32)
        room = torch.full((len(x) + offset + 8,), 9.0, dtype=torch.float32).to(dt).cuda()
        room[offset:offset + len(x)] = torch.from_numpy(x).to(dt).cuda()
        return room[offset:offset + len(x)]
    p, g = rng.normal(size=n), rng.normal(size=n) * np.exp(rng.normal(size=n))
    m, r = rng.normal(size=n) * 0.3, np.exp(rng.normal(size=n)) * 0.5
    P = t(p, pdt)
    s = dict(master=t(p, F32)) if pdt == BF16 else {}
    if bits == 32:
        s.update(m=t(m, F32), v=t(r * r, F32))
    else:
        for k, x in (("m", m), ("v", r)):
            sc = oa.scales(x)
            y = x / np.repeat(sc, 128)[:n]
            s[k] = t(y, F8)
            s[k + "_scale"] = t(sc, F32)
    return P, t(g, gdt), s


def host(t):
    return t.to(F32).double().cpu().numpy() if t is not None else None


def check_step(before, after, T, index=0, seed=0, clip=1.0, lr=2e-3, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1):
    """One tensor's step.  Bars in roundings e: m and v are two products and a sum of float32 factors
    (each beta and its rest rounded once, the gradient's factor once more): 6 e of the sum of magnitudes;
    v has g twice, 8 e.  The update goes by m / (sqrt(v) root + eps): m's error over the denominator, and
    of the quotient 4 e of v's, 12 e for root, the sum, size and products, and 2^-21 for the division."""
    (P0, G, S0), (P1, S1) = before, after
    n = P0.numel()
    packed = "m_scale" in S0
    p0 = host(S0.get("master", P0))
    g = host(G) * clip
    m0, v0 = host(S0["m"]), host(S0["v"])
    if packed:
        m0 = m0 * np.repeat(host(S0["m_scale"]), 128)[:n]
        v0 = (v0 * np.repeat(host(S0["v_scale"]), 128)[:n]) ** 2
    b1, b2 = betas
    p, m, v = oa.step(p0, g, m0, v0, T, lr, b1, b2, eps, weight_decay)
    m_bar = 6 * E * (b1 * np.abs(m0) + (1 - b1) * np.abs(g))
    den = np.sqrt(v / (1 - b2 ** T)) + eps
    size = lr / (1 - b1 ** T)
    q = host(S1.get("master", P1))
    bar = 3 * E * np.abs(p0) + size * (m_bar + np.abs(m) * (16 * E + 2.0 ** -21)) / den + E * np.abs(p)
    assert (np.abs(q - p) <= bar).all(), (np.abs(q - p) / bar).max()
    if "master" in S0:
        assert torch.equal(P1, S1["master"].to(BF16))
    if not packed:
        assert (np.abs(host(S1["m"]) - m) <= m_bar).all()
        assert (np.abs(host(S1["v"]) - v) <= 8 * E * v).all()
        return 0
    near = 0
    for k, x, rnd, bar, root in (("m", m, 0, m_bar, False), ("v", np.sqrt(v), 1, 6 * E * np.sqrt(v), True)):
        random = oa.random16(seed, n, T, index)[rnd]
        got = S1[k].view(torch.uint8).cpu().numpy().astype(np.int64)
        # a block whose largest value is that near to a power of two may take either scale
        s, s_got = oa.scales(x), host(S1[k + "_scale"])
        ends = [oa.scales(np.maximum(np.abs(x) + sign * bar, 0)) for sign in (-1, 1)]
        assert ((s_got == s) | (s_got == ends[0]) | (s_got == ends[1])).all()
        code, s, margin = oa.encode(x, random, root, s_got)
        # a code may differ where the value's error takes the sum with the random number across 1: its margin,
        # and 2^-16 as the kernel keeps 16 to 20 bits of what is left over
        spacing = np.maximum(np.abs(x) / 16, np.repeat(s, 128)[:n] * 2.0 ** -9)
        loose = margin <= 2.0 ** -16 + bar / spacing
        # (values, as a value that near to 0 has either sign)
        assert ((oa.code_value(got) == oa.code_value(code)) | loose).all()
        assert (np.abs((got & 127) - (code & 127)) <= 1).all()
        near += int((oa.code_value(got) != oa.code_value(code)).sum())
    assert near <= 2 + n // 5000      # 2^-15 of the entries are that near: three times as many, and two
    return near


def step_and_check(items, T=1, seed=0, clip=None, **kw):
    kw = {**HYPER, **kw}
    before = [(p.clone(), g.clone(), {k: x.clone() for k, x in s.items()}) for p, g, s in items]
    table = vsd.adamw_table([i[0] for i in items], [i[1] for i in items], [i[2] for i in items])
    step = torch.full((1,), T - 1, dtype=torch.int32, device="cuda")
    scale = None if clip is None else torch.full((1,), clip, device="cuda")
    r = vsd.adamw(table, step, grad_scale=scale, seed=seed, **kw)
    assert int(step) == T and vsd.device_status(r["ws"]) == 0
    for i, (b, (p, g, s)) in enumerate(zip(before, items)):
        check_step(b, (p, s), T, i, seed, 1.0 if clip is None else float(np.float32(clip)), **kw)
        assert torch.equal(b[1], g)
    return table


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt,gdt", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("n", [1, 3, 4, 127, 128, 129, 1000, 2048, 5001, 70000])
def test_sizes_and_types(spec, n, pdt, gdt, bits):
    step_and_check([make(n, pdt, gdt, bits, seed=n)], T=3)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("offset", [1, 2, 4])
def test_offsets_and_neighbours(spec, bits, offset):
    """Tensors that begin anywhere in their buffers: what lies around them stays."""
    items = [make(n, pdt, BF16, bits, seed=n, offset=offset) for n, pdt in ((1001, F32), (515, BF16), (4096, BF16))]
    step_and_check(items, T=5)
    for p, g, s in items:
        for t in (p, g, *s.values()):
            room = t.as_strided((t.numel() + offset + 8,), (1,), 0).float()
            assert (room[:offset] == 9.0).all() and (room[offset + t.numel():] == 9.0).all()


@pytest.mark.parametrize("tensors", [2, 33, 450, 900])
def test_many_tensors(spec, tensors):
    """Mixed types and state sizes; tables longer than one launch takes."""
    kinds = [(F32, F32, 32), (BF16, BF16, 8), (BF16, F32, 32), (F32, BF16, 8)]
    items = [make(1 + (i * 67) % 900, *kinds[i % 4], seed=i) for i in range(tensors)]
    step_and_check(items, T=2, seed=77, clip=0.37)


@pytest.mark.parametrize("T", [1, 2, 1000, 2**31 - 1])
def test_bias_correction(spec, T):
    step_and_check([make(3000, F32, F32, 32, seed=1)], T=T, betas=(0.9, 0.999))
    step_and_check([make(3000, BF16, BF16, 8, seed=2)], T=T, seed=(5 << 40) + 9, betas=(0.0, 0.0))


def test_steps_in_a_row(spec):
    """Ten steps, each against the oracle from the state before it; fresh states."""
    g = torch.Generator().manual_seed(3)
    params = [torch.randn((37, 55), generator=g).cuda(), torch.randn((3001,), generator=g).to(BF16).cuda()]
    for bits in (32, 8):
        ps = [p.clone() for p in params]
        grads = [torch.empty_like(p) for p in ps]
        states = [vsd.adamw_state(p, bits) for p in ps]
        table = vsd.adamw_table(ps, grads, states)
        step = torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = vsd.workspace(vsd.OP_ADAMW, 2, 1, 1)
        for T in range(1, 11):
            for t in grads:
                t.copy_(torch.randn(t.shape, generator=g))
            flat = [(p.reshape(-1).clone(), t.reshape(-1).clone(), {k: x.reshape(-1).clone() for k, x in s.items()})
                    for p, t, s in zip(ps, grads, states)]
            vsd.adamw(table, step, seed=T * 7, ws=ws, **HYPER)
            for i, b in enumerate(flat):
                check_step(b, (ps[i].reshape(-1), {k: x.reshape(-1) for k, x in states[i].items()}), T, i, T * 7, **HYPER)
        assert int(step) == 10 and vsd.device_status(ws) == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_that_are_not_finite(spec, bits):
    """Their entries stay, the others move; a factor that is not finite leaves everything."""
    p, g, s = make(1000, F32, F32, bits, seed=9)
    at = [0, 130, 131, 999]
    g[at[0]], g[at[1]], g[at[2]], g[at[3]] = torch.nan, torch.inf, -torch.inf, 3e38
    p0, s0 = p.clone(), {k: x.clone() for k, x in s.items()}
    table = vsd.adamw_table([p], [g], [s])
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = vsd.adamw(table, step, **HYPER)
    assert vsd.device_status(r["ws"]) == vsd.DEV_NONFINITE and int(step) == 1
    moved = p != p0
    assert not moved[at].any() and moved.sum() == 996 and torch.isfinite(p).all()
    for k in ("m", "v"):
        assert torch.isfinite(s[k].float()).all()
        if bits == 32:
            assert torch.equal(s[k][at], s0[k][at])
        else:   # within the block's new scale: a code's spacing
            sc0, sc1 = (x[k + "_scale"][torch.tensor(at, device="cuda") // 128] for x in (s0, s))
            old, new = s0[k][at].float() * sc0, s[k][at].float() * sc1
            assert ((new - old).abs() <= torch.maximum(old.abs() / 8, sc1 * 2.0 ** -9)).all()
    p1 = p.clone()
    r = vsd.adamw(table, step, grad_scale=torch.full((1,), torch.nan, device="cuda"), **HYPER)
    assert torch.equal(p, p1) and vsd.device_status(r["ws"]) == vsd.DEV_NONFINITE


@pytest.mark.parametrize("bits", [32, 8])
def test_entries_without_a_gradient(spec, bits):
    """Rows of a table that no token touched: zero states stay zero, the weights only decay."""
    p = torch.randn((64, 100), generator=torch.Generator().manual_seed(2)).cuda()
    g = torch.zeros_like(p)
    g[3], g[40, 7] = 1.0, -1e-20
    s = vsd.adamw_state(p, bits)
    p0 = p.clone()
    vsd.adamw(vsd.adamw_table([p], [g], [s]), torch.zeros(1, dtype=torch.int32, device="cuda"), lr=0.1, weight_decay=0.5)
    rest = g == 0
    assert torch.equal(p[rest], p0[rest] * (1.0 - 0.05)) and (s["m"].float()[rest] == 0).all() and (s["v"].float()[rest] == 0).all()
    assert (p[3] < p0[3] * 0.95).all() and torch.isfinite(p).all()


def test_steps_out_of_range(spec):
    p, g, s = make(500, F32, F32, 32, seed=4)
    p0 = p.clone()
    for at in (-1, 2**31 - 1):
        step = torch.full((1,), at, dtype=torch.int32, device="cuda")
        r = vsd.adamw(vsd.adamw_table([p], [g], [s]), step, **HYPER)
        assert int(step) == at and torch.equal(p, p0) and vsd.device_status(r["ws"]) == vsd.DEV_TOKEN


def test_tensors_without_entries(spec):
    e = torch.empty((0,), device="cuda")
    p, g, s = make(300, F32, F32, 32, seed=5)
    p0 = p.clone()
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    vsd.adamw(vsd.adamw_table([e, p, e], [e, g, e], [vsd.adamw_state(e), s, vsd.adamw_state(e, 8)]), step, **HYPER)
    assert int(step) == 1 and (p != p0).all()
    vsd.adamw(vsd.adamw_table([e], [e], [vsd.adamw_state(e)]), step, **HYPER)
    assert int(step) == 2


@pytest.mark.parametrize("bits", [32, 8])
def test_entries_past_32_bits(spec, bits):
    """A tensor of 2.2e9 entries: its ends and the entries around 2^31 against a short tensor's."""
    n = (1 << 31) + 5003
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, dtype=BF16, device="cuda")
    s = vsd.adamw_state(p, bits)
    parts = [slice(0, 1024), slice((1 << 31) - 1024, (1 << 31) + 1024), slice(n - 1024 - n % 128, n)]
    gen = torch.Generator(device="cuda").manual_seed(1)
    for a in parts:
        p[a], g[a] = torch.randn(a.stop - a.start, generator=gen, device="cuda"), torch.randn(a.stop - a.start, generator=gen, device="cuda")
    before = [(p[a].clone(), g[a].clone(), {k: (x[a] if x.numel() == n else x[a.start // 128:(a.stop + 127) // 128]).clone()
                                           for k, x in s.items()}) for a in parts]
    r = vsd.adamw(vsd.adamw_table([p], [g], [s]), torch.zeros(1, dtype=torch.int32, device="cuda"), **HYPER)
    assert vsd.device_status(r["ws"]) == 0
    for a, b in zip(parts, before):
        after = (p[a], {k: (x[a] if x.numel() == n else x[a.start // 128:(a.stop + 127) // 128]) for k, x in s.items()})
        if bits == 32:
            check_step(b, after, 1, **HYPER)
        else:   # the random numbers are those of the entries' own places
            keep = oa.random16
            try:
                oa.random16 = lambda seed, m, T, tensor: keep(seed, m, T, tensor, a.start)
                check_step(b, after, 1, **HYPER)
            finally:
                oa.random16 = keep
    assert (p[2048:1 << 20] == 0).all() and (s["m"][2048:1 << 20].float() == 0).all()


def test_refusals(spec):
    p, g, s = make(300, F32, F32, 32, seed=6)
    h, hg, hs = make(300, BF16, BF16, 8, seed=6)
    for bad in (([p], [g[:299]], [s]), ([p], [g.cpu()], [s]), ([p], [g], [dict(m=s["m"])]), ([p], [g], [dict(s, m=s["m"][:5])]),
                ([p], [g], [dict(s, master=p)]), ([h], [hg], [{k: x for k, x in hs.items() if k != "master"}]),
                ([h], [hg], [dict(hs, m_scale=None)]), ([h], [hg], [dict(hs, v=s["v"])]),
                ([h], [hg], [dict(hs, v_scale=hs["v_scale"][:2])]), ([torch.zeros((4, 6), device="cuda").t()], [g], [s])):
        with pytest.raises(ValueError):
            vsd.adamw_table(*bad)
    with pytest.raises(TypeError):
        vsd.adamw_table([p.double()], [g], [s])
    table = vsd.adamw_table([p, h], [g, hg], [s, hs])
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in (None, step.cpu(), step.long(), torch.zeros(2, dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError):
            vsd.adamw(table, bad, lr=0.1)
    with pytest.raises(ValueError):
        vsd.adamw(table, step, lr=0.1, grad_scale=torch.ones(1))
    for bad in (dict(lr=-1.0), dict(lr=0.1, betas=(1.0, 0.9)), dict(lr=0.1, eps=0.0), dict(lr=0.1, weight_decay=-1.0)):
        with pytest.raises(vsd.SpecError):
            vsd.adamw(table, step, **bad)
    with pytest.raises(vsd.SpecError):
        vsd.adamw(table, step, lr=0.1, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert int(step) == 0


def test_memory_used_twice_is_refused(spec):
    p, g = torch.zeros(256, device="cuda"), torch.ones(256, device="cuda")
    state = lambda t: vsd.adamw_state(t, 8)
    for bad in (([p, p], [g, g], [state(p), state(p)]), ([p], [p], [state(p)]),
                ([p[:200], p[100:]], [g[:200], g[100:]], [state(p[:200]), state(p[100:])])):
        with pytest.raises(ValueError, match="overlaps"):
            vsd.adamw_table(*bad)
    s = state(p)
    with pytest.raises(ValueError, match="overlaps"):
        vsd.adamw_table([p, p.clone()], [g, g], [s, s])
    vsd.adamw_table([p[:100], p[100:]], [g[:100], g[:156]], [state(p[:100]), state(p[100:])])    # one gradient for two


def test_a_table_keeps_its_memory(spec):
    p = torch.zeros(1 << 20, device="cuda")
    g = torch.ones(1 << 20, device="cuda")
    table = vsd.adamw_table([p], [g], [vsd.adamw_state(p)])
    at = p.data_ptr()
    p.data = torch.full((1 << 20,), 5.0, device="cuda")
    other = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(4)]     # would take what had been freed
    assert all(o.data_ptr() != at for o in other)
    vsd.adamw(table, torch.zeros(1, dtype=torch.int32, device="cuda"), lr=0.1)
    assert (p == 5.0).all() and all((o == 7.0).all() for o in other)
