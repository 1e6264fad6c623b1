"""Argument checks of policy_loss, markov_grad and adamw that need no GPU: every call carries an
invalid argument, so it returns before its first CUDA call."""

import ctypes

import pytest

import verify_spec_draft_gb300 as vsd
from verify_spec_draft_gb300 import build

A = 0x10000          # a 16-byte aligned fake device address
MIS = 0x10008        # misaligned
OK, INVALID, SHAPE, DTYPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4, 9
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if build.needs_build():
        build.build()
    return vsd.load()


def test_workspace_bytes(lib):
    wb = lib.spec_workspace_bytes
    assert wb(vsd.OP_POLICY_LOSS, 1 << 24, 1, 1 << 20, 0) > 0
    assert wb(vsd.OP_POLICY_LOSS, (1 << 24) + 1, 1, 8, 0) == 0 and wb(vsd.OP_POLICY_LOSS, 0, 1, 8, 0) == 0
    assert wb(vsd.OP_POLICY_LOSS, 1, 1, (1 << 20) + 1, 0) == 0
    assert wb(vsd.OP_MARKOV_GRAD, 256, 7, 248320, 256) > 0
    for B, G, V, r in ((0, 7, 100, 8), (1, 0, 100, 8), (1, 65, 100, 8), (1, 7, 0, 8), (1, 7, (1 << 20) + 1, 8),
                       (1, 7, 100, 0), (1, 7, 100, 257), (1 << 16, 2, 100, 8)):
        assert wb(vsd.OP_MARKOV_GRAD, B, G, V, r) == 0
    assert wb(vsd.OP_ADAMW, 1 << 16, 1, 1, 0) > 0 and wb(vsd.OP_ADAMW, (1 << 16) + 1, 1, 1, 0) == 0


def test_policy_loss_argument_errors(lib):
    def call(z=A, dt=vsd.BF16, rows=4, V=100, ld=100, tok=A, old=A, adv=A, ref=A, w=0, t=1.0, lo=0.2, hi=0.2, kl=0.1,
             loss=A, logp=A, grad=A, ws=A, wsb=1 << 20):
        return lib.spec_policy_loss(z, dt, rows, V, ld, tok, old, adv, ref, w, t, lo, hi, kl, loss, logp, grad, ws, wsb,
                                    None)
    assert call(dt=2) == DTYPE
    assert call(rows=0) == SHAPE and call(rows=(1 << 24) + 1) == SHAPE
    assert call(V=0, ld=0) == SHAPE and call(V=(1 << 20) + 1, ld=1 << 21) == SHAPE and call(ld=99) == SHAPE
    for t in (0.0, -1.0, INF, NAN, 1e-39):
        assert call(t=t) == INVALID
    for bad in (dict(lo=-0.1), dict(lo=1.1), dict(lo=NAN), dict(hi=-0.1), dict(hi=INF), dict(hi=NAN), dict(kl=-1.0),
                dict(kl=INF), dict(kl=NAN), dict(ref=0), dict(z=0), dict(tok=0), dict(old=0), dict(adv=0), dict(loss=0),
                dict(logp=0)):
        assert call(**bad) == INVALID, bad
    assert call(z=MIS) == ALIGN and call(grad=MIS) == ALIGN and call(ws=MIS) == ALIGN
    assert call(ws=0) == WORKSPACE and call(wsb=100) == WORKSPACE


def test_markov_grad_argument_errors(lib):
    def call(g=A, gdt=vsd.BF16, B=2, G=4, V=100, ld=100, anc=A, tok=A, U=A, Wt=A, wdt=vsd.BF16, r=8, dU=2 * A, dW=3 * A,
             odt=vsd.F32, ws=A, wsb=1 << 30):
        return lib.spec_markov_grad(g, gdt, B, G, V, ld, anc, tok, U, Wt, wdt, r, dU, dW, odt, ws, wsb, None)
    assert call(gdt=2) == DTYPE and call(wdt=-1) == DTYPE and call(odt=7) == DTYPE
    for bad in (dict(B=0), dict(G=0), dict(G=65), dict(B=1 << 15), dict(V=0, ld=0), dict(V=(1 << 20) + 1, ld=1 << 21),
                dict(ld=99), dict(r=0), dict(r=257)):
        assert call(**bad) == SHAPE, bad
    for name in ("g", "anc", "tok", "U", "Wt", "dU", "dW"):
        assert call(**{name: 0}) == INVALID, name
    for bad in (dict(dU=A), dict(dW=A), dict(dU=3 * A), dict(U=2 * A), dict(Wt=2 * A), dict(Wt=3 * A), dict(g=3 * A)):
        assert call(**bad) == INVALID, bad          # an output that is an input, or the other output
    for name in ("g", "U", "Wt", "dU", "dW", "ws"):
        assert call(**{name: MIS}) == ALIGN, name
    need = lib.spec_workspace_bytes(vsd.OP_MARKOV_GRAD, 2, 4, 100, 8)
    assert call(ws=0) == WORKSPACE and call(wsb=need - 1) == WORKSPACE


def test_adamw_argument_errors(lib):
    def entry(**kw):
        return vsd.AdamwTensor(**{**dict(param=A, master=0, grad=A, m=A, v=A, m_scale=0, v_scale=0, n=10, param_dtype=0,
                                         grad_dtype=0, state_bits=32), **kw})

    def call(t=None, n=1, step=A, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.01, gs=0, ws=A, wsb=1 << 20):
        t = entry() if t is None else t
        return lib.spec_adamw(ctypes.byref(t) if t else None, n, step, lr, b1, b2, eps, wd, gs, 0, ws, wsb, None)
    assert call(n=-1) == SHAPE and call(n=(1 << 16) + 1) == SHAPE
    assert call(step=0) == INVALID and call(t=0) == INVALID
    for bad in (dict(lr=-1.0), dict(lr=NAN), dict(lr=INF), dict(b1=1.0), dict(b1=-0.1), dict(b1=NAN), dict(b2=1.0),
                dict(b2=-0.1), dict(eps=0.0), dict(eps=1e-40), dict(eps=INF), dict(wd=-0.1), dict(wd=INF), dict(wd=NAN)):
        assert call(**bad) == INVALID, bad
    assert call(step=A + 2) == ALIGN and call(gs=A + 1) == ALIGN and call(ws=MIS) == ALIGN
    for kw in (dict(param_dtype=2), dict(grad_dtype=-1), dict(state_bits=16)):
        assert call(entry(**kw)) == DTYPE, kw
    assert call(entry(n=-1)) == SHAPE and call(entry(n=1 << 40)) == SHAPE
    for kw in (dict(param=0), dict(grad=0), dict(m=0), dict(v=0), dict(master=A), dict(param_dtype=1), dict(m_scale=A),
               dict(state_bits=8), dict(state_bits=8, m_scale=A), dict(state_bits=8, v_scale=A)):
        assert call(entry(**kw)) == INVALID, kw
    for kw in (dict(param=A + 2), dict(grad=A + 2), dict(m=A + 1), dict(v=A + 2), dict(param=A + 1, param_dtype=1, master=A),
               dict(param_dtype=1, master=A + 2), dict(grad=A + 1, grad_dtype=1),
               dict(state_bits=8, m_scale=A + 2, v_scale=A)):
        assert call(entry(**kw)) == ALIGN, kw
    assert call(ws=0) == WORKSPACE and call(wsb=100) == WORKSPACE


def test_the_table_entry_is_the_headers_struct():
    assert ctypes.sizeof(vsd.AdamwTensor) == 80
    assert [getattr(vsd.AdamwTensor, k).offset for k in ("param", "v_scale", "n", "param_dtype", "state_bits")] == [0, 48, 56, 64, 72]


def test_binding_refuses(lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 3, 8))
    with pytest.raises(ValueError, match="CUDA tensor"):
        vsd.policy_loss(x, x, x, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        vsd.markov_grad(x, x, x, x, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        vsd.adamw_table([x], [x], [vsd.adamw_state(x)])
    with pytest.raises(ValueError, match="empty"):
        vsd.adamw_table([], [], [])
    with pytest.raises(ValueError):
        vsd.adamw_table([x], [], [])
    with pytest.raises(ValueError, match="32 or 8"):
        vsd.adamw_state(x, bits=4)
    with pytest.raises(ValueError, match="master"):
        vsd.adamw_state(x, master=x)
    with pytest.raises(TypeError):
        vsd.adamw_state(x.double())
    s = vsd.adamw_state(torch.zeros(300, dtype=torch.bfloat16), bits=8)
    assert s["m"].dtype == torch.float8_e4m3fn and s["v_scale"].shape == (3,) and s["master"].dtype == torch.float32


@pytest.mark.parametrize("spans, clash", [
    ([(100, 10, True, "a"), (110, 10, True, "b"), (90, 10, False, "c")], None),
    ([(100, 10, False, "a"), (100, 10, False, "b"), (105, 20, False, "c")], None),     # gradients are only read
    ([(100, 0, True, "a"), (100, 10, True, "b"), (0, 0, True, "c"), (0, 0, True, "d")], None),
    ([(100, 10, True, "a"), (100, 10, True, "b")], "b overlaps a"),
    ([(100, 10, True, "a"), (100, 10, False, "b")], "b overlaps a"),
    ([(100, 10, False, "a"), (100, 10, True, "b")], "b overlaps a"),
    ([(100, 50, True, "a"), (110, 5, False, "b"), (140, 1, True, "c")], "b overlaps a"),
    ([(100, 50, True, "a"), (150, 5, True, "b"), (140, 1, True, "c")], "c overlaps a"),
    ([(100, 50, False, "a"), (110, 5, False, "b"), (149, 9, True, "c")], "c overlaps a"),
])
def test_a_table_uses_no_memory_twice(spans, clash):
    if clash is None:
        return vsd._distinct(spans)
    with pytest.raises(ValueError, match=clash):
        vsd._distinct(spans)
