"""spec_process_logits on the GPU against the float64 oracle.

Bar per entry: float32 does at most 8 roundings (two of the reciprocals, one product, the
penalty's fma and its subtraction, the bias, the temperature), each at most 2^-24 of the
largest magnitude on the way, (|l| max(rho, 1/rho) + |penalty| + |bias|) / T; a bf16 result
rounds once more, by at most 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

import verify_spec_draft_gb300 as vsd
from oracle import process as op

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def make(B, R, V, L, dtype, seed, nb=0, mask=None, ld=None):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.rand(s, generator=g)     # noqa: E731
    d = dict()
    logits = torch.zeros((B, R, ld or V), dtype=dtype)[..., :V]
    logits.copy_(torch.randn((B, R, V), generator=g) * 4)
    d["logits"] = logits
    tok = lambda *s: (V ** rnd(*s) - 1).to(torch.int32).clamp(0, V - 1)      # noqa: E731
    if L:
        d["history"] = tok(B, L)
        d["lengths"] = (rnd(B) * (L + 1)).to(torch.int32).clamp(0, L)
        d["lengths"][-1] = L
        d["prompt_lengths"] = (rnd(B) * (d["lengths"] + 1)).to(torch.int32).clamp(min=0).minimum(d["lengths"])
    if R > 1:
        d["block"] = tok(B, R - 1)
    d["repetition"] = 0.7 + 0.8 * rnd(B)
    d["frequency"] = rnd(B) - 0.3
    d["presence"] = rnd(B) - 0.5
    d["temperature"] = 0.4 + 1.5 * rnd(B)
    if nb:
        d["bias_ids"] = torch.randint(-1, V, (B, nb), generator=g, dtype=torch.int32)
        d["bias_values"] = 5 * torch.randn((B, nb), generator=g)
    if mask:
        W = (V + 31) // 32
        shape = (B, R, W) if mask == "rows" else (B, W)
        d["mask"] = torch.randint(-2**31, 2**31, shape, generator=g, dtype=torch.int64).to(torch.int32)
        d["mask"].view(-1, W)[0] = 0            # a row that allows nothing
    return d


def cuda(d):
    out = {}
    for k, t in d.items():
        if k == "logits" and t.stride(1) != t.shape[2] and t.shape[1] > 1:   # keep the row stride
            full = torch.zeros((*t.shape[:-1], t.stride(1)), dtype=t.dtype, device="cuda")
            out[k] = full[..., :t.shape[2]]
            out[k].copy_(t)
        else:
            out[k] = t.cuda()
    return out


def expect(d):
    n = {k: (t.double().numpy() if t.is_floating_point() else t.numpy()) for k, t in d.items()}
    ref = op.process_logits(**n)
    B = ref.shape[0]
    rep, temp = n["repetition"].reshape(B, 1, 1), n["temperature"].reshape(B, 1, 1)
    most = 70 + (n["history"].shape[1] if "history" in n else 0)
    pen = np.abs(n["frequency"]).reshape(B, 1, 1) * most + np.abs(n["presence"]).reshape(B, 1, 1)
    bias = np.abs(n["bias_values"]).max() if "bias_values" in n else 0.0
    big = (np.abs(n["logits"]) * np.maximum(rep, 1 / rep) + pen + bias) / temp
    tol = 8 * 2.0 ** -24 * big
    if d["logits"].dtype == BF16:
        tol = tol + 2.0 ** -8 * np.where(np.isfinite(ref), np.abs(ref), 0)
    return ref, tol


def check(got, ref, tol):
    got = got.double().cpu().numpy()
    fin = np.isfinite(ref)
    assert (got[~fin] == ref[~fin]).all()
    assert np.isfinite(got[fin]).all()
    assert (np.abs(got[fin] - ref[fin]) <= tol[fin]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,R,V,L,nb,mask", [
    (1, 1, 1, 3, 1, "rows"), (2, 3, 7, 5, 2, "rows"), (1, 2, 31, 40, 0, None), (3, 1, 33, 0, 4, "request"),
    (2, 5, 1000, 100, 10, "rows"), (1, 4, 8191, 300, 3, "rows"), (2, 2, 8192, 64, 0, "request"),
    (1, 3, 8200, 2000, 2047, None), (3, 8, 20001, 777, 40, "rows"), (1, 65, 1030, 50, 1, "rows"),
    (70, 2, 517, 9, 2, "rows")])
def test_against_oracle(spec, dtype, B, R, V, L, nb, mask):
    d = make(B, R, V, L, dtype, seed=B + R + V + L, nb=nb, mask=mask)
    ref, tol = expect(d)
    c = cuda(d)
    out = vsd.process_logits(**c)
    check(out["logits"], ref, tol)
    assert vsd.device_status(out["ws"]) == 0
    # the rows themselves are not touched, and a second call gives the same bits
    assert torch.equal(c["logits"].cpu(), d["logits"])
    again = vsd.process_logits(**c, ws=out["ws"])["logits"]
    assert torch.equal(again.view(torch.int16 if dtype == BF16 else torch.int32),
                       out["logits"].view(torch.int16 if dtype == BF16 else torch.int32))


@pytest.mark.parametrize("dtype,V,ld", [(F32, 1001, 1003), (BF16, 1001, 1009), (BF16, 1000, 1024), (F32, 50, 64)])
def test_row_stride(spec, dtype, V, ld):
    d = make(3, 4, V, 60, dtype, seed=5, nb=3, mask="rows", ld=ld)
    ref, tol = expect(d)
    c = cuda(d)
    assert c["logits"].stride(1) == ld
    out = torch.full((3, 4, ld), 7.0, dtype=dtype, device="cuda")
    vsd.process_logits(**c, out=dict(logits=out[..., :V]))
    check(out[..., :V], ref, tol)
    assert (out[..., V:] == 7.0).all()      # between the rows nothing is written
    made = vsd.process_logits(**c)["logits"]
    assert made.stride(1) == ld
    assert torch.equal(made, out[..., :V])


@pytest.mark.parametrize("dtype,V", [(F32, 20001), (BF16, 4096)])
def test_in_place(spec, dtype, V):
    d = make(2, 4, V, 100, dtype, seed=6, nb=3, mask="rows")
    ref, tol = expect(d)
    c = cuda(d)
    r = vsd.process_logits(**c, out=dict(logits=c["logits"]))
    assert r["logits"] is c["logits"]
    check(c["logits"], ref, tol)


def test_nothing_asked_copies(spec):
    x = torch.randn((2, 3, 1001), device="cuda")
    x[0, 1, 5] = -torch.inf
    assert torch.equal(vsd.process_logits(x)["logits"], x)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_special_values(spec, dtype):
    V, low = 100, torch.finfo(dtype).min
    x = torch.randn((1, 2, V)).to(dtype)
    x[0, 0, :4] = torch.tensor([float("nan"), float("inf"), float("-inf"), low])
    x[0, 1, :4] = torch.tensor([float("nan"), float("inf"), float("-inf"), low])
    mask = torch.full((1, 2, 4), -1, dtype=torch.int32)
    mask[0, 1, 0] = -16                     # the second row masks them
    hist = torch.tensor([[2, 3, 50]], dtype=torch.int32)
    r = vsd.process_logits(x.cuda(), history=hist.cuda(), repetition=torch.tensor([1.5]).cuda(), mask=mask.cuda())
    y = r["logits"].cpu()
    assert torch.isnan(y[0, 0, 0]) and y[0, 0, 1] == torch.inf and y[0, 0, 2] == -torch.inf
    assert y[0, 0, 3] == torch.tensor(low, dtype=torch.float32).mul(1.5).to(dtype)
    assert (y[0, 1, :4] == -torch.inf).all() and torch.isfinite(y[0, 1, 4:]).all()


def test_bad_tokens_and_parameters(spec):
    B, V = 4, 64
    x = torch.randn((B, 2, V), device="cuda")
    hist = torch.tensor([[1, -1, 3], [1, V, 3], [1, 2, 3], [1, 2, 3]], dtype=torch.int32, device="cuda")
    freq = torch.full((B,), 1.0, device="cuda")
    r = vsd.process_logits(x, history=hist, frequency=freq)
    assert vsd.device_status(r["ws"]) == vsd.DEV_TOKEN
    want = x.clone()
    for b, toks in enumerate([[1, 3], [1, 3], [1, 2, 3], [1, 2, 3]]):
        want[b][:, toks] -= 1.0
    assert torch.equal(r["logits"], want)   # a bad token counts for nothing
    for lengths in ([4, 3, 3, 3], [3, -1, 3, 3]):
        r = vsd.process_logits(x, history=hist.clamp(0, 3), lengths=torch.tensor(lengths, dtype=torch.int32).cuda())
        assert vsd.device_status(r["ws"]) == vsd.DEV_TOKEN
    r = vsd.process_logits(x, block=torch.full((B, 1), V, dtype=torch.int32, device="cuda"))
    assert vsd.device_status(r["ws"]) == vsd.DEV_TOKEN and torch.equal(r["logits"], x)
    r = vsd.process_logits(x, bias_ids=torch.full((B, 1), -2, dtype=torch.int32, device="cuda"),
                           bias_values=torch.ones((B, 1), device="cuda"))
    assert vsd.device_status(r["ws"]) == vsd.DEV_TOKEN and torch.equal(r["logits"], x)
    for name, bad in (("repetition", 0.0), ("repetition", float("nan")), ("temperature", -1.0),
                      ("temperature", float("inf")), ("frequency", float("inf")), ("presence", float("nan"))):
        v = torch.ones(B, device="cuda")
        v[2] = bad
        r = vsd.process_logits(x, **{name: v})
        assert vsd.device_status(r["ws"]) == vsd.DEV_NONFINITE
        assert torch.isnan(r["logits"][2]).all() and torch.isfinite(r["logits"][[0, 1, 3]]).all()


def test_last_bias_slot_wins(spec):
    x = torch.zeros((1, 1, 10), device="cuda")
    ids = torch.tensor([[4, 4, -1, 4, 2]], dtype=torch.int32, device="cuda")
    val = torch.tensor([[1.0, 2.0, 9.0, 3.0, 5.0]], device="cuda")
    y = vsd.process_logits(x, bias_ids=ids, bias_values=val)["logits"][0, 0].tolist()
    assert y == [0, 0, 5, 0, 3, 0, 0, 0, 0, 0]


def test_long_history_of_one_token(spec):
    L = 1 << 19                              # the longest history there is
    x = torch.zeros((1, 2, 40), device="cuda")
    hist = torch.full((1, L), 7, dtype=torch.int32, device="cuda")
    y = vsd.process_logits(x, history=hist, prompt_lengths=torch.tensor([10], dtype=torch.int32).cuda(),
                           block=torch.tensor([[7]], dtype=torch.int32).cuda(),
                           frequency=torch.tensor([1.0]).cuda())["logits"]
    assert y[0, 0, 7] == -(L - 10) and y[0, 1, 7] == -(L - 9) and y.sum() == -(2 * L - 19)


def test_offsets_past_32_bits(spec):
    B, R, V = 135, 65, 248320                # 2.18e9 entries
    x = torch.zeros((B, R, V), dtype=BF16, device="cuda")
    block = torch.arange(B * (R - 1), dtype=torch.int32, device="cuda").view(B, R - 1)
    y = vsd.process_logits(x, block=block, presence=torch.full((B,), 2.0, device="cuda"),
                           out=dict(logits=x))["logits"]
    assert (y[-1, -1].nonzero()[:, 0] == block[-1].sort().values).all()
    assert (y[-1, -1, block[-1].long()] == -2).all() and (y[:, 0] == 0).all()


def test_refusals(spec):
    x = torch.zeros((2, 3, 40), device="cuda")
    i = torch.int32
    with pytest.raises(ValueError):
        vsd.process_logits(x[0])                                       # not [B, R, V]
    with pytest.raises(TypeError):
        vsd.process_logits(x.half())
    with pytest.raises(ValueError):
        vsd.process_logits(x.transpose(1, 2))
    with pytest.raises(ValueError):
        vsd.process_logits(x, history=torch.zeros((3, 4), dtype=i, device="cuda"))
    with pytest.raises(ValueError):
        vsd.process_logits(x, history=torch.zeros((2, 4), device="cuda"))
    with pytest.raises(ValueError):
        vsd.process_logits(x, block=torch.zeros((2, 3), dtype=i, device="cuda"))
    with pytest.raises(ValueError):
        vsd.process_logits(x, mask=torch.zeros((2, 3, 1), dtype=i, device="cuda"))
    with pytest.raises(ValueError):
        vsd.process_logits(x, bias_ids=torch.zeros((2, 1), dtype=i, device="cuda"))
    with pytest.raises(ValueError):
        vsd.process_logits(x, out=dict(logits=torch.zeros((2, 3, 41), device="cuda")))
    with pytest.raises(vsd.SpecError):
        vsd.process_logits(torch.zeros((2, 66, 8), device="cuda"))
