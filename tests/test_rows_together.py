"""process_logits, top_logits and distill used together, at their limits and in graphs."""

import importlib.util
import os

import pytest
import torch

import verify_spec_draft_gb300 as vsd

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_learns(spec):
    """The example's drafter ends with less loss and more accepted drafts than it began with."""
    at = importlib.util.spec_from_file_location("online_distill", os.path.join(ROOT, "examples", "online_distill.py"))
    ex = importlib.util.module_from_spec(at)
    at.loader.exec_module(ex)
    loss, accepted = ex.run(steps=25, requests=8, gamma=5, vocab=5003, k=32, report=lambda s: None)
    assert sum(loss[-5:]) < 0.7 * sum(loss[:5])
    assert sum(accepted[-5:]) > sum(accepted[:5])


def test_processed_rows_verify_as_token_by_token(spec):
    """A block's processed rows equal the rows that one-token calls give with the drafted tokens
    appended to the history."""
    g = torch.Generator().manual_seed(5)
    B, G, V, L = 3, 4, 6007, 40
    x = torch.randn((B, G + 1, V), generator=g).cuda()
    hist = torch.randint(0, V, (B, L), generator=g, dtype=torch.int32)
    block = torch.randint(0, V, (B, G), generator=g, dtype=torch.int32)
    block[1, 2], block[1, 3] = block[1, 0], hist[1, 3]
    kw = dict(repetition=torch.tensor([1.2, 0.9, 1.0]).cuda(), frequency=torch.tensor([0.3, 0.1, 0.0]).cuda(),
              presence=torch.tensor([0.2, -0.4, 1.0]).cuda(), temperature=torch.tensor([0.7, 1.0, 1.3]).cuda())
    whole = vsd.process_logits(x, history=hist.cuda(), block=block.cuda(), **kw)["logits"]
    for j in range(G + 1):
        h = torch.cat([hist, block[:, :j]], 1).contiguous().cuda()
        one = vsd.process_logits(x[:, j:j + 1].contiguous(), history=h, **kw)["logits"]
        # the sums are formed from the same counts in the same order
        assert torch.equal(one[:, 0], whole[:, j]), j


def test_a_mask_that_leaves_nothing_is_reported(spec):
    x = torch.randn((2, 4, 1000), device="cuda")
    mask = torch.full((2, 4, 32), -1, dtype=torch.int32, device="cuda")
    mask[1, 2] = 0
    y = vsd.process_logits(x, mask=mask)["logits"]
    assert (y[1, 2] == -torch.inf).all()
    v = vsd.verify(y, None, y[:, :3].argmax(-1).to(torch.int32), 0)
    assert v["n"].tolist() == [3, -1] and vsd.device_status(v["ws"]) & vsd.DEV_NONFINITE
    t = vsd.top_logits(y, 5)
    assert (t["ids"][1, 2] == -1).all() and t["lse"][1, 2] == -torch.inf
    assert vsd.device_status(t["ws"]) == vsd.DEV_NONFINITE


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_largest_vocabulary(spec, dtype):
    """V = 2^20 (and 2^26 for process_logits): the last entries and the log-sum-exp."""
    V = 1 << 20
    z = torch.zeros((2, V), dtype=dtype, device="cuda")
    z[0, V - 1], z[1, 0], z[1, V - 2] = 9.0, 3.0, 5.0
    t = vsd.top_logits(z, 128)
    assert t["ids"][0, 0] == V - 1 and t["ids"][1, :2].tolist() == [V - 2, 0]
    assert torch.equal(t["ids"][0, 1:], torch.arange(127, dtype=torch.int32, device="cuda"))
    want = torch.logsumexp(z.double(), 1)
    # 2^20 equal weights: sums of 2^8 in blocks, then at most 2^13 of them
    assert (t["lse"].double() - want).abs().max() < 1e-5
    d = vsd.distill(z, t["values"], t["ids"], tail=t["tail"], grad=True)
    assert d["loss"].abs().max() < 1e-4 and d["grad"].float().abs().max() < 1e-6
    assert (d["lse"].double() - want).abs().max() < 1e-5
    if dtype == BF16:
        V = 1 << 26
        x = torch.zeros((1, 1, V), dtype=dtype, device="cuda")
        h = torch.tensor([[0, V - 1, V - 1]], dtype=torch.int32, device="cuda")
        y = vsd.process_logits(x, history=h, frequency=torch.ones(1, device="cuda"))["logits"]
        assert y[0, 0, 0] == -1 and y[0, 0, V - 1] == -2 and y.float().sum() == -3


def test_loss_and_gradient_share_a_workspace(spec):
    g = torch.Generator().manual_seed(7)
    z = (torch.randn((60, 20001), generator=g) * 3).to(BF16).cuda()
    t = vsd.top_logits((z.float() + torch.randn(z.shape, generator=g).cuda()).to(BF16), 20)
    ws = vsd.workspace(vsd.OP_DISTILL, 60, 20, 20001)
    first = vsd.distill(z, t["values"], t["ids"], tail=t["tail"], ws=ws)
    loss = first["loss"].clone()
    for _ in range(3):
        a = vsd.distill(z, t["values"], t["ids"], tail=t["tail"], grad=True, ws=ws)
        b = vsd.distill(z, t["values"], t["ids"], tail=t["tail"], ws=ws)
        assert torch.equal(b["loss"], loss)
        # two summations of the same row: each within its bar, 2^-24 (4 max|z| + 100) and as much
        # for the teacher's, twice over
        assert ((a["loss"] - loss).abs() <= 4 * 2.0 ** -24 * (8 * 20 + 200) * (1 + loss)).all()


@pytest.mark.parametrize("V", [5000, 5001])
def test_many_rows_in_a_graph(spec, V):
    """Enough rows that the picks are a launch of their own."""
    g = torch.Generator().manual_seed(9)
    z = (torch.randn((100, V), generator=g) * 3).to(BF16).cuda()
    ws = vsd.workspace(vsd.OP_TOP_LOGITS, 100, 24, V)
    wd = vsd.workspace(vsd.OP_DISTILL, 100, 24, V)
    t = vsd.top_logits(z, 24, ws=ws)
    d = vsd.distill(z, t["values"], t["ids"], grad=True, ws=wd)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vsd.top_logits(z, 24, ws=ws, out=t)
        vsd.distill(z, t["values"], t["ids"], grad=True, ws=wd, out=d)
    z.copy_((torch.randn((100, V), generator=g) * 3).to(BF16))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    t2 = vsd.top_logits(z, 24)
    d2 = vsd.distill(z, t2["values"], t2["ids"], grad=True)
    for k in ("values", "ids", "tail", "lse"):
        assert torch.equal(t[k], t2[k])
    for k in ("loss", "lse", "grad"):
        assert torch.equal(d[k], d2[k])


def test_calls_on_two_streams(spec):
    """Calls with workspaces of their own overlap on two streams and give what they give alone."""
    g = torch.Generator().manual_seed(11)
    z = (torch.randn((20, 9001), generator=g) * 3).cuda()
    t = vsd.top_logits(z, 16)
    teacher = dict(values=t["values"], ids=t["ids"], tail=t["tail"])
    grads = vsd.distill(z, **teacher, grad=True)
    loss = vsd.distill(z, **teacher)
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    made = []
    for _ in range(10):
        made.append((vsd.distill(z, **teacher, grad=True, stream=one), vsd.top_logits(z, 16, stream=two),
                     vsd.distill(z, **teacher, stream=two)))
    torch.cuda.synchronize()
    for a, b, c in made:
        assert torch.equal(a["grad"], grads["grad"]) and torch.equal(a["loss"], grads["loss"])
        assert torch.equal(b["ids"], t["ids"]) and torch.equal(b["tail"], t["tail"])
        assert torch.equal(c["loss"], loss["loss"])
        for m in (a, b, c):
            assert vsd.device_status(m["ws"]) == 0


def test_outputs_and_workspaces_of_another_call(spec):
    """What a caller passes to be written is refused where it does not fit, before anything runs."""
    z = torch.randn((6, 1000), generator=torch.Generator().manual_seed(1)).cuda()
    top = vsd.top_logits(z, 20)
    with pytest.raises(ValueError):
        vsd.top_logits(z, 64, out=top)                                    # room for 20
    for name in ("values", "tail", "lse"):
        with pytest.raises(ValueError):
            vsd.top_logits(z, 20, out=dict(top, **{name: top[name].double()}))
    with pytest.raises(ValueError):
        vsd.top_logits(z, 20, out=dict(top, ids=top["ids"].long()))
    d = vsd.distill(z, top["values"], top["ids"], tail=top["tail"], grad=True)
    for bad in (dict(loss=d["loss"][:5]), dict(lse=d["lse"].cpu()), dict(loss=None), dict(grad=d["grad"][:, :999])):
        with pytest.raises(ValueError):
            vsd.distill(z, top["values"], top["ids"], tail=top["tail"], grad=True, out=dict(d, **bad))
    host = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError):
        vsd.top_logits(z, 20, ws=host)
    with pytest.raises(ValueError):
        vsd.distill(z, top["values"], top["ids"], ws=host)
    with pytest.raises(ValueError):
        vsd.process_logits(z.view(1, 6, 1000), ws=host)
    again = vsd.top_logits(z, 20, out=dict(values=top["values"], ids=top["ids"], tail=top["tail"], lse=None))
    assert again["lse"] is None
