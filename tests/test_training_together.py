"""policy_loss, markov_grad and adamw as a drafter's training step uses them: behind draft_block and
verify, in a graph, on several streams and threads."""

import importlib.util
import os
import threading

import numpy as np
import pytest
import torch

import verify_spec_draft_gb300 as vsd
from oracle import markov as om, policy as op
from verify_spec_draft_gb300 import synth

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


class Step:
    """A drafter's weights, and one step of policy training on blocks that it drew."""

    def __init__(self, B=6, G=5, V=3001, r=64, bits=32, seed=0):
        self.B, self.G, self.V, self.r = B, G, V, r
        target, draft = synth.target_and_draft(B, G, V, "gaussian", 1.0, BF16, seed=seed, device="cuda")
        self.target, self.rows = target, draft
        self.U, self.Wt = (w.cuda() for w in synth.markov_weights(V, r, BF16, seed=seed, scale=0.2))
        self.anchor = synth.anchors(B, V, seed=seed).cuda()
        self.grads = [torch.empty((V, r), dtype=BF16, device="cuda") for _ in range(2)]
        self.states = [vsd.adamw_state(w, bits) for w in (self.U, self.Wt)]
        self.table = vsd.adamw_table([self.U, self.Wt], self.grads, self.states)
        self.count = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = dict(policy=vsd.workspace(vsd.OP_POLICY_LOSS, B * G, 1, V), markov=vsd.workspace(vsd.OP_MARKOV_GRAD, B, G, V, r),
                       adamw=vsd.workspace(vsd.OP_ADAMW, 2, 1, 1))
        seeds = synth.seeds_for(B, 0, "cuda")
        d = vsd.draft_block(self.rows, self.anchor, self.U, self.Wt, 1, seeds, qlogits=True)
        v = vsd.verify(self.target, d["qlogits"], d["tokens"], 1, seeds)
        self.z, self.tokens, self.old = d["qlogits"], d["tokens"], d["qtok"].log()
        # accepted drafts are good, the first rejected one is not, what follows does not count
        at = torch.arange(G, device="cuda")[None]
        n = v["n"][:, None]
        self.adv = torch.where(at < n, 1.0, -1.0).contiguous()
        self.weight = (at <= n).float() / (at <= n).sum()
        self.prev = torch.where(at[:, :G] < n, self.tokens, -1).contiguous()   # blocks end at the rejection
        self.loss = dict(loss=torch.empty((B, G), device="cuda"), logp=torch.empty((B, G), device="cuda"),
                         grad=torch.empty((B, G, V), device="cuda"))

    def biased(self):
        """The rows with the bias of the present weights, for the tokens that were drawn."""
        x = torch.cat([self.anchor[:, None], self.tokens[:, :-1]], 1).long()
        return self.rows.float() + (self.U[x].float() @ self.Wt.float().t())

    def __call__(self, z, stream=None):
        vsd.policy_loss(z, self.tokens, self.old, self.adv, weight=self.weight, grad=True, ws=self.ws["policy"],
                        out=self.loss, stream=stream)
        vsd.markov_grad(self.loss["grad"], self.anchor, self.prev, self.U, self.Wt, ws=self.ws["markov"],
                        out=dict(U=self.grads[0], Wt=self.grads[1]), stream=stream)
        vsd.adamw(self.table, self.count, lr=1e-2, seed=3, ws=self.ws["adamw"], stream=stream)

    def all(self):
        return [self.U, self.Wt, self.count, *self.grads, *self.loss.values(), *(x for s in self.states for x in s.values())]

    def healthy(self):
        return all(vsd.device_status(w) == 0 for w in self.ws.values())


def test_a_step_against_the_oracle(spec):
    t = Step()
    U0, W0 = t.U.clone(), t.Wt.clone()
    t(t.z)
    torch.cuda.synchronize()
    # the drawn tokens' probabilities are the draft's own, which gives them to 1e-5
    e = 2.0 ** -24
    on = (t.weight > 0).cpu().numpy()
    bar = (200 + 6 * t.z.abs().max().item()) * e + 1e-5 / t.old.exp().cpu().numpy().clip(1e-30)
    assert (np.abs((t.loss["logp"] - t.old).cpu().numpy()) <= bar)[on].all()
    flat = lambda x: x.reshape(t.B * t.G, *x.shape[2:]).double().cpu().numpy()   # noqa: E731
    want = op.policy_loss(flat(t.z), flat(t.tokens).astype(int), flat(t.old), flat(t.adv), None, flat(t.weight))
    g = om.markov_grad(want["grad"].reshape(t.B, t.G, t.V), t.anchor.cpu().numpy(), t.prev.cpu().numpy(),
                       U0.double().cpu().numpy(), W0.double().cpu().numpy())
    # q and the slope are off by some 200 e of themselves (their largest is |slope|: row errors go by q),
    # products by (n, V / 8) e more, and the result is rounded to bf16
    for k, got in zip(("U", "Wt"), t.grads):
        err = np.abs(got.double().cpu().numpy() - g[k])
        assert (err <= 2.0 ** -8 * np.abs(g[k]) + (1000 + t.V / 8) * e * g[k + "_abs"] + 2.0 ** -134).all(), k
    assert int(t.count) == 1 and (t.U != U0).any() and t.healthy()


def test_gradients_of_the_weights_against_differences(spec):
    """The loss of the rows as the weights give them, by central differences in float64."""
    t = Step(B=3, G=3, V=501, r=16, seed=2)
    x = torch.cat([t.anchor[:, None], t.tokens[:, :-1]], 1).long().cpu()
    rows, old, adv, w = (a.double().cpu().numpy() for a in (t.rows.float(), t.old, t.adv, t.weight))
    # away from the clip's border at u = 1 + 0
    U, Wt = t.U.double().cpu().numpy(), t.Wt.double().cpu().numpy()
    t(t.biased())

    def loss(U, Wt):
        z = rows + U[x.numpy()] @ Wt.T
        r = op.policy_loss(z.reshape(9, -1), t.tokens.cpu().numpy().reshape(-1), old.reshape(-1), adv.reshape(-1), None, w.reshape(-1))
        return (r["loss"] * w.reshape(-1)).sum()
    rng = np.random.default_rng(1)
    g = om.markov_grad(np.zeros((3, 3, 501)), t.anchor.cpu().numpy(), t.prev.cpu().numpy(), U, Wt)   # (shapes)
    for k, (got, M) in enumerate(zip(t.grads, (U, Wt))):
        for _ in range(4):
            h = rng.normal(size=M.shape)
            if k == 0:
                h[np.setdiff1d(np.arange(501), x.numpy().ravel())] = 0
            eps = 1e-5
            num = (loss(U + eps * h, Wt) - loss(U - eps * h, Wt)) if k == 0 else (loss(U, Wt + eps * h) - loss(U, Wt - eps * h))
            ana = (got.double().cpu().numpy() * h).sum()
            # bf16's rounding of every entry, float32's of the sums, h^2 of third derivatives
            bar = (2.0 ** -8 + 1e-4) * np.abs(got.double().cpu().numpy() * h).sum() + 1e-8
            assert abs(num / (2 * eps) - ana) <= bar
    assert g["U"].shape == U.shape


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_in_a_graph(spec, bits):
    """Replays give what eager steps give, bit for bit, the step count on the device included."""
    a, b = Step(bits=bits), Step(bits=bits)
    za, zb = a.biased(), b.biased()
    a(za)
    b(zb)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a(za)
    for k in range(3):
        za.copy_(a.biased() * (1 + 0.1 * k))
        zb.copy_(b.biased() * (1 + 0.1 * k))
        graph.replay()
        b(zb)
    torch.cuda.synchronize()
    assert int(a.count) == 4
    for x, y in zip(a.all(), b.all()):
        x, y = (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in (x, y))
        assert torch.equal(x, y)
    assert a.healthy() and b.healthy()


def test_two_graphs_share_workspaces(spec):
    """Two captured steps of one drafter on different rows, replayed in turn."""
    a, b = Step(seed=4), Step(seed=4)
    z1, z2 = a.biased(), a.biased() * 1.2
    graphs = []
    a(z1), b(z1)
    torch.cuda.synchronize()
    for z in (z1, z2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            a(z)
        graphs.append(g)
    for k in (0, 1, 1, 0):
        graphs[k].replay()
        b((z1, z2)[k])
    torch.cuda.synchronize()
    for x, y in zip(a.all(), b.all()):
        assert torch.equal(x, y)


def test_steps_on_two_streams(spec):
    """Drafters of their own on streams of their own; inputs made on another stream."""
    steps = [Step(seed=5, V=20011, B=20), Step(seed=6, V=20000, B=20)]
    alone = [Step(seed=5, V=20011, B=20), Step(seed=6, V=20000, B=20)]
    zs = [t.biased() for t in steps]
    for t, z in zip(alone, zs):
        for _ in range(4):
            t(z)
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(4):
        for t, z, s in zip(steps, zs, streams):
            t(z, stream=s)
    torch.cuda.synchronize()
    for t, u in zip(steps, alone):
        assert t.healthy()
        for x, y in zip(t.all(), u.all()):
            assert torch.equal(x, y)


def test_host_threads(spec):
    """Threads inside the calls at the same time, with sizes that take different kernels."""
    made = [dict(B=2, G=3, V=3001, r=32), dict(B=30, G=5, V=9000, r=256), dict(B=4, G=7, V=70001, r=64)]
    alone = [Step(**k) for k in made]
    for t in alone:
        z = t.z
        for _ in range(5):
            t(z)
    steps = [Step(**k) for k in made]
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    errors = []

    def run(t, s):
        try:
            with torch.cuda.stream(s):
                for _ in range(5):
                    t(t.z)
            s.synchronize()
        except Exception as e:   # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=run, args=(t, s)) for t, s in zip(steps, streams)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors
    for t, u in zip(steps, alone):
        for x, y in zip(t.all(), u.all()):
            assert torch.equal(x, y)


def test_gradients_of_the_other_losses(spec):
    """distill's and e2etv's gradients go to the weights the same way."""
    t = Step(B=4, G=5, V=2000, r=64)
    top = vsd.top_logits(t.target[:, :t.G].reshape(-1, t.V), 16)
    z = t.z.view(-1, t.V)
    d = vsd.distill(z, top["values"], top["ids"], tail=top["tail"], grad=True)
    tv = vsd.e2etv(t.target[:, :t.G].reshape(-1, t.V).contiguous(), z.to(BF16), t.B, t.G)
    for grad in (d["grad"], tv["grad"]):
        got = vsd.markov_grad(grad.view(t.B, t.G, t.V), t.anchor, t.tokens, t.U, t.Wt, dtype=F32)
        want = om.markov_grad(grad.view(t.B, t.G, t.V).double().cpu().numpy(), t.anchor.cpu().numpy(), t.tokens.cpu().numpy(),
                              t.U.double().cpu().numpy(), t.Wt.double().cpu().numpy())
        for k in ("U", "Wt"):
            err = np.abs(got[k].double().cpu().numpy() - want[k])
            assert (err <= (t.V / 8 + 64) * 2.0 ** -24 * want[k + "_abs"] + 2.0 ** -24 * np.abs(want[k])).all()


@pytest.mark.parametrize("rank", [32, 64])
def test_example_trains_its_bias(spec, rank):
    """The example's drafter with a bias runs, and its calls report nothing."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    at = importlib.util.spec_from_file_location("online_distill", os.path.join(root, "examples", "online_distill.py"))
    ex = importlib.util.module_from_spec(at)
    at.loader.exec_module(ex)
    loss, accepted = ex.run(steps=4, requests=3, gamma=4, vocab=5003, k=16, rank=rank, report=lambda s: None)
    assert len(loss) == len(accepted) == 4 and np.isfinite(loss).all()
