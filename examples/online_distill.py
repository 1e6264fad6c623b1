"""A drafter that learns from the rows it is verified on.

Serves blocks of a synthetic target with a DSpark drafter and trains the drafter's logits on
the way, with the library's calls in the order a server would make them:

    draft_block      gamma tokens per request from the drafter's rows
    process_logits   penalties, biases, a grammar and the temperature on the target's rows, the
                     drafted tokens counted for the rows behind them
    verify           accepted drafts and the bonus token, at T=1
    top_logits       the processed target rows, kept as a teacher in a few hundred bytes each
    distill          loss and gradient of the drafter's rows from that teacher; rows behind the
                     first rejection do not count (their target rows follow tokens that were
                     not committed)

The "drafter" is a table of logits per context that the gradient is applied to, so the script
needs no model: it prints the loss and the accepted drafts per step, which fall and rise.

    python examples/online_distill.py [--steps 30] [--requests 16] [--gamma 7] [--vocab 32000]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import verify_spec_draft_gb300 as vsd  # noqa: E402
from verify_spec_draft_gb300 import synth  # noqa: E402


def run(steps=30, requests=16, gamma=7, vocab=32000, k=64, lr=60.0, seed=0, report=print):
    dev = torch.device("cuda")
    B, G, V = requests, gamma, vocab
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    # the target's rows and the drafter's first guess of them, fixed per request and position
    target, draft = synth.target_and_draft(B, G, V, "gaussian", 2.0, torch.bfloat16, seed=seed, device=dev)
    master = draft.float()                                   # the drafter's parameters
    history = torch.randint(0, V, (B, 64), generator=g, device=dev, dtype=torch.int32)
    prompts = torch.full((B,), 48, dtype=torch.int32, device=dev)
    ones = torch.ones(B, device=dev)
    sampling = dict(repetition=1.1 * ones, frequency=0.2 * ones, presence=0.1 * ones, temperature=0.8 * ones)
    grammar = torch.randint(-2**31, 2**31, (B, G + 1, (V + 31) // 32), generator=g, device=dev,
                            dtype=torch.int64).to(torch.int32)
    anchor = history[:, -1].contiguous()
    # workspaces are made once and kept
    ws = dict(process=vsd.workspace(vsd.OP_PROCESS_LOGITS, B, G + 1, V), draft=vsd.workspace(vsd.OP_DRAFT, B, G, V, 0),
              verify=vsd.workspace(vsd.OP_VERIFY, B, G, V), top=vsd.workspace(vsd.OP_TOP_LOGITS, B * (G + 1), k, V),
              distill=vsd.workspace(vsd.OP_DISTILL, B * G, k, V))
    position = torch.arange(G, device=dev)
    losses, accepted = [], []
    for step in range(steps):
        seeds = synth.seeds_for(B, step * B, dev)
        rows = master.to(torch.bfloat16)
        d = vsd.draft_block(rows, anchor, temperature=1, seeds=seeds, qlogits=True, ws=ws["draft"])
        p = vsd.process_logits(target, history=history, prompt_lengths=prompts, block=d["tokens"], mask=grammar,
                               ws=ws["process"], **sampling)
        v = vsd.verify(p["logits"], d["qlogits"], d["tokens"], 1, seeds, ws=ws["verify"])
        t = vsd.top_logits(p["logits"].view(B * (G + 1), V), k, ws=ws["top"])
        teach = {key: t[key].view(B, G + 1, *t[key].shape[1:])[:, :G].reshape(B * G, *t[key].shape[1:])
                 for key in ("values", "ids", "tail")}
        # position j's target row follows x_1..x_j, so it counts while those were accepted
        weight = (position[None, :] <= v["n"][:, None]).float()
        weight = (weight / weight.sum()).reshape(B * G)
        s = vsd.distill(rows.view(B * G, V), teach["values"], teach["ids"], tail=teach["tail"], weight=weight,
                        grad=True, ws=ws["distill"])
        master.view(B * G, V).sub_(lr * s["grad"].float())
        losses.append((s["loss"] * weight).sum())
        accepted.append(v["n"].float().mean())
    for w in ws.values():
        if vsd.device_status(w) != 0:
            raise RuntimeError("a call reported an invalid row or token")
    losses, accepted = torch.stack(losses).tolist(), torch.stack(accepted).tolist()
    for i in range(0, steps, max(1, steps // 10)):
        report(f"step {i:3d}  loss {losses[i]:7.4f}  accepted {accepted[i]:5.2f} of {G}")
    report(f"last      loss {losses[-1]:7.4f}  accepted {accepted[-1]:5.2f} of {G}")
    return losses, accepted


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--gamma", type=int, default=7)
    ap.add_argument("--vocab", type=int, default=32000)
    a = ap.parse_args()
    vsd.load()
    run(a.steps, a.requests, a.gamma, a.vocab)
