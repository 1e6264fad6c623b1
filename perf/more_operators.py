"""The operators of a drafter's training step: cases, inputs, plain forms.

    policy   the clipped policy loss of sampled blocks with a KL term against a reference,
             a row of V logits per token, with the gradient of the logits or without it
    markov   the gradients of the Markov bias weights U and Wt from the rows' gradient
    adamw    one AdamW step over many tensors at once, states in 32 bits or in 8

``run`` computes them with elementary torch operations in float32, or (``own``) through
the library's public calls ``policy_loss``, ``markov_grad`` and ``adamw``.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
CLIP_LOW, CLIP_HIGH = 0.2, 0.28
LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.01
BLOCK = 128                       # entries of an 8-bit state that share a scale


# ---------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------
def _policy(R, V, dtype, t, kl, grad):
    return dict(op="policy", R=R, V=V, dtype=dtype, t=t, kl=kl, grad=grad)


def _markov(B, gamma, V, r, dtype, out):
    return dict(op="markov", B=B, gamma=gamma, V=V, r=r, dtype=dtype, out=out)


def _adamw(tensors, n, even, param, grad, bits, clip):
    return dict(op="adamw", tensors=tensors, n=n, even=even, param=param, grad=grad, bits=bits, clip=clip)


def listed():
    return [
        # one block of 7 sampled tokens: a step of online training, latency
        dict(_policy(7, 32000, "f32", 1.0, 0.05, True), name="policy_branch"),
        # a training batch: 256 branches of 7 positions, a reference policy
        dict(_policy(1792, 248320, "bf16", 1.0, 0.05, True), name="policy_train"),
        # log-probabilities and losses of a held-out batch (64 x 7), without a gradient
        dict(_policy(448, 248320, "bf16", 1.0, 0.0, False), name="policy_score"),
        # a training batch with an odd vocabulary, sampled at a temperature
        dict(_policy(455, 50257, "bf16", 0.7, 0.02, True), name="policy_odd"),
        # the smallest drafter: one block of 7, float32 rows and weights of rank 32
        dict(_markov(1, 7, 32000, 32, "f32", "f32"), name="markov_branch"),
        # the training batch: 256 branches of 7 positions, rank 256
        dict(_markov(256, 7, 248320, 256, "bf16", "bf16"), name="markov_train"),
        # an odd vocabulary, float32 gradients of bf16 weights
        dict(_markov(65, 7, 50257, 128, "bf16", "f32"), name="markov_odd"),
        # norms and biases of a small head: latency
        dict(_adamw(6, 4096, False, "f32", "f32", 32, False), name="adamw_small"),
        # the two weight tables of the drafter's bias, float32 states and masters
        dict(_adamw(2, 248320 * 256, True, "bf16", "bf16", 32, False), name="adamw_tables"),
        # the same with 8-bit states, gradients scaled by a clip factor
        dict(_adamw(2, 248320 * 256, True, "bf16", "bf16", 8, True), name="adamw_tables_8bit"),
        # a drafter's layers: many tensors of ragged sizes
        dict(_adamw(180, 2000003, False, "bf16", "f32", 8, False), name="adamw_many"),
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["policy", "policy", "markov", "markov", "adamw"])
    V = rng.choice([_between(rng, 1000, 248320), _between(rng, 1000, 248320) // 8 * 8, 32000, 151936, 248320])
    if op == "policy":
        dtype = rng.choice(["f32", "bf16"])
        grad = rng.random() < 0.6
        rows = 1792 if grad else 448
        most = rows * 248320 * 2 // (V * (4 if dtype == "f32" else 2))
        R = _between(rng, 1, max(1, min(4096, most)))
        return _policy(R, V, dtype, rng.choice([1.0, 0.7, 1.5]), rng.choice([0.0, 0.02, 0.1]), grad)
    if op == "markov":
        gamma = rng.choice([1, 3, 5, 7, 8, 15])
        if rng.random() < 0.25:
            V = _between(rng, 1000, 50257)
            return _markov(_between(rng, 1, 32), gamma, V, rng.choice([8, 16, 32, 50]), "f32", "f32")
        r = rng.choice([32, 64, 128, 192, 256])
        most = min(1792, 1792 * 248320 * 256 // (V * r)) // gamma
        return _markov(_between(rng, 1, max(1, most)), gamma, V, r, "bf16", rng.choice(["f32", "bf16"]))
    tensors = _between(rng, 1, 300)
    return _adamw(tensors, _between(rng, 100, 100000000 // tensors), rng.random() < 0.3, *rng.choice(
        [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]), rng.choice([32, 8]), rng.random() < 0.5)


def _sizes(case):
    """The tensors' entries: all alike, or ragged (whole fractions of n and some more)."""
    if case["even"]:
        return [case["n"]] * case["tensors"]
    return [case["n"] // (1 + i * i % 11) + i * 37 % 101 for i in range(case["tensors"])]


# ---------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------
def _rows(R, V, g, dev):
    """Logits: a few strong tokens at independent places over a broad bulk."""
    z = torch.randn((R, V), generator=g, device=dev) * 2.0
    u = torch.rand((R, V), generator=g, device=dev)
    return z.sub_(torch.log_(u.clamp_(min=1e-7)))


def _logp(z, x):
    m = z.max(1, keepdim=True).values
    s = torch.exp(z - m).sum(1)
    return torch.gather(z, 1, x.long()[:, None]).squeeze(1) - m.squeeze(1) - torch.log(s)


def _prepare_policy(case, g, dev):
    R, V, t = case["R"], case["V"], case["t"]
    s = dict(case=case)
    rows = _rows(R, V, g, dev)
    # the sampled tokens: mostly likely ones, by Gumbel noise
    tokens = torch.empty((R,), dtype=torch.int32, device=dev)
    for lo in range(0, R, 256):
        u = torch.rand(rows[lo:lo + 256].shape, generator=g, device=dev).clamp_(min=1e-20)
        tokens[lo:lo + 256] = (rows[lo:lo + 256] / t - torch.log(-torch.log(u))).argmax(1).to(torch.int32)
    s["tokens"] = tokens
    s["logits"] = rows.to(DTYPES[case["dtype"]])
    logp = torch.cat([_logp(z.float() / t, x) for z, x in zip(s["logits"].split(256), tokens.split(256))])
    # the policy has moved a little since the tokens were drawn; no row lies on a clip border
    moved = 0.25 * torch.randn((R,), generator=g, device=dev)
    for border in (math.log(1 - CLIP_LOW), math.log(1 + CLIP_HIGH)):
        moved = torch.where((moved - border).abs() < 1e-3, moved + 4e-3, moved)
    s["old_logp"] = logp - moved
    s["advantage"] = torch.randn((R,), generator=g, device=dev)
    s["ref_logp"] = logp + 0.5 * torch.randn((R,), generator=g, device=dev) if case["kl"] else None
    # the mean over the rows that count: about one in ten is padding
    keep = (torch.rand((R,), generator=g, device=dev) > 0.1).float()
    keep[0] = 1.0
    s["weight"] = keep / keep.sum()
    return s


def _prepare_markov(case, g, dev):
    B, gamma, V, r = case["B"], case["gamma"], case["V"], case["r"]
    dt = DTYPES[case["dtype"]]
    s = dict(case=case)
    # what a distillation or policy loss leaves: a difference of distributions over the batch's mean
    d = torch.empty((B * gamma, V), dtype=dt, device=dev)
    for lo in range(0, B * gamma, 256):
        z = _rows(min(256, B * gamma - lo), V, g, dev)
        q = torch.softmax(z, 1)
        p = torch.softmax(z + 0.8 * torch.randn(z.shape, generator=g, device=dev), 1)
        d[lo:lo + 256] = ((q - p) / (B * gamma)).to(dt)
    # text: a few tokens come back often; some branches end early
    u = torch.rand((B, gamma + 1), generator=g, device=dev)
    x = (torch.pow(float(V), u) - 1.0).to(torch.int32).clamp_(0, V - 1)
    ends = torch.randint(1, 8 * gamma + 2, (B, 1), generator=g, device=dev)
    ends[0] = gamma + 1
    position = torch.arange(gamma + 1, device=dev)
    x = torch.where(position < ends, x, torch.full_like(x, -1))
    s["anchor"], s["tokens"] = x[:, 0].contiguous(), x[:, 1:].contiguous()
    s["grad"] = d.view(B, gamma, V).mul_((position[:gamma] < ends)[:, :, None].to(dt))
    for name in ("U", "Wt"):
        s[name] = (0.02 * torch.randn((V, r), generator=g, device=dev)).to(dt)
    return s


def _prepare_adamw(case, g, dev):
    sizes = _sizes(case)
    # the tensors lie in one buffer of each kind, each on a block of its own
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += (n + BLOCK - 1) // BLOCK * BLOCK

    def cut(flat, per=1):
        return [flat[a // per:a // per + (n + per - 1) // per] for a, n in zip(starts, sizes)]

    s = dict(case=case, sizes=sizes, starts=starts)
    inside = torch.zeros((total,), dtype=torch.bool, device=dev)
    for part in cut(inside):
        part.fill_(True)
    master = 0.05 * torch.randn((total,), generator=g, device=dev)
    s["grad"] = (0.01 * torch.randn((total,), generator=g, device=dev)).to(DTYPES[case["grad"]])
    m = 2e-3 * torch.randn((total,), generator=g, device=dev) * inside
    root = (torch.exp(0.7 * torch.randn((total,), generator=g, device=dev)) * 5e-3) * inside   # sqrt(v)
    s["param"] = master.to(DTYPES[case["param"]])
    s["master"] = master if case["param"] == "bf16" else None
    if case["bits"] == 32:
        s["m"], s["v"] = m, root * root
        s["m_scale"] = s["v_scale"] = None
    else:
        for name, x in (("m", m), ("v", root)):
            top = x.abs().view(-1, BLOCK).amax(1)
            scale = torch.exp2(torch.floor(torch.log2(top.clamp(min=1e-30))) - 7.0)
            s[name] = (x.view(-1, BLOCK) / scale[:, None]).clamp(-256, 256).to(torch.float8_e4m3fn).view(-1)
            s[name + "_scale"] = scale
    s["step"] = torch.full((1,), 100, dtype=torch.int32, device=dev)
    s["clip"] = 0.5 + torch.rand((1,), generator=g, device=dev) if case["clip"] else None
    s["seed"] = 12345
    return s, cut


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 29)
    if case["op"] == "policy":
        s = _prepare_policy(case, g, dev)
    elif case["op"] == "markov":
        s = _prepare_markov(case, g, dev)
    else:
        s, cut = _prepare_adamw(case, g, dev)
    if own:
        import verify_spec_draft_gb300 as vsd
        if case["op"] == "policy":
            s["ws"] = vsd.workspace(vsd.OP_POLICY_LOSS, case["R"], 1, case["V"])
        elif case["op"] == "markov":
            s["ws"] = vsd.workspace(vsd.OP_MARKOV_GRAD, case["B"], case["gamma"], case["V"], case["r"])
        else:
            names = ["m", "v"] + (["master"] if s["master"] is not None else [])
            states = [dict(zip(names, parts)) for parts in zip(*(cut(s[k]) for k in names))]
            if case["bits"] == 8:
                for d, a, b in zip(states, cut(s["m_scale"], BLOCK), cut(s["v_scale"], BLOCK)):
                    d["m_scale"], d["v_scale"] = a, b
            s["table"] = vsd.adamw_table(cut(s["param"]), cut(s["grad"]), states)
            s["ws"] = vsd.workspace(vsd.OP_ADAMW, len(s["sizes"]), 1, 1)
    return s


# ---------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------
def _plain_policy(s):
    case, z, w = s["case"], s["logits"], s["weight"]
    t = case["t"]
    x = z.float() / t
    m = x.max(1, keepdim=True).values
    e = torch.exp(x - m)
    Z = e.sum(1, keepdim=True)
    at = s["tokens"].long()[:, None]
    logp = (torch.gather(x, 1, at) - m - torch.log(Z)).squeeze(1)
    A = s["advantage"]
    ratio = torch.exp(logp - s["old_logp"])
    clipped = torch.clamp(ratio, 1.0 - CLIP_LOW, 1.0 + CLIP_HIGH)
    loss = -torch.minimum(ratio * A, clipped * A)
    flows = torch.where(A >= 0, ratio <= 1.0 + CLIP_HIGH, ratio >= 1.0 - CLIP_LOW)
    slope = torch.where(flows, -A * ratio, torch.zeros_like(A))
    if s["ref_logp"] is not None:
        d = s["ref_logp"] - logp
        loss = loss + case["kl"] * (torch.expm1(d) - d)
        slope = slope - case["kl"] * torch.expm1(d)
    counts = w != 0
    loss = torch.where(counts, loss, torch.zeros_like(loss))
    logp = torch.where(counts, logp, torch.zeros_like(logp))
    if not case["grad"]:
        return loss, logp
    k = (torch.where(counts, slope * w, torch.zeros_like(w)) / t)[:, None]
    d = e * (-k / Z)
    # at the token: slope (1 - q), with 1 - q from what the others weigh
    others = e.scatter(1, at, 0.0).sum(1, keepdim=True)
    d.scatter_(1, at, k * (others / Z))
    return loss, logp, d.to(z.dtype)


def _plain_markov(s):
    case = s["case"]
    V, r = case["V"], case["r"]
    prev = torch.cat([s["anchor"][:, None], s["tokens"][:, :-1]], 1).reshape(-1).long()
    there = prev >= 0
    at = torch.where(there, prev, torch.zeros_like(prev))
    d = s["grad"].reshape(-1, V).float() * there[:, None].float()
    rows = s["U"][at].float() * there[:, None].float()
    dWt = d.t() @ rows
    dU = torch.zeros((V, r), device=d.device).index_add_(0, at, d @ s["Wt"].float())
    out = DTYPES[case["out"]]
    return dU.to(out), dWt.to(out)


def _philox(seed, blocks, step, tensor):
    """Philox4x32-10 (Salmon, Moraes, Dror, Shaw, SC'11): key (seed's halves), counter (block's
    halves, step, tensor).  Words are held in 64 bits."""
    low = 0xFFFFFFFF
    c0, c1 = blocks & low, (blocks >> 32) & low
    c2, c3 = step & low, torch.full_like(blocks, tensor)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c0, c1, c2, c3


def _packed(x, random, least):
    """x in e4m3 against a power of two per block, rounded at random: up where 16 random bits
    exceed what is left.  `least`: the smallest code of a value above 0."""
    top = x.abs().view(-1, BLOCK).amax(1)
    e = torch.clamp((top.view(torch.int32) >> 23) - 7, min=1)
    y = (x.view(-1, BLOCK) * ((254 - e) << 23).view(torch.float32)[:, None]).view(-1)
    mag = y.abs()
    normal = ((mag.view(torch.int32) + (random << 4)) >> 20) - 960
    small = ((mag * 33554432.0).to(torch.int32) + random) >> 16
    code = torch.where(mag >= 0.015625, normal, small)
    code = torch.where((x > 0) & (code < least), torch.full_like(code, least), code)
    code = code | torch.where(x < 0, torch.full_like(code, 128), torch.zeros_like(code))
    return code.to(torch.uint8).view(torch.float8_e4m3fn), (e << 23).view(torch.float32)


def _plain_adamw(s):
    case = s["case"]
    s["step"] += 1
    t = s["step"].double()
    size = (LR / (1.0 - torch.pow(BETA1, t))).float()
    root = (1.0 / torch.sqrt(1.0 - torch.pow(BETA2, t))).float()
    for i, (a, n) in enumerate(zip(s["starts"], s["sizes"])):
        inside = slice(a, a + n)
        g = s["grad"][inside].float()
        if s["clip"] is not None:
            g = g * s["clip"]
        if case["bits"] == 8:
            blocks = (n + BLOCK - 1) // BLOCK
            codes = slice(a, a + blocks * BLOCK)
            scales = slice(a // BLOCK, a // BLOCK + blocks)
            m, q = ((s[k][codes].float().view(-1, BLOCK) * s[k + "_scale"][scales][:, None]).view(-1)[:n]
                    for k in ("m", "v"))
            v = q * q
        else:
            m, v = s["m"][inside], s["v"][inside]
        m = m * BETA1 + g * (1.0 - BETA1)
        v = v * BETA2 + g * (1.0 - BETA2) * g
        q = torch.sqrt(v)
        p = s["master"] if s["master"] is not None else s["param"]
        new = p[inside] * (1.0 - LR * DECAY) - size * (m / (q * root + EPS))
        p[inside] = new
        if s["master"] is not None:
            s["param"][inside] = new.to(s["param"].dtype)
        if case["bits"] == 32:
            s["m"][inside], s["v"][inside] = m, v
            continue
        index = torch.arange(blocks * BLOCK // 4, device=g.device)
        random = torch.stack(_philox(s["seed"], index, s["step"].long(), i), 1).view(-1)
        pad = blocks * BLOCK - n
        for k, x, bits, least in (("m", m, random & 0xFFFF, 0), ("v", q, random >> 16, 1)):
            code, scale = _packed(torch.nn.functional.pad(x, (0, pad)), bits.to(torch.int32), least)
            s[k].view(torch.uint8)[inside] = code.view(torch.uint8)[:n]
            s[k + "_scale"][scales] = scale


def _adamw_outputs(s):
    return [s[k] for k in ("param", "master", "m", "v", "m_scale", "v_scale", "step") if s[k] is not None]


def run(state):
    s = state
    case = s["case"]
    if own:
        import verify_spec_draft_gb300 as vsd
        if case["op"] == "policy":
            r = vsd.policy_loss(s["logits"], s["tokens"], s["old_logp"], s["advantage"], ref_logp=s["ref_logp"],
                                weight=s["weight"], temperature=case["t"], clip=(CLIP_LOW, CLIP_HIGH),
                                kl=case["kl"], grad=case["grad"], ws=s["ws"])
            return (r["loss"], r["logp"], r["grad"]) if case["grad"] else (r["loss"], r["logp"])
        if case["op"] == "markov":
            r = vsd.markov_grad(s["grad"], s["anchor"], s["tokens"], s["U"], s["Wt"], dtype=DTYPES[case["out"]],
                                ws=s["ws"])
            return r["U"], r["Wt"]
        vsd.adamw(s["table"], s["step"], lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY,
                  grad_scale=s["clip"], seed=s["seed"], ws=s["ws"])
        return _adamw_outputs(s)
    if case["op"] == "policy":
        return _plain_policy(s)
    if case["op"] == "markov":
        return _plain_markov(s)
    _plain_adamw(s)
    return _adamw_outputs(s)


def work(case):
    if case["op"] == "policy":
        R, row = case["R"], case["V"] * (4 if case["dtype"] == "f32" else 2)
        return {"bytes": R * ((2 if case["grad"] else 1) * row + 28), "flops": (8 if case["grad"] else 4) * R * case["V"]}
    if case["op"] == "markov":
        R, V, r = case["B"] * case["gamma"], case["V"], case["r"]
        size, out = (4 if case["dtype"] == "f32" else 2), (4 if case["out"] == "f32" else 2)
        return {"bytes": R * (V + r) * size + V * r * size + 2 * V * r * out, "flops": 4 * R * V * r}
    n = sum(_sizes(case))
    param = 10 if case["param"] == "bf16" else 8        # the master read and written, and its bf16 copy
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * (param + (4 if case["grad"] == "f32" else 2) + state), "flops": 16 * n}


# ---------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------
def _exact_policy(s):
    case, t = s["case"], s["case"]["t"]
    R, V = s["logits"].shape
    losses, logps, grads = [], [], []
    step = max(1, (1 << 25) // V)
    for lo in range(0, R, step):
        rows = slice(lo, min(R, lo + step))
        lq = torch.log_softmax(s["logits"][rows].double() / t, 1)
        n = lq.shape[0]
        i = torch.arange(n, device=lq.device)
        x = s["tokens"][rows].long()
        logp = lq[i, x]
        A, w = s["advantage"][rows].double(), s["weight"][rows].double()
        u = torch.exp(logp - s["old_logp"][rows].double())
        inside = (u >= 1 - CLIP_LOW) & (u <= 1 + CLIP_HIGH)
        bounded = u.clip(1 - CLIP_LOW, 1 + CLIP_HIGH)
        loss = torch.maximum(-u * A, -bounded * A)
        # the gradient passes where the smaller of the two products is the one that moves
        slope = torch.where(inside | (u * A < bounded * A), -A * u, 0.0 * A)
        if s["ref_logp"] is not None:
            gap = s["ref_logp"][rows].double() - logp
            loss = loss + case["kl"] * (torch.exp(gap) - gap - 1.0)
            slope = slope + case["kl"] * (1.0 - torch.exp(gap))
        losses.append(loss * (w != 0))
        logps.append(logp * (w != 0))
        if case["grad"]:
            d = -torch.exp(lq)
            d[i, x] += 1.0
            grads.append(d * (slope * w / t)[:, None])
    if not case["grad"]:
        return torch.cat(losses), torch.cat(logps)
    return torch.cat(losses), torch.cat(logps), torch.cat(grads)


def _exact_markov(s):
    V = s["case"]["V"]
    before = [s["anchor"]] + list(s["tokens"].unbind(1))[:-1]
    prev = torch.stack(before, 1).flatten().long()
    rows = torch.nonzero(prev >= 0).squeeze(1)
    prev = prev[rows]
    d = s["grad"].flatten(0, 1)[rows].double()
    dU = torch.zeros(s["U"].shape, dtype=torch.float64, device=d.device)
    dWt = torch.zeros_like(dU)
    dx = torch.zeros((len(rows), s["U"].shape[1]), dtype=torch.float64, device=d.device)
    u = s["U"].double()[prev]
    for lo in range(0, V, 65536):
        part = d[:, lo:lo + 65536]
        dWt[lo:lo + 65536] = torch.einsum("nv,nr->vr", part, u)
        dx += part @ s["Wt"][lo:lo + 65536].double()
    order = torch.argsort(prev, stable=True)
    token, count = torch.unique_consecutive(prev[order], return_counts=True)
    end = torch.cumsum(count, 0)
    run = torch.cat([torch.zeros_like(dx[:1]), torch.cumsum(dx[order], 0)])
    dU[token] = run[end] - run[end - count]
    return dU, dWt


def _exact_adamw(s):
    case = s["case"]
    t = int(s["step"]) + 1
    out = {k: s[k].double() for k in ("param", "master", "m", "v", "m_scale", "v_scale") if s[k] is not None}
    for a, n in zip(s["starts"], s["sizes"]):
        at = slice(a, a + n)
        blocks = slice(a // BLOCK, (a + n + BLOCK - 1) // BLOCK)
        g = s["grad"][at].double() * (1.0 if s["clip"] is None else s["clip"].double())
        if case["bits"] == 8:
            per = torch.arange(n, device=g.device) // BLOCK
            m = s["m"][at].double() * s["m_scale"][blocks].double()[per]
            v = (s["v"][at].double() * s["v_scale"][blocks].double()[per]) ** 2
        else:
            m, v = s["m"][at].double(), s["v"][at].double()
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g * g
        hat_m, hat_v = m / (1 - BETA1 ** t), v / (1 - BETA2 ** t)
        p = (s["param"] if s["master"] is None else s["master"])[at].double()
        p = p - LR * DECAY * p - LR * hat_m / (hat_v.sqrt() + EPS)
        out["param"][at] = p
        if s["master"] is not None:
            out["master"][at] = p
        if case["bits"] == 32:
            out["m"][at], out["v"][at] = m, v
            continue
        # the codes before they are rounded at random
        for k, x in (("m", m), ("v", v.sqrt())):
            top = torch.zeros((blocks.stop - blocks.start,), dtype=torch.float64, device=g.device)
            top.scatter_reduce_(0, per, x.abs(), "amax")
            scale = 2.0 ** (torch.frexp(top).exponent.double() - 8)
            out[k][at] = x / scale[per]
            out[k + "_scale"] = None    # a power of two that a 32-bit value next to a border picks
    out["step"] = s["step"] + 1
    return [out[k] for k in ("param", "master", "m", "v", "m_scale", "v_scale", "step") if k in out]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "policy":
        return _exact_policy(s)
    if case["op"] == "markov":
        return _exact_markov(s)
    return _exact_adamw(s)
