"""The vocabulary-wide operators around verification and distillation: cases, inputs,
plain forms.

    process  penalties for repeated tokens, biases, temperature and grammar masks on the
             logits rows of a block, before they are verified
    top      each row's K largest logits and the log-sum-exp of the rest: a teacher row in
             its compact form
    distill  the distillation loss of a drafter's rows from such a teacher (forward)
    grad     the same loss with the gradient of the drafter's logits

``run`` computes them with elementary torch operations in float32, or (``own``) through
the library's public calls ``process_logits``, ``top_logits`` and ``distill``.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------
def _process(B, R, V, L, dtype, mask, biases):
    return dict(op="process", B=B, R=R, V=V, L=L, dtype=dtype, mask=mask, biases=biases)


def _top(R, V, K, t, dtype, grammar):
    return dict(op="top", R=R, V=V, K=K, t=t, dtype=dtype, grammar=grammar)


def _distill(op, R, V, K, t, dtype, tail):
    return dict(op=op, R=R, V=V, K=K, t=t, dtype=dtype, tail=tail)


def listed():
    return [
        # one request, one token at a time, a short chat: the call's latency is what counts
        dict(_process(1, 1, 32000, 60, "f32", False, 0), name="process_one_token"),
        # the latency configuration: one request, a block of 15, a grammar and a long context
        dict(_process(1, 16, 248320, 4096, "bf16", True, 16), name="process_block15"),
        # the serving configuration: 32 requests, blocks of 7, grammars, 300 biased tokens each
        dict(_process(32, 8, 248320, 8192, "bf16", True, 300), name="process_serve"),
        # a vocabulary that is no multiple of anything, float32 rows
        dict(_process(5, 6, 50257, 777, "f32", True, 5), name="process_odd"),
        # the teacher's row for one token of a response
        dict(_top(1, 32000, 20, 1.0, "f32", False), name="top_one_row"),
        # the verified rows of a serving step (32 requests x 8 rows), some under a grammar
        dict(_top(256, 248320, 64, 1.0, "bf16", True), name="top_serve"),
        # a recorded batch: odd vocabulary, many entries kept, softened
        dict(_top(611, 50257, 100, 2.0, "f32", False), name="top_odd"),
        # held-out branches scored without a gradient (64 anchors x 7 positions)
        dict(_distill("distill", 448, 248320, 64, 1.0, "bf16", True), name="distill_eval"),
        # a small held-out set, odd vocabulary, teacher renormalised over its entries
        dict(_distill("distill", 37, 20001, 33, 1.5, "f32", False), name="distill_odd"),
        # one branch of 7 positions: a step of online distillation, latency
        dict(_distill("grad", 7, 32000, 20, 1.0, "f32", True), name="grad_branch"),
        # a training batch: 256 branches of 7 positions
        dict(_distill("grad", 1792, 248320, 64, 1.0, "bf16", True), name="grad_train"),
        # a training batch with an odd vocabulary, softened, renormalised teacher
        dict(_distill("grad", 455, 50257, 100, 2.0, "bf16", False), name="grad_odd"),
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["process", "top", "distill", "grad"])
    V = rng.choice([_between(rng, 1000, 248320), _between(rng, 1000, 248320) // 8 * 8, 32000, 151936, 248320])
    dtype = rng.choice(["f32", "bf16"])
    size = 4 if dtype == "f32" else 2
    # bytes of the rows: up to the largest listed case of the same operator
    most = {"process": 32 * 8 * 248320 * 2, "top": 256 * 248320 * 2, "distill": 448 * 248320 * 2,
            "grad": 1792 * 248320 * 2}[op] // (V * size)
    if op == "process":
        R = min(rng.choice([1, 2, 4, 6, 8, 16]), most)
        B = _between(rng, 1, max(1, min(64, most // R)))
        return _process(B, R, V, _between(rng, 1, 8192), dtype, rng.random() < 0.6, rng.choice([0, 3, 40, 300]))
    R = _between(rng, 1, max(1, min(4096, most)))
    K = _between(rng, 1, 128)
    t = rng.choice([1.0, 0.7, 1.5, 2.0])
    if op == "top":
        return _top(R, V, K, t, dtype, rng.random() < 0.5)
    return _distill(op, R, V, K, t, dtype, rng.random() < 0.6)


# ---------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------
def _rows(R, V, g, dev):
    """Target logits: a few strong tokens at independent places over a broad bulk."""
    z = torch.randn((R, V), generator=g, device=dev) * 2.0
    u = torch.rand((R, V), generator=g, device=dev)
    return z.sub_(torch.log_(u.clamp_(min=1e-7)))   # an exponential upper tail: a skewed head


def _top_of(rows, K):
    """The K largest of each row, descending, ties to the lowest index; -inf is not taken."""
    x = rows.float()
    bits = x.contiguous().view(torch.int32).to(torch.int64)
    order = torch.where(bits >= 0, bits, -2147483648 - bits)          # ordered as the floats are; -0.0 as 0.0
    V = x.shape[1]
    key = order * 4294967296 + (V - 1 - torch.arange(V, device=x.device))
    k = min(K, V)
    at = torch.topk(key, k, dim=1).indices
    val = torch.gather(x, 1, at)
    ids = torch.where(val > -math.inf, at, torch.full_like(at, -1)).to(torch.int32)
    if k < K:
        pad = K - k
        val = torch.cat([val, torch.full((x.shape[0], pad), -math.inf, device=x.device)], 1)
        ids = torch.cat([ids, torch.full((x.shape[0], pad), -1, dtype=torch.int32, device=x.device)], 1)
    return val, ids


def _plain_top(rows, K, t):
    val, ids = _top_of(rows, K)
    x = rows.float() / t
    m = x.max(1, keepdim=True).values
    e = torch.exp(x - m)
    lse = (m + torch.log(e.sum(1, keepdim=True))).squeeze(1)
    taken = torch.cat([x, torch.zeros_like(x[:, :1])], 1)
    taken.scatter_(1, torch.where(ids >= 0, ids, torch.full_like(ids, x.shape[1])).long(), -math.inf)
    rest = taken[:, :-1]
    mr = rest.max(1, keepdim=True).values
    some = mr > -math.inf
    mr = torch.where(some, mr, torch.zeros_like(mr))
    tail = (mr + torch.log(torch.exp(rest - mr).sum(1, keepdim=True))).squeeze(1)
    return val, ids, tail, lse


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 17)
    dt = DTYPES[case["dtype"]]
    V = case["V"]
    s = dict(case=case)
    if case["op"] == "process":
        B, R, L = case["B"], case["R"], case["L"]
        s["logits"] = _rows(B * R, V, g, dev).view(B, R, V).to(dt)
        lengths = torch.randint((L + 1) // 2, L + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        lengths[0] = L
        s["lengths"] = lengths
        s["prompt_lengths"] = (lengths.float() * torch.rand((B,), generator=g, device=dev)).to(torch.int32)

        def tokens(*shape):   # text: a few tokens come back often
            u = torch.rand(shape, generator=g, device=dev)
            return (torch.pow(float(V), u) - 1.0).to(torch.int32).clamp_(0, V - 1)

        s["history"] = tokens(B, L)
        s["block"] = tokens(B, R - 1)
        s["repetition"] = 1.0 + 0.3 * torch.rand((B,), generator=g, device=dev)
        s["frequency"] = 0.5 * torch.rand((B,), generator=g, device=dev)
        s["presence"] = torch.rand((B,), generator=g, device=dev) - 0.2
        s["temperature"] = 0.5 + torch.rand((B,), generator=g, device=dev)
        s["bias_ids"] = s["bias_values"] = s["mask"] = None
        nb = case["biases"]
        if nb:
            # distinct tokens of each request: a random place, then steps over the vocabulary
            first = torch.randint(0, V, (B, 1), generator=g, device=dev)
            step = max(1, V // (nb + 1))
            ids = (first + step * torch.arange(nb, device=dev)) % V
            s["bias_ids"] = ids.to(torch.int32)
            s["bias_values"] = 4.0 * torch.randn((B, nb), generator=g, device=dev)
        if case["mask"]:
            # a grammar allows most tokens in some states and a handful in others
            W = (V + 31) // 32
            bits = torch.randint(-2**31, 2**31, (B, R, W), generator=g, device=dev, dtype=torch.int64)
            more = torch.randint(-2**31, 2**31, (B, R, W), generator=g, device=dev, dtype=torch.int64)
            wide = torch.rand((B, R, 1), generator=g, device=dev) < 0.5
            s["mask"] = torch.where(wide, bits | more, bits & more & (more >> 3)).to(torch.int32)
    elif case["op"] == "top":
        rows = _rows(case["R"], V, g, dev)
        if case["grammar"]:
            # one row in eight allows a few dozen tokens only
            few = torch.rand((case["R"], 1), generator=g, device=dev) < 0.125
            ban = torch.rand((case["R"], V), generator=g, device=dev) > 40.0 / V
            ban[:, 0] = False
            rows = rows.masked_fill_(few & ban, -math.inf)
        s["rows"] = rows.to(dt)
    else:
        R, K = case["R"], case["K"]
        rows = _rows(R, V, g, dev)
        parts = [_plain_top(r, K, case["t"]) for r in rows.to(dt).split(128)]
        s["values"], s["ids"], tail, _ = (torch.cat(p) for p in zip(*parts))
        s["tail"] = tail if case["tail"] else None
        rows += 0.8 * torch.randn((R, V), generator=g, device=dev)
        s["student"] = rows.to(dt)
        if case["op"] == "grad":
            # the mean over the rows that count: about one in ten is padding
            keep = (torch.rand((R,), generator=g, device=dev) > 0.1).float()
            keep[0] = 1.0
            s["weight"] = keep / keep.sum()
    if own:
        import verify_spec_draft_gb300 as vsd
        if case["op"] == "process":
            s["ws"] = vsd.workspace(vsd.OP_PROCESS_LOGITS, case["B"], case["R"], V)
        elif case["op"] == "top":
            s["ws"] = vsd.workspace(vsd.OP_TOP_LOGITS, case["R"], case["K"], V)
        else:
            s["ws"] = vsd.workspace(vsd.OP_DISTILL, case["R"], case["K"], V)
    return s


# ---------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------
def _plain_process(s):
    logits = s["logits"]
    B, R, V = logits.shape
    dev = logits.device
    L = s["history"].shape[1]
    pos = torch.arange(L, device=dev)
    live = pos < s["lengths"][:, None]
    made = live & (pos >= s["prompt_lengths"][:, None])
    hist = s["history"].long()
    ones = torch.ones((B, L), device=dev)
    said = torch.zeros((B, V), device=dev).scatter_add_(1, hist, ones * live)      # prompt and output
    count = torch.zeros((B, V), device=dev).scatter_add_(1, hist, ones * made)     # output
    bias = None
    if s["bias_ids"] is not None:
        bias = torch.zeros((B, V), device=dev).scatter_(1, s["bias_ids"].long(), s["bias_values"])
    rep, freq, pres, temp = (s[k][:, None] for k in ("repetition", "frequency", "presence", "temperature"))
    out = torch.empty_like(logits)
    shift = torch.arange(32, device=dev, dtype=torch.int32)
    for j in range(R):
        if j > 0:
            x = s["block"][:, j - 1:j].long()
            one = torch.ones((B, 1), device=dev)
            said.scatter_add_(1, x, one)
            count.scatter_add_(1, x, one)
        y = logits[:, j].float()
        y = torch.where(said > 0, torch.where(y > 0, y / rep, y * rep), y)
        y = y - (freq * count + pres * (count > 0))
        if bias is not None:
            y = y + bias
        y = y / temp
        if s["mask"] is not None:
            allowed = ((s["mask"][:, j, :, None] >> shift) & 1).reshape(B, -1)[:, :V]
            y = torch.where(allowed > 0, y, torch.full_like(y, -math.inf))
        out[:, j] = y.to(logits.dtype)
    return out


def _plain_distill(s, grad):
    z, ids, t = s["student"], s["ids"].long(), s["case"]["t"]
    R, V = z.shape
    x = z.float() / t
    m = x.max(1, keepdim=True).values
    e = torch.exp(x - m)
    there = ids >= 0
    at = torch.where(there, ids, torch.full_like(ids, V))
    named = torch.cat([e, torch.zeros_like(e[:, :1])], 1)
    qe = torch.gather(named, 1, at)                                # 0 for an absent entry
    named.scatter_(1, at, 0.0)
    st = named.sum(1, keepdim=True)                                # what no id names
    Z = st + qe.sum(1, keepdim=True)
    a = torch.where(there, s["values"].float() / t, torch.full_like(qe, -math.inf))
    at_tail = s["tail"][:, None] if s["tail"] is not None else torch.full_like(m, -math.inf)
    b = torch.cat([a, at_tail], 1)
    mb = b.max(1, keepdim=True).values
    taught = mb > -math.inf
    mb = torch.where(taught, mb, torch.zeros_like(mb))
    pe = torch.exp(b - mb)
    P = torch.where(taught, pe.sum(1, keepdim=True), torch.ones_like(mb))
    p = pe / P
    logp = (b - mb) - torch.log(P)
    xk = torch.gather(torch.cat([x, torch.zeros_like(x[:, :1])], 1), 1, at) - m
    logq = torch.cat([xk, torch.log(st)], 1) - torch.log(Z)
    loss = torch.where(p > 0, p * (logp - logq), torch.zeros_like(p)).sum(1)
    lse = (m + torch.log(Z)).squeeze(1)
    if not grad:
        return loss, lse
    w = s["weight"]
    loss = torch.where(w != 0, loss, torch.zeros_like(loss))
    lse = torch.where(w != 0, lse, torch.zeros_like(lse))
    pt = p[:, -1:]
    d = torch.cat([e * (1.0 / Z - torch.where(st > 0, pt / st, torch.zeros_like(st))), torch.zeros_like(e[:, :1])], 1)
    d.scatter_(1, at, qe / Z - p[:, :-1])
    d = d[:, :V] * (w[:, None] / t)
    d = torch.where(taught & (w[:, None] != 0), d, torch.zeros_like(d))
    return loss, lse, d.to(z.dtype)


def run(state):
    s = state
    case = s["case"]
    if own:
        import verify_spec_draft_gb300 as vsd
        if case["op"] == "process":
            return vsd.process_logits(
                s["logits"], history=s["history"], lengths=s["lengths"], prompt_lengths=s["prompt_lengths"],
                block=s["block"], repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                bias_ids=s["bias_ids"], bias_values=s["bias_values"], mask=s["mask"],
                temperature=s["temperature"], ws=s["ws"])["logits"]
        if case["op"] == "top":
            r = vsd.top_logits(s["rows"], case["K"], temperature=case["t"], ws=s["ws"])
            return r["values"], r["ids"], r["tail"], r["lse"]
        if case["op"] == "distill":
            r = vsd.distill(s["student"], s["values"], s["ids"], tail=s["tail"], temperature=case["t"], ws=s["ws"])
            return r["loss"], r["lse"]
        r = vsd.distill(s["student"], s["values"], s["ids"], tail=s["tail"], weight=s["weight"],
                        temperature=case["t"], grad=True, ws=s["ws"])
        return r["loss"], r["lse"], r["grad"]
    if case["op"] == "process":
        return _plain_process(s)
    if case["op"] == "top":
        return _plain_top(s["rows"], case["K"], case["t"])
    return _plain_distill(s, case["op"] == "grad")


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    V = case["V"]
    if case["op"] == "process":
        B, R = case["B"], case["R"]
        mask = B * R * ((V + 31) // 32) * 4 if case["mask"] else 0
        return {"bytes": 2 * B * R * V * size + mask + B * (4 * case["L"] + 8 * case["biases"] + 4 * R + 20),
                "flops": 2 * B * R * V}
    R, K = case["R"], case["K"]
    if case["op"] == "top":
        return {"bytes": R * (V * size + 8 * K + 8), "flops": 4 * R * V}
    if case["op"] == "distill":
        return {"bytes": R * (V * size + 8 * K + 12), "flops": 4 * R * V}
    return {"bytes": R * (2 * V * size + 8 * K + 16), "flops": 8 * R * V}


# ---------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------
def _exact_process(s):
    logits = s["logits"]
    B, R, V = logits.shape
    out = torch.empty((B, R, V), dtype=torch.float64, device=logits.device)
    for b in range(B):
        n, n0 = int(s["lengths"][b]), int(s["prompt_lengths"][b])
        h = s["history"][b, :n].long()
        prompt = torch.bincount(h[:n0], minlength=V)
        rep, freq, pres, temp = (float(s[k][b]) for k in ("repetition", "frequency", "presence", "temperature"))
        for j in range(R):
            said = torch.cat([h[n0:], s["block"][b, :j].long()])
            c = torch.bincount(said, minlength=V).double()
            y = logits[b, j].double()
            scale = torch.where(y > 0, 1.0 / rep, rep)
            seen = (c + prompt) > 0
            y[seen] = y[seen] * scale[seen]
            y = y - freq * c
            y[c > 0] -= pres
            if s["bias_ids"] is not None:
                y.index_add_(0, s["bias_ids"][b].long(), s["bias_values"][b].double())
            y = y / temp
            if s["mask"] is not None:
                v = torch.arange(V, device=y.device)
                word = s["mask"][b, j].long()[v // 32]
                y[torch.bitwise_and(torch.bitwise_right_shift(word, v % 32), 1) == 0] = -math.inf
            out[b, j] = y
    return out


def _exact_top(s):
    K, t = s["case"]["K"], s["case"]["t"]
    rows = s["rows"]
    V = rows.shape[1]
    vals, idss, tails, lses = [], [], [], []
    for part in rows.split(32):
        z = part.double()
        o, at = torch.sort(z, dim=1, descending=True, stable=True)
        k = min(K, V)
        val, ids = o[:, :k].clone(), at[:, :k].clone()
        ids[val == -math.inf] = -1
        x = o / t
        if k < V:
            rest = x[:, k:]
            tails.append(torch.logsumexp(rest, 1))
        else:
            tails.append(torch.full_like(x[:, 0], -math.inf))
        lses.append(torch.logsumexp(x, 1))
        if k < K:
            val = torch.nn.functional.pad(val, (0, K - k), value=-math.inf)
            ids = torch.nn.functional.pad(ids, (0, K - k), value=-1)
        vals.append(val)
        idss.append(ids.to(torch.int32))
    return torch.cat(vals), torch.cat(idss), torch.cat(tails), torch.cat(lses)


def _exact_distill(s, grad):
    t = s["case"]["t"]
    R, V = s["student"].shape
    losses, lses, grads = [], [], []
    step = max(1, (1 << 25) // V)
    for lo in range(0, R, step):
        z = s["student"][lo:lo + step].double()
        n = z.shape[0]
        ids = s["ids"][lo:lo + step].long()
        lq = torch.log_softmax(z / t, 1)
        named = torch.zeros((n, V), dtype=torch.bool, device=z.device)
        r, k = torch.nonzero(ids >= 0, as_tuple=True)
        v = ids[r, k]
        named[r, v] = True
        lqt = torch.logsumexp(lq.masked_fill(named, -math.inf), 1)
        b = torch.full((n, ids.shape[1] + 1), -math.inf, dtype=torch.float64, device=z.device)
        b[r, k] = s["values"][lo:lo + step].double()[r, k] / t
        if s["tail"] is not None:
            b[:, -1] = s["tail"][lo:lo + step].double()
        lp = b - torch.logsumexp(b, 1, keepdim=True)
        p = torch.exp(lp)
        lqb = torch.zeros_like(lp)
        lqb[r, k] = lq[r, v]
        lqb[:, -1] = lqt
        loss = torch.where(p > 0, p * (lp - lqb), torch.zeros_like(p)).sum(1)
        lse = torch.logsumexp(z / t, 1)
        if grad:
            w = s["weight"][lo:lo + step].double()
            q = torch.exp(lq)
            d = q - torch.exp(lq - lqt[:, None]) * p[:, -1:]
            d[r, v] = q[r, v] - p[r, k]
            d = d * (w / t)[:, None]
            grads.append(d)
            loss, lse = loss * (w != 0), lse * (w != 0)
        losses.append(loss)
        lses.append(lse)
    if not grad:
        return torch.cat(losses), torch.cat(lses)
    return torch.cat(losses), torch.cat(lses), torch.cat(grads)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "process":
        return _exact_process(s)
    if case["op"] == "top":
        return _exact_top(s)
    return _exact_distill(s, case["op"] == "grad")
