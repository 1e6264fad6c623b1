"""Penalties, biases, temperature and grammar masks on a block's logits rows (oracle
side, float64).

Test infrastructure only (see ``oracle/__init__.py``).

Row j of request b is the distribution after the request's history and the block tokens
x_1..x_j.  With c(v) the occurrences of v in the generated part of that context and
seen(v) = v anywhere in it:

    y = l;  seen: y > 0 ? y / repetition : y * repetition
    y -= frequency * c + presence * [c > 0];  y += bias;  y /= temperature
    masked: -inf, whatever y is

Pins (``tests/test_oracle_process.py``): worked examples; row j of a block equals row 0
of the history extended by x_1..x_j (token-by-token decoding); neutral parameters leave
the rows as they are; masked entries hide NaN and +inf.
"""

import numpy as np

from ._rows import as_f64


def row(logits, history, prompt_length, block=(), repetition=1.0, frequency=0.0, presence=0.0, bias=(), mask=None,
        temperature=1.0):
    """One row [V].  history: the context's tokens, the first prompt_length the prompt;
    block: the drafted tokens before this row; bias: (id, value) pairs, a later pair of
    the same id replacing an earlier one; mask: booleans [V] or None."""
    y = as_f64(logits).copy()
    V = y.shape[0]
    ok = [int(t) for t in history[prompt_length:] if 0 <= t < V] + [int(t) for t in block if 0 <= t < V]
    count = np.bincount(ok, minlength=V)
    seen = count > 0
    seen[[int(t) for t in history[:prompt_length] if 0 <= t < V]] = True
    with np.errstate(all="ignore"):
        y = np.where(seen, np.where(y > 0, y / repetition, y * repetition), y)
        y = y - (frequency * count + presence * (count > 0))
        for i, v in dict((int(i), float(v)) for i, v in bias if 0 <= i < V).items():
            y[i] += v
        y = y / temperature
    if mask is not None:
        y[~np.asarray(mask, dtype=bool)] = -np.inf
    return y


def unpack(mask_row, V):
    """The booleans of a packed mask row of 32-bit words."""
    w = np.asarray(mask_row).astype(np.uint32)
    v = np.arange(V)
    return ((w[v // 32] >> (v % 32).astype(np.uint32)) & 1).astype(bool)


def process_logits(logits, history=None, lengths=None, prompt_lengths=None, block=None, repetition=None,
                   frequency=None, presence=None, bias_ids=None, bias_values=None, mask=None, temperature=None):
    """Every row of a batch: logits [B, R, V]; the other arguments as the library's."""
    L = as_f64(logits)
    B, R, V = L.shape
    out = np.empty((B, R, V))
    at = lambda a, b, d: d if a is None else float(a[b])   # noqa: E731
    for b in range(B):
        Lmax = 0 if history is None else history.shape[1]
        n = Lmax if lengths is None else min(max(int(lengths[b]), 0), Lmax)
        m = 0 if prompt_lengths is None else min(max(int(prompt_lengths[b]), 0), n)
        h = [] if history is None else history[b, :n]
        bias = [] if bias_ids is None else list(zip(bias_ids[b], bias_values[b]))
        for j in range(R):
            mk = None
            if mask is not None:
                mk = unpack(mask[b, j] if np.ndim(mask) == 3 else mask[b], V)
            out[b, j] = row(L[b, j], h, m, [] if block is None else block[b, :j], at(repetition, b, 1.0),
                            at(frequency, b, 0.0), at(presence, b, 0.0), bias, mk, at(temperature, b, 1.0))
    return out
