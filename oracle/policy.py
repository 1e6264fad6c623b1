"""The clipped policy loss of sampled tokens with a KL term (oracle side, float64).

Test infrastructure only (see ``oracle/__init__.py``).

For a row z, its token x and q = softmax(z / t): lp = ln q_x, u = exp(lp - old),
d = ref - lp,

    loss = -min(u A, clip(u, 1 - low, 1 + high) A) + kl (e^d - d - 1)
    grad = (weight / t) (d loss / d lp) ([v = x] - q_v)

where the clipped product's derivative is 0 and, at a border, the unclipped one's holds.

Pins (``tests/test_oracle_training.py``): a worked row on each side of both borders; without
clipping and KL term the gradient is the policy gradient; the gradient against central
finite differences of the loss; its rows sum to zero; the KL term is never negative and 0 at
the reference; at u = 1 the loss is -A.
"""

import numpy as np

from ._rows import as_f64, row_valid
from .teacher import lse


def row(z, x, old, A, ref=None, weight=1.0, t=1.0, low=0.2, high=0.2, kl=0.0):
    """dict(loss, logp, grad [V], slope, q [V]) of one row."""
    z = as_f64(z)
    V = z.shape[0]
    if weight == 0.0:
        return dict(loss=0.0, logp=0.0, grad=np.zeros(V), slope=0.0, q=np.zeros(V))
    nan = dict(loss=np.nan, logp=np.nan, grad=np.full(V, np.nan), slope=np.nan, q=np.full(V, np.nan))
    ref = ref if kl > 0 else None
    numbers = [old, A, weight] + ([ref] if ref is not None else [])
    if not 0 <= x < V or not row_valid(z) or not np.isfinite(numbers).all():
        return nan
    q = np.exp(z / t - lse(z / t))
    lp = z[x] / t - lse(z / t)
    with np.errstate(over="ignore", invalid="ignore"):
        u = np.exp(lp - old)
        loss = slope = 0.0
        if A != 0.0:
            loss = -min(u * A, min(max(u, 1.0 - low), 1.0 + high) * A)
            if (u <= 1.0 + high) if A > 0 else (u >= 1.0 - low):
                slope = -u * A
        if ref is not None:
            d = ref - lp
            e = np.expm1(d)
            loss += kl * (e - d) if d < np.inf else np.inf
            slope -= kl * e
        grad = slope * (weight / t) * (-q)
        grad[x] = slope * (weight / t) * np.delete(q, x).sum()
    return dict(loss=loss, logp=lp, grad=grad if np.isfinite(slope) else np.full(V, np.nan), slope=slope, q=q)


def policy_loss(rows, tokens, old, A, ref=None, weight=None, t=1.0, low=0.2, high=0.2, kl=0.0):
    Z = as_f64(rows)
    out = [row(Z[i], int(tokens[i]), float(old[i]), float(A[i]), None if ref is None else float(ref[i]),
               1.0 if weight is None else float(weight[i]), t, low, high, kl) for i in range(Z.shape[0])]
    return {k: np.stack([o[k] for o in out]) for k in out[0]}
