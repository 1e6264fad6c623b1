"""A row's largest logits with the log-sum-exp of the rest, and distillation from them
(oracle side, float64).

Test infrastructure only (see ``oracle/__init__.py``).

``top_logits``: the K largest entries, descending, ties to the lowest index, never an
entry of -inf (slots left over: id -1, value -inf); tail = ln sum exp(z_v / t) over the
entries not taken, lse over all.

``distill``: the teacher's buckets are its named entries and the rest, p = softmax over
(values / t, tail); the student's q = softmax(z / t), its rest the entries no id names:

    loss = sum_k p_k ln(p_k / q_k) + p_T ln(p_T / q_T)
    grad = (weight / t) (q_v - p_k) for a named v, (weight / t) q_v (1 - p_T / q_T) else

Pins (``tests/test_oracle_teacher.py``): a worked example; K = V without a rest is the
full KL divergence; one entry is the cross entropy; the gradient against central finite
differences of the loss; its rows sum to zero; a student equal to the teacher's row has
loss 0 and gradient 0; the loss is never negative; tail and lse against the sums they
stand for, with a rest 1e-12 of the row.
"""

import numpy as np

from ._rows import as_f64, row_valid


def lse(x):
    """ln sum exp(x), -inf for nothing."""
    x = as_f64(x)
    x = x[x > -np.inf]
    if x.size == 0:
        return -np.inf
    m = x.max()
    return float(m + np.log(np.exp(x - m).sum()))


def top_row(z, K, t=1.0):
    """(values [K], ids [K], tail, lse) of one row."""
    z = as_f64(z)
    V = z.shape[0]
    values, ids = np.full(K, -np.inf), np.full(K, -1, dtype=np.int64)
    if np.isnan(z).any() or np.isposinf(z).any():
        return np.full(K, np.nan), ids, np.nan, np.nan
    order = np.lexsort((np.arange(V), -z))
    order = order[z[order] > -np.inf][:K]
    values[:order.size] = z[order]
    ids[:order.size] = order
    rest = np.ones(V, dtype=bool)
    rest[order] = False
    return values, ids, lse(z[rest] / t), lse(z / t)


def top_logits(rows, K, t=1.0):
    out = [top_row(r, K, t) for r in as_f64(rows)]
    return dict(values=np.stack([o[0] for o in out]), ids=np.stack([o[1] for o in out]),
                tail=np.array([o[2] for o in out]), lse=np.array([o[3] for o in out]))


def distill_row(z, values, ids, tail=-np.inf, weight=1.0, t=1.0):
    """dict(loss, lse, grad [V], p [K + 1], q [V], qt) of one row."""
    z = as_f64(z)
    V = z.shape[0]
    zero = dict(loss=0.0, lse=0.0, grad=np.zeros(V), p=np.zeros(len(ids) + 1), q=np.zeros(V), qt=0.0)
    if weight == 0.0:
        return zero
    named = [int(i) for i in ids if i >= 0]
    vals = as_f64([v for v, i in zip(values, ids) if i >= 0])
    nan = dict(loss=np.nan, lse=np.nan, grad=np.full(V, np.nan), p=zero["p"], q=zero["q"], qt=0.0)
    if any(not -1 <= int(i) < V for i in ids) or len(set(named)) != len(named) or not row_valid(z):
        return nan
    b = np.append(vals / t, tail)
    if np.isnan(b).any() or np.isposinf(b).any():
        return nan
    lq = z / t - lse(z / t)
    q = np.exp(lq)
    rest = np.ones(V, dtype=bool)
    rest[named] = False
    lqt = lse(lq[rest])
    if lse(b) == -np.inf:
        return dict(zero, lse=lse(z / t), q=q, qt=float(np.exp(lqt)))
    lp = b - lse(b)
    p = np.exp(lp)
    lqb = np.append(lq[named], lqt)
    on = p > 0
    with np.errstate(all="ignore"):
        loss = float((p[on] * (lp[on] - lqb[on])).sum())
    grad = q - (np.exp(lq - lqt) * p[-1] if lqt > -np.inf else 0.0)
    grad[named] = q[named] - p[:-1]
    full = np.zeros(len(ids) + 1)
    full[[k for k, i in enumerate(ids) if i >= 0]] = p[:-1]
    full[-1] = p[-1]
    return dict(loss=loss, lse=lse(z / t), grad=grad * (weight / t), p=full, q=q, qt=float(np.exp(lqt)))


def distill(student, values, ids, tail=None, weight=None, t=1.0):
    """Every row: dict(loss [R], lse [R], grad [R, V], p, q, qt)."""
    S = as_f64(student)
    out = [distill_row(S[r], values[r], ids[r], -np.inf if tail is None else float(tail[r]),
                       1.0 if weight is None else float(weight[r]), t) for r in range(S.shape[0])]
    return {k: np.stack([o[k] for o in out]) for k in out[0]}
