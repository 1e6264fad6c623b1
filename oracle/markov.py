"""The gradients of the Markov bias weights (oracle side, float64).

Test infrastructure only (see ``oracle/__init__.py``).

The draft's rows are z_j = l_j + U[x_{j-1}] Wt^T (``draft``), x_0 the anchor, so with dz the
gradient of the rows, dWt = sum of dz outer U[x_{j-1}] and dU[x_{j-1}] += dz Wt, over the
positions whose x_{j-1} is a token.

Pins (``tests/test_oracle_training.py``): finite differences of a linear functional of the
rows that ``draft.draft_block`` returns; a token that comes back gets the sum; positions
behind an ended block count for nothing, whatever their dz holds.
"""

import numpy as np

from ._rows import as_f64


def markov_grad(dz, anchor, tokens, U, Wt):
    """dict(U, Wt) and their sums of magnitudes (U_abs, Wt_abs), what rounding errors go by."""
    dz, U, Wt = as_f64(dz), as_f64(U), as_f64(Wt)
    B, gamma, V = dz.shape
    g = {k: np.zeros_like(U) for k in ("U", "Wt", "U_abs", "Wt_abs")}
    for b in range(B):
        for j in range(gamma):
            x = int(anchor[b]) if j == 0 else int(tokens[b, j - 1])
            if not 0 <= x < V:
                continue
            d = dz[b, j]
            g["Wt"] += np.outer(d, U[x])
            g["U"][x] += d @ Wt
            g["Wt_abs"] += np.outer(np.abs(d), np.abs(U[x]))
            g["U_abs"][x] += np.abs(d) @ np.abs(Wt)
    return g
