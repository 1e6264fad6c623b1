"""Pins of oracle.process: worked examples and token-by-token equivalence."""

import numpy as np
import pytest

from oracle import process as op


def test_worked_example():
    # history: prompt [1, 2], generated [2, 3, 3]; block [0]
    l = np.array([1.0, -2.0, 4.0, 3.0, 5.0])
    y = op.row(l, np.array([1, 2, 2, 3, 3]), 2, [0], repetition=2.0, frequency=0.5, presence=0.25,
               bias=[(4, -1.0), (-1, 99.0), (0, 7.0), (0, 3.0)], temperature=0.5)
    # 0: in the block: 1/2 - .5 - .25 + 3 (the later bias); 1: prompt only: -2*2
    # 2: 4/2 - .5 - .25; 3: 3/2 - 1 - .25; 4: 5 - 1
    np.testing.assert_allclose(y, np.array([2.75, -4.0, 1.25, 0.25, 4.0]) / 0.5, rtol=1e-15)


def test_block_rows_equal_token_by_token():
    rng = np.random.default_rng(3)
    B, R, V, L = 2, 5, 40, 17
    logits = rng.normal(size=(B, R, V)) * 3
    hist, block = rng.integers(0, V, (B, L)), rng.integers(0, V, (B, R - 1))
    lengths, prompts = np.array([17, 9]), np.array([4, 9])
    kw = dict(repetition=np.array([1.3, 0.8]), frequency=np.array([0.4, 0.1]), presence=np.array([0.2, -0.3]),
              temperature=np.array([0.7, 1.5]))
    got = op.process_logits(logits, hist, lengths, prompts, block, **kw)
    for b in range(B):
        for j in range(R):
            h = np.concatenate([hist[b, :lengths[b]], block[b, :j]])[None]
            one = op.process_logits(logits[b:b + 1, j:j + 1], h, None, prompts[b:b + 1],
                                    **{k: v[b:b + 1] for k, v in kw.items()})
            np.testing.assert_array_equal(got[b, j], one[0, 0])


def test_neutral_and_masked():
    rng = np.random.default_rng(4)
    logits = rng.normal(size=(1, 2, 70))
    hist = rng.integers(0, 70, (1, 30))
    np.testing.assert_array_equal(op.process_logits(logits, hist), logits)
    bad = logits.copy()
    bad[0, 0, 3], bad[0, 1, 69] = np.nan, np.inf
    mask = np.full((1, 2, 3), -1, dtype=np.int32)
    mask[0, 0, 0] &= ~(1 << 3)
    mask[0, 1, 2] = 0
    y = op.process_logits(bad, hist, mask=mask)
    assert y[0, 0, 3] == -np.inf and np.isfinite(np.delete(y[0, 0], 3)).all()
    assert (y[0, 1, 64:] == -np.inf).all() and np.isfinite(y[0, 1, :64]).all()
    assert (op.process_logits(logits, mask=np.zeros((1, 3), dtype=np.int32)) == -np.inf).all()


@pytest.mark.parametrize("V", [1, 31, 32, 33, 64])
def test_unpack(V):
    rng = np.random.default_rng(V)
    bits = rng.random(V) < 0.5
    words = np.zeros((V + 31) // 32, dtype=np.uint32)
    for v in np.nonzero(bits)[0]:
        words[v // 32] |= np.uint32(1 << (int(v) % 32))
    np.testing.assert_array_equal(op.unpack(words.astype(np.int32), V), bits)
