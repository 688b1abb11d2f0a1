"""The oracle of the filtered distributions against enumeration in exact fractions (CPU)."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import sample as os_


def brute(weights, k, p, mp):
    """Kept tokens by the definition, weights as fractions (the largest 1)."""
    rank = sorted((i for i, w in enumerate(weights) if w > 0), key=lambda i: (-weights[i], i))
    n_k = k if 1 <= k < len(rank) else len(rank)
    total = sum(weights[i] for i in rank[:n_k])
    n_p = len(rank)
    if p < 1:
        n_p = next(n for n in range(1, len(rank) + 1) if sum(weights[i] for i in rank[:n]) >= p * total)
    n_m = sum(weights[i] >= min(mp, 1) for i in rank) if mp > 0 else len(rank)
    return rank[:min(n_k, n_p, n_m)]


@pytest.mark.parametrize("seed", range(60))
def test_against_enumeration(seed):
    rng = np.random.default_rng(seed)
    e = rng.integers(0, 6, size=rng.integers(1, 12))
    e = e - e.min()
    weights = [Fraction(1, 2 ** int(x)) for x in e]
    l = -np.log(2.0) * e.astype(np.float64)
    k = int(rng.integers(0, 8))
    # borders that no sum of these weights meets: odd denominators
    p, mp = (Fraction(int(rng.integers(1, 101)), 101) for _ in range(2))
    kept = brute(weights, k, p, mp)
    assert os_.counts(l, 1.0, k, float(p), float(mp)) == (len(kept), len(kept))
    mask = os_.kept(l, len(kept))
    assert np.flatnonzero(mask).tolist() == sorted(kept)
    total = sum(weights[i] for i in kept)
    u = Fraction(int(rng.integers(0, 103)), 103)
    run, want = Fraction(0), None
    for i in sorted(kept):
        run += weights[i]
        if run > u * total:
            want = i
            break
    lo, hi, logp = os_.draws(l, 1.0, mask, float(u))
    assert lo == hi == want
    assert abs(np.exp(logp[want]) - float(weights[want] / total)) < 1e-15


def test_edges():
    l = np.array([0.0, 1.0, -np.inf, 1.0, 0.5])
    assert os_.ranking(l).tolist() == [1, 3, 4, 0]
    assert os_.counts(l, 0.0, 3, 0.5, 0.5) == (1, 1)
    assert os_.counts(l) == (4, 4)
    assert os_.counts(l, 1.0, 0, 0.0) == (1, 1)
    assert os_.counts(l, 1.0, 0, 1.0, 5.0) == (2, 2)  # both of the largest
    assert os_.draws(l, 0.0, os_.kept(l, 1), 0.99)[:2] == (1, 1)


def test_min_p_near_one_counts_logits_and_not_rounded_weights():
    l = np.array([3e-25, 1e-25, 3e-25, -2.0])
    assert os_.counts(l, 1.0, mp=1.0) == (2, 2)
    assert os_.counts(l, 1e30, mp=1.0) == (2, 2)
    assert os_.counts(l, 1.0, mp=0.5) == (3, 3)
    assert os_.counts(np.array([0.0, np.log(0.25), np.log(0.25) - 1e-9]), 1.0, mp=0.25, slack=1e-6) == (1, 3)
