"""fp64 statement of the filtered distributions: which tokens of a row are kept, and which one is drawn.

From the definitions: the weights w_i = exp((l_i - max l) / T), the ranking by logit (equal ones by index, -inf not at
all), and its first min(n_k, n_p, n_m) tokens.
"""
from __future__ import annotations

import numpy as np


def ranking(l):
    """Indices in the ranking's order; tokens of -inf are not in it."""
    l = np.asarray(l, dtype=np.float64)
    order = np.lexsort((np.arange(len(l)), -l))
    return order[:np.count_nonzero(l > -np.inf)]


def counts(l, T=1.0, k=0, p=1.0, mp=0.0, slack=0.0):
    """(fewest, most) tokens that may be kept when every sum of weights is off by `slack` of itself; equal for 0."""
    l = np.asarray(l, dtype=np.float64)
    rank = ranking(l)
    if T == 0:
        return 1, 1
    z = (l[rank] - l[rank[0]]) / T
    w = np.exp(z)
    most = len(rank)
    if k >= 1:
        most = min(most, k)
    out = []
    for sign in (-1, 1):
        n = most
        if p < 1:
            c = np.cumsum(w[:most])
            n = min(n, int(np.searchsorted(c, p * c[-1] * (1 + sign * slack), side="left")) + 1)
        if mp > 0:
            # by logarithms: a weight just below 1 is 1 in fp64
            n = min(n, int(np.count_nonzero(z >= (np.log(mp) + np.log1p(-sign * slack) if mp < 1 else 0.0))))
        out.append(max(n, 1))
    return out[0], out[1]


def kept(l, n):
    """The first n of the ranking, as booleans."""
    m = np.zeros(len(l), dtype=bool)
    m[ranking(l)[:n]] = True
    return m


def draws(l, T, keep, u, slack=0.0):
    """(lowest, highest) token that may be drawn from the kept ones, and the log of every kept token's probability."""
    l = np.asarray(l, dtype=np.float64)
    at = np.flatnonzero(keep)
    w = np.ones(len(at)) if T == 0 else np.exp((l[at] - l[at].max()) / T)
    c = np.cumsum(w)
    ends = [min(int(np.searchsorted(c, max(0.0, u - s) * c[-1], side="right")), len(at) - 1) for s in (slack, -slack)]
    logp = np.full(len(l), -np.inf)
    logp[at] = (0.0 if T == 0 else (l[at] - l[at].max()) / T) - np.log(c[-1])
    return int(at[ends[0]]), int(at[ends[1]]), logp
