"""fp64 oracle: log probabilities of given tokens, entropies, most likely classes
and the gradient of the first two.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""
from __future__ import annotations

import numpy as np


def token_logprobs(z, tokens, n_top: int):
    """Returns a dict of logprob [N], entropy [N], norm [N, 2] (the largest logit,
    log of the sum against it), top_id and top_logprob [N, n_top]."""
    z = np.asarray(z, np.float64)
    N, V = z.shape
    r = dict(logprob=np.zeros(N), entropy=np.zeros(N), norm=np.full((N, 2), -np.inf), top_id=np.full((N, n_top), -1),
             top_logprob=np.full((N, n_top), -np.inf))
    for n in range(N):
        m = z[n].max()
        t = int(tokens[n])
        if m == -np.inf:
            r["logprob"][n] = -np.inf if 0 <= t < V else 0.0
            continue
        x = z[n] - m
        e = np.exp(x)
        s = e.sum()
        r["norm"][n] = m, np.log(s)
        lp = x - np.log(s)
        p = e / s
        r["entropy"][n] = -np.sum(p[p > 0] * lp[p > 0])
        if 0 <= t < V:
            r["logprob"][n] = lp[t]
        order = sorted(np.argpartition(-x, min(V - 1, 2 * n_top))[:2 * n_top + 1] if n_top and V > 4 * n_top and len(np.unique(x)) == V else range(V),
                       key=lambda j: (-x[j], j))[:n_top]
        for k, j in enumerate(order):
            if x[j] > -np.inf:
                r["top_id"][n, k], r["top_logprob"][n, k] = j, lp[j]
    return r


def token_logprobs_bwd(z, tokens, d_logprob, d_entropy):
    """dz [N, V] of sum d_logprob * logprob + d_entropy * entropy."""
    z = np.asarray(z, np.float64)
    dz = np.zeros_like(z)
    for n in range(z.shape[0]):
        m = z[n].max()
        if m == -np.inf:
            continue
        e = np.exp(z[n] - m)
        p = e / e.sum()
        lp = z[n] - m - np.log(e.sum())
        plp = np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0)
        dz[n] = -d_entropy[n] * (plp - p * plp.sum())
        t = int(tokens[n])
        if 0 <= t < z.shape[1]:
            dz[n] -= d_logprob[n] * p
            dz[n, t] += d_logprob[n]
    return dz
