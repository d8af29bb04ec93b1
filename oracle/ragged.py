"""fp64 oracle: the operators of a ragged step over the paged cache.

TEST INFRASTRUCTURE ONLY (see the package docstring). Plain definitions, one
request after the other.

Request b feeds n[b] new tokens as rows cu[b] .. cu[b+1] - 1, the first at
position ctx[b]; the paged cache is that of the paged oracle.
"""
from __future__ import annotations

import numpy as np


def ragged_plan(n_new, ctx, table, held, free_list, n_free: int, block_size: int, T: int):
    """One step's planning. table [B, max_blocks], held [B], free_list are
    copied; returns a dict of the new state and the step's arrays (pos, slots
    for the rows there are, at most T)."""
    table, held, free = np.array(table), np.array(held), np.array(free_list)
    B, max_blocks = table.shape
    taken = missing = 0
    short = False
    cu, pos, slots = [0], [], []
    for b in range(B):
        n, c = max(0, int(n_new[b])), max(0, int(ctx[b]))
        want = min(-(-(c + n) // block_size), max_blocks) if n else 0
        lack = max(0, want - int(held[b]))
        if lack and (short or taken + lack > n_free):
            short = True
            missing += lack
            table[b, held[b]:want] = -1
        else:
            for _ in range(lack):
                table[b, held[b]] = free[n_free - 1 - taken]
                held[b] += 1
                taken += 1
        for p in range(c, c + n):
            lb = p // block_size
            pos.append(p)
            slots.append(int(table[b, lb]) * block_size + p % block_size if lb < held[b] and table[b, lb] >= 0 else -1)
        cu.append(cu[-1] + n)
    left = n_free - taken
    for b in range(B):
        if n_new[b] < 0:
            free[left:left + held[b]] = table[b, :held[b]]
            left += int(held[b])
            held[b] = 0
    return dict(table=table, held=held, free_list=free, n_free=left, cu=np.minimum(cu, T), pos=np.array(pos[:T], np.int64),
                slots=np.array(slots[:T], np.int64), missing=missing)


def ragged_attention(q, k_pool, v_pool, table, cu, ctx):
    """Row cu[b] + i of q [T, Hq, d] attends to positions 0 .. ctx[b] + i of its
    request. Returns (O [T, Hq, d], lse [T, Hq], A) with A = sum_j p_j |v_j|,
    what a rounding of every weight p_j by a relative step can move O by."""
    q = np.asarray(q, np.float64)
    T, Hq, d = q.shape
    nb, bs, Hkv, _ = k_pool.shape
    O, A, lse = np.zeros_like(q), np.zeros_like(q), np.zeros((T, Hq))
    for b in range(len(ctx)):
        n = int(cu[b + 1] - cu[b])
        L = int(ctx[b]) + n
        if n == 0:
            continue
        p = np.arange(L)
        at = np.asarray(table[b])[p // bs]
        K, V = np.asarray(k_pool[at, p % bs], np.float64), np.asarray(v_pool[at, p % bs], np.float64)
        hidden = p[None, :] > int(ctx[b]) + np.arange(n)[:, None]
        rows = slice(int(cu[b]), int(cu[b + 1]))
        for h in range(Hq):
            j = h // (Hq // Hkv)
            s = q[rows, h] @ K[:, j].T / np.sqrt(d)
            s[hidden] = -np.inf
            top = s.max(1, keepdims=True)
            e = np.exp(s - top)
            den = e.sum(1, keepdims=True)
            lse[rows, h] = (top + np.log(den))[:, 0]
            O[rows, h] = e / den @ V[:, j]
            A[rows, h] = e / den @ np.abs(V[:, j])
    return O, lse, A


def draft_verify(p, q, tokens, cu, u_accept, u_sample):
    """Accept-or-resample of drafted tokens. p, q [T, V] (q may be None: the
    draft's probability is one at its token); returns (accepted, next) lists."""
    accepted, token = [], []
    for b in range(len(cu) - 1):
        r, last = int(cu[b]), int(cu[b + 1]) - 1
        if last < r:
            accepted.append(0)
            token.append(-1)
            continue
        while r < last:
            t = int(tokens[r + 1])
            if not (0 <= t < p.shape[1]) or not float(u_accept[r]) * (1.0 if q is None else float(q[r, t])) < float(p[r, t]):
                break
            r += 1
        w = np.nan_to_num(np.asarray(p[r], np.float64), nan=0.0).clip(min=0)
        if r < last:
            if q is None:
                rest = w.copy()
                if 0 <= int(tokens[r + 1]) < len(rest):
                    rest[int(tokens[r + 1])] = 0.0
            else:
                rest = np.nan_to_num(np.asarray(p[r], np.float64) - np.asarray(q[r], np.float64), nan=0.0).clip(min=0)
            w = rest if rest.sum() > 0 else w
        c = np.cumsum(w)
        if c[-1] > 0:
            i = int(np.searchsorted(c, float(u_sample[b]) * c[-1], side="right"))
            token.append(min(i, int(np.nonzero(w)[0][-1])))
        else:
            token.append(-1)
        accepted.append(r - int(cu[b]))
    return np.array(accepted), np.array(token)
