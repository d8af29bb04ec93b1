"""The precision of draft verification's sums over long rows."""
import numpy as np
import pytest
import torch

from test_gpu_ragged import _verify

pytestmark = pytest.mark.gpu

V = 1 << 24


def _plain_pair(x):
    """x summed one by one into hi with each addition's error into lo, all in fp32: the error against the exact sum."""
    hi, lo = np.float32(0), np.float32(0)
    for v in x:
        s = np.float32(hi + v)
        b = np.float32(s - hi)
        lo = np.float32(lo + np.float32(np.float32(hi - np.float32(s - b)) + np.float32(v - b)))
        hi = s
    return float(hi) + float(lo) - float(x.astype(np.float64).sum())


def _one_lane(elements):
    """Weights for one lane: 0.5 and many below half a step of it, all multiples of 2^-48, so every sum of them is exact in
    fp64. Their exact sum C lies 2^-33 below the fp32 number W."""
    # rounding a running error sum in its last binade (2^-15 .. 2^-14 for 2048 elements) to 24 bits gains 0.4 of a step
    step = 2.0 ** (np.floor(np.log2(elements * 2.0 ** -25.2)) - 23)
    w = (np.floor(2.0 ** -25.2 / step) + 0.6) * step
    w = np.float32(np.round(w * 2.0 ** 48) * 2.0 ** -48)
    c = 0.5 + (elements - 2) * float(w)
    W = np.float32(np.ceil((c + 2.0 ** -33) * 2.0 ** 24) * 2.0 ** -24)
    last = float(W) - 2.0 ** -33 - c
    assert 0 <= last < 2.0 ** -24 and np.float32(last) == last
    x = np.concatenate([[np.float32(0.5)], np.full(elements - 2, w, np.float32), [np.float32(last)]])
    assert x.astype(np.float64).sum() == float(W) - 2.0 ** -33
    return x, W


# requests, CTAs a request, warps a CTA; elements a vector (one where p and q start at different places of it)
@pytest.mark.parametrize("B,ctas,warps", [(1, 16, 16), (10, 8, 16), (20, 8, 8)])
@pytest.mark.parametrize("given_q,E", [(False, 4), (True, 4), (True, 1)])
def test_a_long_sum_next_to_its_mark(kl, B, ctas, warps, given_q, E):
    """u = 0.5 and two weights' worth: C in one lane's share, W = C + 2^-33 at the row's end. The sum of all up to W's
    place is C < (C + W) / 2, so the token is W's. Were C off by more than 2^-33, it would be one of the lane's. The header
    promises 2^-41 of the sum."""
    lanes = [5 + 32 * i for i in range(V // E // ctas // warps // 32)]
    cols = np.array([j * E + e for j in lanes for e in range(E)])
    x, W = _one_lane(len(cols))
    assert _plain_pair(x) > 2.0 ** -32               # what a sum without care loses here
    # request 0 has a rejected draft (probability zero) where q is given; its rows start at `first`
    first, rows = (1, B + 2) if E == 1 else (0, B + 1)
    p = torch.zeros(rows, V, device="cuda")
    p[first, torch.as_tensor(cols, device="cuda")] = torch.as_tensor(x, device="cuda")
    p[first, V - 2] = float(W)
    cu = np.concatenate([[first], first + 2 + np.arange(B)]) if given_q else first + np.arange(B + 1)
    q = torch.zeros(rows * (V + 1), device="cuda") if given_q else None
    us = np.full(B, 0.5, np.float32)
    acc, nxt = _verify(kl, p, q, np.full(rows, V - 1), cu, np.full(rows, 0.5, np.float32), us, ldq=(V + 1 if E == 1 else V) if given_q else None)
    assert kl.kl_device_status() == 0
    assert acc[0] == 0 and nxt[0] == V - 2
    assert (nxt[1:] == -1).all()
