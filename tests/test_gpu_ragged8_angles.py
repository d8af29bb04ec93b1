"""The 8-bit append's rotation at far positions: codes and queries that fp32 arithmetic gives, but for values that lie within its error
of the middle between two."""
import numpy as np
import pytest
import torch

import oracle as O
from test_gpu_ragged import D, _bf, _dev, _host, _i
from test_gpu_ragged8 import _append, _codes, _f

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("far", [100, 1 << 20])
def test_codes_and_queries_are_the_nearest(kl, far, inter):
    """Sine and cosine are off by 2^-23.3, each product and their sum by 2^-24 of themselves: 2^-22 (|x| + |z|) in all for a plane (x, z),
    beside half a step of the result's type."""
    Hq, Hkv, bs, T = 8, 8, 16, 4000
    rng = np.random.default_rng(far)
    q, k, v = (_bf(rng, T, h, D) for h in (Hq, Hkv, Hkv))
    pos, nb = rng.integers(0, far, T), T // bs
    pools = [_codes(np.zeros((nb, bs, Hkv, D))), _codes(np.zeros((nb, bs, Hkv, D))), _f(np.ones((nb, Hkv))), _f(np.ones((nb, Hkv)))]
    out = _append(kl, kl.RaggedCfg(1, T, bs, 4, nb), Hq, Hkv, _dev(q), _dev(k), _dev(v), _i([0, T]), _i(pos), _i(np.arange(T)), pools, inter=int(inter))
    assert kl.kl_device_status() == 0

    def turned(x):
        y = O.rope_at(x, pos, 1e6, inter)
        a = np.abs(x)
        pair = np.repeat(a[..., 0::2] + a[..., 1::2], 2, -1) if inter else np.concatenate([a[..., :D // 2] + a[..., D // 2:]] * 2, -1)
        return y, 2.0 ** -22 * pair

    y, off = turned(q)
    half = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y) + off, 1e-30))) - 8)
    assert (np.abs(_host(out) - y) <= half + off).all()
    y, off = turned(k)
    scale = np.repeat(_host(pools[2]), bs, 0)[..., None]
    err = np.abs(_host(pools[0]).reshape(T, Hkv, D) * scale - y)
    tol = O.e4m3_half_step((np.abs(y) + off) / scale) * scale + off
    assert (err <= tol).all(), int((err > tol).sum())
