"""The ragged step's operators together, in the ways a server runs them: a pool that runs short."""
import numpy as np
import pytest
import torch

import oracle as O
from _parity import TOL_BF16, assert_rel
from test_gpu_ragged import D, Planner, _bf, _dev, _host, _i

pytestmark = pytest.mark.gpu


def test_a_step_of_a_pool_that_runs_short(kl):
    """Three requests, blocks for two: the plan counts what is missing and reports no error, the granted requests' rows are
    right, the third's read zeros for the blocks it lacks (reported); fed again when there are blocks it is right too."""
    B, T, bs, maxb, nb, Hq, Hkv = 3, 80, 8, 6, 7, 8, 2
    rng = np.random.default_rng(3)
    s = Planner(kl, B, T, bs, maxb, nb, rng.permutation(nb), nb)
    kp, vp = (torch.full((nb, bs, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.empty(kl.kl_ragged_attention_ws_bytes(s.rc, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    tokens = [[_bf(rng, 40, h, D) for h in (Hq, Hkv, Hkv)] for _ in range(B)]      # each request's q, k and v by position
    ctx = np.zeros(B, int)

    def step(n):
        r = s.step(n, ctx)
        rows = [np.concatenate([np.zeros((0, h, D))] + [tokens[b][j][ctx[b]:ctx[b] + max(n[b], 0)] for b in range(B)]) for j, h in enumerate((Hq, Hkv, Hkv))]
        q, k, v = (_dev(np.concatenate([x, np.full((T - len(x),) + x.shape[1:], np.nan)])) for x in rows)
        o = torch.full_like(q, 7.0)
        kl.kl_ragged_qkv_rope(s.rc, Hq, Hkv, D, kl.KL_BF16, q.data_ptr(), k.data_ptr(), v.data_ptr(), 0, 0, 1e-6, 1e4, 0, s.cu.data_ptr(), s.pos.data_ptr(), s.slots.data_ptr(),
                              q.data_ptr(), kp.data_ptr(), vp.data_ptr())
        kl.kl_ragged_attention(s.rc, Hq, Hkv, D, kl.KL_BF16, q.data_ptr(), kp.data_ptr(), vp.data_ptr(), s.d["table"].data_ptr(), s.cu.data_ptr(), s.ctx.data_ptr(), o.data_ptr(),
                               0, ws.data_ptr(), ws.numel())
        torch.cuda.synchronize()
        return r, q, o

    def check(r, q, o, b):
        x = slice(int(r["cu"][b]), int(r["cu"][b + 1]))
        end = ctx[b] + x.stop - x.start
        k = O.rope_at(tokens[b][1][:end], np.arange(end), 1e4)
        want, _, A = O.ragged_attention(_host(q)[x], k[:, None], tokens[b][2][:end, None], np.arange(end)[None], [0, x.stop - x.start], [ctx[b]])
        # the cache holds k rounded to bf16, which moves a score by 2^-9 |q k| / sqrt(d) a product, 128 of them with random
        # signs: 2^-9; the weights and the result are bf16 too (2^-9 each on average): 6e-3 in all
        assert_rel(_host(o)[x], want, TOL_BF16, f"request {b}")

    r, q, o = step([5, 17, 3])                       # 1 + 3 + 1 blocks
    assert r["missing"] == 0 and kl.kl_device_status() == 0
    for b in range(B):
        check(r, q, o, b)
    ctx += [5, 17, 3]
    n = [4, 4, 20]                                   # 1 + 0 + 2 blocks: two are left
    r, q, o = step(n)
    assert r["missing"] == 2
    with pytest.raises(kl.KLError) as e:             # the attention's: the plan itself reports none
        kl.kl_device_status()
    assert e.value.status == kl.KL_ERR_DEVICE and "0x8" in str(e.value)
    check(r, q, o, 0)
    check(r, q, o, 1)
    x = slice(int(r["cu"][2]), int(r["cu"][3]))
    assert (r["slots"][x][:5] >= 0).all() and (r["slots"][x][5:] == -1).all()
    check(dict(cu=[0, 0, x.start, x.start + 5]), q, o, 2)     # the rows that see held blocks only
    assert torch.isfinite(o[x]).all()
    assert (o[x.stop:] == 7.0).all()
    ctx += [4, 4, 0]
    r, q, o = step([0, -1, 0])                       # request 1 ends
    assert r["missing"] == 0 and kl.kl_device_status() == 0
    ctx[1] = 0
    r, q, o = step([1, 0, 20])                       # the same tokens again
    assert r["missing"] == 0 and kl.kl_device_status() == 0
    check(r, q, o, 0)
    check(r, q, o, 2)


def test_plan_alone_reports_no_error_for_a_short_pool(kl):
    s = Planner(kl, 2, 20, 4, 4, 3, np.arange(3), 3)
    assert s.step([8, 8], [0, 0])["missing"] == 2
    assert kl.kl_device_status() == 0
