"""NaN in queries, keys and values of the paged cache: where a row sees one its result is NaN, whether one CTA held the
row's keys or several did, and a later token's does not reach the query tiles that do not see it."""
import numpy as np
import pytest
import torch

from test_gpu_ragged import D, _bf, _dev, _i, _step

pytestmark = pytest.mark.gpu


def _attention(kl, Hq, Hkv, bs, shape, q, kp, vp, table, cu, ctx):
    maxb, nb = shape
    rc = kl.RaggedCfg(len(ctx), q.shape[0], bs, maxb, nb)
    ws = torch.empty(kl.kl_ragged_attention_ws_bytes(rc, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
    kl.kl_ragged_attention(rc, Hq, Hkv, D, kl.KL_BF16, q.data_ptr(), kp.data_ptr(), vp.data_ptr(), table.data_ptr(), cu.data_ptr(), ctx.data_ptr(),
                           o.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel())
    assert kl.kl_device_status() == 0
    return o, lse


def _case(seed, reqs, Hq, Hkv, bs):
    rng, n, ctx, table, maxb, nb, kp, vp, cu, T = _step(seed, reqs, Hkv, bs)
    slot = lambda b, p: (int(table[b, p // bs]), p % bs)  # noqa: E731
    return (maxb, nb), _dev(_bf(rng, T, Hq, D)), _dev(kp), _dev(vp), _i(table), _i(cu), _i(ctx), slot


@pytest.mark.parametrize("Hq,Hkv,reqs,row", [
    (8, 1, [(1, 20000)], 0),                       # cut into many pieces
    (64, 8, [(3, 3000), (1, 500)], 2),
    (8, 2, [(1, 20)] * 400, 77),                   # items held whole
])
def test_a_query_of_nan_gives_nan(kl, Hq, Hkv, reqs, row):
    shape, q, kp, vp, table, cu, ctx, _ = _case(1, reqs, Hq, Hkv, 16)
    want, want_lse = _attention(kl, Hq, Hkv, 16, shape, q, kp, vp, table, cu, ctx)
    assert torch.isfinite(want).all() and torch.isfinite(want_lse).all()
    q[row, 1, 5] = float("nan")
    o, lse = _attention(kl, Hq, Hkv, 16, shape, q, kp, vp, table, cu, ctx)
    assert torch.isnan(o[row, 1]).all() and torch.isnan(lse[row, 1])
    want[row, 1], want_lse[row, 1] = o[row, 1], lse[row, 1]
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[row, 1] = False
    assert torch.equal(o[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])


@pytest.mark.parametrize("bs", [16, 5])
@pytest.mark.parametrize("cached", [128 * 160, 128 * 2, 0])
def test_a_key_of_nan_gives_nan(kl, cached, bs):
    """The request's own key, alone in its last key tile (for the longest: alone in a piece)."""
    Hq, Hkv = 8, 1
    shape, q, kp, vp, table, cu, ctx, slot = _case(2, [(1, cached), (1, 40)], Hq, Hkv, bs)
    want, _ = _attention(kl, Hq, Hkv, bs, shape, q, kp, vp, table, cu, ctx)
    kp[slot(0, cached)][0, 3] = float("nan")
    o, lse = _attention(kl, Hq, Hkv, bs, shape, q, kp, vp, table, cu, ctx)
    assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all()
    assert torch.equal(o[1], want[1])


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("bs", [16, 5, 128])
@pytest.mark.parametrize("Hq,Hkv,n,cached,at", [(64, 8, 200, 0, 100), (64, 8, 200, 77, 150), (8, 8, 300, 0, 250), (4, 1, 130, 1000, 40)])
def test_a_later_value_stays_with_the_query_tiles_that_see_it(kl, Hq, Hkv, n, cached, at, bs, value):
    """Query tiles are 128 / (Hq / Hkv) tokens. Tiles that end before the new token `at` keep their bits; the tokens from it
    on get what the formula gives."""
    shape, q, kp, vp, table, cu, ctx, slot = _case(3, [(n, cached), (1, 40)], Hq, Hkv, bs)
    want, _ = _attention(kl, Hq, Hkv, bs, shape, q, kp, vp, table, cu, ctx)
    vp[slot(0, cached + at)][0, 3] = value
    o, _ = _attention(kl, Hq, Hkv, bs, shape, q, kp, vp, table, cu, ctx)
    G = Hq // Hkv
    before = at // (128 // G) * (128 // G)
    assert torch.equal(o[:before], want[:before])
    assert torch.equal(o[n], want[n])
    assert not torch.isfinite(o[at:n, :G, 3]).any()
    others = torch.arange(D, device="cuda") != 3
    assert torch.equal(o[at:][..., others], want[at:][..., others])


@pytest.mark.parametrize("bs", [16, 5])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_later_key_reaches_no_earlier_token(kl, bs, value):
    Hq, Hkv, n, at = 64, 8, 200, 100
    shape, q, kp, vp, table, cu, ctx, slot = _case(4, [(n, 30)], Hq, Hkv, bs)
    want, _ = _attention(kl, Hq, Hkv, bs, shape, q, kp, vp, table, cu, ctx)
    kp[slot(0, 30 + at)][:, 3] = value
    o, _ = _attention(kl, Hq, Hkv, bs, shape, q, kp, vp, table, cu, ctx)
    assert torch.equal(o[:at], want[:at])


@pytest.mark.parametrize("B,Hq,Hkv,n_new,ctx", [
    (1, 64, 8, 1, 2000),          # context split over CTAs
    (40, 64, 8, 1, 700),          # some items whole, some cut
    (64, 8, 1, 1, 40),
    (3, 12, 4, 3, 190),
])
def test_a_query_or_key_of_nan_in_the_uniform_step(kl, B, Hq, Hkv, n_new, ctx):
    bs = 16
    shape, q, kp, vp, table, cu, ctxd, slot = _case(5, [(n_new, ctx)] * B, Hq, Hkv, bs)
    kp, vp = torch.nan_to_num(kp), torch.nan_to_num(vp)
    table = table.clamp(max=shape[1] - 1)
    pc = kl.PagedCfg(B, n_new, bs, *shape)
    ws = torch.empty(max(256, kl.kl_paged_attention_ws_bytes(pc, Hq, Hkv, D)), dtype=torch.uint8, device="cuda")

    def call():
        o, lse = torch.zeros_like(q), torch.zeros(B, Hq, n_new, device="cuda")
        kl.kl_paged_attention(pc, Hq, Hkv, D, kl.KL_BF16, q.data_ptr(), kp.data_ptr(), vp.data_ptr(), table.data_ptr(), ctxd.data_ptr(), o.data_ptr(), lse.data_ptr(),
                              ws.data_ptr(), ws.numel())
        assert kl.kl_device_status() == 0
        return o.view(B, n_new, Hq, D), lse

    want, want_lse = call()
    for b in range(0, B, 7):                       # every seventh sequence has a NaN query in head 1 of its last token
        q.view(B, n_new, Hq, D)[b, -1, 1, 5] = float("nan")
    o, lse = call()
    keep = torch.ones(B, n_new, Hq, dtype=torch.bool, device="cuda")
    keep[::7, -1, 1] = False
    assert torch.isnan(o[~keep]).all() and torch.isnan(lse.transpose(1, 2)[~keep]).all()
    assert torch.equal(o[keep], want[keep]) and torch.equal(lse.transpose(1, 2)[keep], want_lse.transpose(1, 2)[keep])
    # a NaN in the last key: every head of its kv head in the last token
    q.copy_(torch.nan_to_num(q))
    kp[slot(B - 1, ctx + n_new - 1)][0, 3] = float("nan")
    o, lse = call()
    G = Hq // Hkv
    assert torch.isnan(o[B - 1, -1, :G]).all() and torch.isnan(lse[B - 1, :G, -1]).all()
