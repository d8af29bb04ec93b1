"""The ragged step over the paged cache through the C ABI against the fp64 oracle (oracle/ragged.py): planning (exact),
norm + rotation + cache write, attention, draft verification (exact), and the four together in a captured step."""
import numpy as np
import pytest
import torch

import oracle as O
from bwd_qwen3_layer_gb300 import layer as L
from bwd_qwen3_layer_gb300 import synth
from _parity import TOL_BF16, assert_rel

pytestmark = pytest.mark.gpu

D = 128


def _i(a):
    return torch.as_tensor(np.ascontiguousarray(a).astype(np.int32)).cuda()


def _bf(rng, *shape):
    """Random values that bf16 holds, on the host."""
    return synth.round_bf16(rng.standard_normal(shape))


def _dev(a):
    return torch.as_tensor(a).to(torch.bfloat16).cuda()


def _host(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------

class Planner:
    """A server's state on the device and the same on the host, stepped together."""

    def __init__(self, kl, B, T, bs, max_blocks, n_blocks, free, n_free):
        self.kl, self.bs, self.T, self.B = kl, bs, T, B
        self.rc = kl.RaggedCfg(B, T, bs, max_blocks, n_blocks)
        self.table, self.held = np.full((B, max_blocks), -1), np.zeros(B, int)
        self.free, self.n_free = np.array(free), n_free
        self.d = dict(table=_i(self.table), held=_i(self.held), free=_i(self.free), n_free=_i([n_free]))
        self.cu, self.pos, self.slots, self.missing = _i(np.full(B + 1, -7)), _i(np.full(T, -7)), _i(np.full(T, -7)), _i([-7])
        self.new, self.ctx = _i(np.zeros(B)), _i(np.zeros(B))

    def launch(self):
        d = self.d
        self.kl.kl_ragged_plan(self.rc, self.new.data_ptr(), self.ctx.data_ptr(), d["table"].data_ptr(), d["held"].data_ptr(), d["free"].data_ptr(),
                               d["n_free"].data_ptr(), self.cu.data_ptr(), self.pos.data_ptr(), self.slots.data_ptr(), self.missing.data_ptr())

    def step(self, n, ctx, launch=None):
        self.new.copy_(_i(n))
        self.ctx.copy_(_i(ctx))
        before = self.pos.cpu().numpy(), self.slots.cpu().numpy()
        (launch or self.launch)()
        torch.cuda.synchronize()
        r = O.ragged_plan(n, ctx, self.table, self.held, self.free, self.n_free, self.bs, self.T)
        self.table, self.held, self.free, self.n_free = r["table"], r["held"], r["free_list"], r["n_free"]
        rows = len(r["pos"])
        for got, want in ((self.cu, r["cu"]), (self.pos[:rows], r["pos"]), (self.slots[:rows], r["slots"]), (self.d["table"], r["table"]),
                          (self.d["held"], r["held"]), (self.d["free"], r["free_list"]), (self.d["n_free"], [r["n_free"]]), (self.missing, [r["missing"]])):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        # rows behind the last stay as they were
        np.testing.assert_array_equal(self.pos.cpu().numpy()[rows:], before[0][rows:])
        np.testing.assert_array_equal(self.slots.cpu().numpy()[rows:], before[1][rows:])
        return r


@pytest.mark.parametrize("B,bs,maxb,nb,T,most", [
    (1, 16, 4, 4, 70, 20),          # one request
    (7, 1, 40, 150, 100, 6),        # pages of one token
    (33, 5, 12, 200, 700, 20),      # odd pages; the pool runs out
    (64, 16, 20, 2000, 5000, 60),   # eight CTAs (rows)
    (1500, 16, 6, 4000, 4000, 3),   # eight CTAs (requests), two rounds of 1024 requests; the pool runs out
])
def test_plan_matches_oracle_over_steps(kl, B, bs, maxb, nb, T, most):
    rng = np.random.default_rng(B)
    s = Planner(kl, B, T, bs, maxb, nb, rng.permutation(nb), nb)
    ctx = np.zeros(B, int)
    for _ in range(12):
        n = np.where(rng.random(B) < 0.15, -1, np.minimum(rng.integers(0, most + 1, B), maxb * bs - ctx))
        r = s.step(n, ctx)
        got = np.array([(r["slots"][r["cu"][b]:r["cu"][b + 1]] >= 0).all() for b in range(B)])
        # a third of the drafted rows are taken back: a request then holds more than its context fills
        kept = np.where(rng.random(B) < 0.3, np.maximum(n, 0) // 2, np.maximum(n, 0))
        ctx = np.where(n < 0, 0, np.where(got, ctx + kept, ctx))
    assert kl.kl_device_status() == 0


def test_plan_reports_rows_and_positions_that_do_not_fit(kl):
    s = Planner(kl, 3, 10, 4, 3, 20, np.arange(20), 20)
    s.step([4, 4, 4], [0, 0, 0])                 # 12 rows in room for 10: two dropped
    with pytest.raises(kl.KLError) as e:
        kl.kl_device_status()
    assert e.value.status == kl.KL_ERR_DEVICE and "0x10" in str(e.value)
    s = Planner(kl, 2, 20, 4, 3, 20, np.arange(20), 20)
    s.step([15, 2], [0, 0])                      # 15 tokens, a table of 12
    with pytest.raises(kl.KLError) as e:
        kl.kl_device_status()
    assert "0x8" in str(e.value)
    assert kl.kl_device_status() == 0


# ---------------------------------------------------------------------------
# a step's data
# ---------------------------------------------------------------------------

def _step(seed, reqs, Hkv, bs, extra_rows=0):
    """reqs: (new, cached) tokens. Tables over a shuffled pool; NaN in every slot behind a request's end and in the blocks
    that nobody has; table entries past a request's blocks lie outside the pool."""
    rng = np.random.default_rng(seed)
    n, ctx = np.array([r[0] for r in reqs]), np.array([r[1] for r in reqs])
    blocks = -(-(n + ctx) // bs)
    maxb, nb = int(max(1, blocks.max())) + 1, int(blocks.sum()) + 3
    order = rng.permutation(nb)
    table, at = np.full((len(reqs), maxb), nb + 5), 0
    kp, vp = np.full((nb, bs, Hkv, D), np.nan), np.full((nb, bs, Hkv, D), np.nan)
    for b in range(len(reqs)):
        table[b, :blocks[b]] = order[at:at + blocks[b]]
        at += blocks[b]
        p = np.arange(n[b] + ctx[b])
        kp[table[b][p // bs], p % bs] = _bf(rng, len(p), Hkv, D)
        vp[table[b][p // bs], p % bs] = _bf(rng, len(p), Hkv, D)
    cu = np.concatenate([[0], np.cumsum(n)])
    return rng, n, ctx, table, maxb, nb, kp, vp, cu, int(cu[-1]) + extra_rows


ATTENTION = [
    (8, 1, 16, [(1, 0)]),                                             # one token, one key
    (8, 8, 16, [(1, 0), (1, 126), (1, 127), (1, 128), (1, 255)]),     # no shared heads; around the key tile's edge
    (64, 8, 16, [(1, 300), (5, 0), (130, 64), (0, 77), (17, 1000)]),  # decode, drafts, chunks and an idle request
    (12, 4, 5, [(3, 7), (1, 0), (2, 190), (90, 3)]),                  # three heads a group, pages of five
    (10, 2, 24, [(1, 500), (60, 100), (26, 0)]),                      # five heads: 25 tokens a tile; pages end inside a key tile
    (7, 1, 8, [(40, 13), (19, 0), (1, 1000)]),                        # seven heads: two rows of a tile unused
    (16, 2, 128, [(300, 0), (1, 129)]),
    (4, 2, 256, [(257, 200), (3, 511)]),                              # pages longer than a key tile
    (4, 1, 1, [(5, 130), (1, 64)]),                                   # pages of one token
    (8, 1, 16, [(1, 20000)]),                                         # one long context: cut into many pieces
    (128, 1, 16, [(3, 200)]),                                         # a tile holds one token
    (8, 2, 16, [(700, 500), (1, 30), (1, 4000)]),
    (64, 8, 16, [(1, 40 * i % 900) for i in range(64)]),              # a decoding batch
]


@pytest.mark.parametrize("Hq,Hkv,bs,reqs", ATTENTION)
def test_attention_matches_oracle(kl, Hq, Hkv, bs, reqs):
    rng, n, ctx, table, maxb, nb, kp, vp, cu, T = _step(5, reqs, Hkv, bs, extra_rows=3)
    q = _bf(rng, T, Hq, D)
    want, want_lse, A = O.ragged_attention(q[:T - 3], kp, vp, table, cu, ctx)
    rc = kl.RaggedCfg(len(reqs), T, bs, maxb, nb)
    qd, kd, vd, td, cd, xd = _dev(q), _dev(kp), _dev(vp), _i(table), _i(cu), _i(ctx)
    ws = torch.empty(kl.kl_ragged_attention_ws_bytes(rc, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    outs = []
    for use_lse in (True, False, True):
        o = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((T, Hq), 7.0, device="cuda")
        kl.kl_ragged_attention(rc, Hq, Hkv, D, kl.KL_BF16, qd.data_ptr(), kd.data_ptr(), vd.data_ptr(), td.data_ptr(), cd.data_ptr(), xd.data_ptr(),
                               o.data_ptr(), lse.data_ptr() if use_lse else 0, ws.data_ptr(), ws.numel())
        assert kl.kl_device_status() == 0
        outs.append((o, lse))
    got, got_lse = _host(outs[0][0]), _host(outs[0][1])
    # Each weight enters its product as bf16 (off by 2^-8 of itself at most: 2^-8 A in all), the result leaves as bf16 (2^-8 |o|).
    # fp32 sums: 128 products of a score, 128 x 2^-24 x sum |q k| / sqrt(d) < 1e-4 (sum |q k| < 130), twice (weights and their
    # sum); at most 2^15 keys, whose running sums stay below 2^15 x 2^-24 = 2^-9 of A.
    tol = (2.0 ** -8 + 2.0 ** -9 + 2e-4) * A + 2.0 ** -8 * np.abs(want)
    assert (np.abs(got[:T - 3] - want) <= tol).all(), np.max(np.abs(got[:T - 3] - want) / tol)
    assert_rel(got[:T - 3], want, 2.0 ** -7, "O")
    L_max = max(a + b for a, b in reqs)
    assert np.max(np.abs(got_lse[:T - 3] - want_lse), initial=0) <= 1e-4 + L_max * 2.0 ** -24
    # rows behind the last request stay as they were; the same bits again, with and without lse
    assert (got[T - 3:] == 7.0).all() and (got_lse[T - 3:] == 7.0).all()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][0], outs[2][0]) and torch.equal(outs[0][1], outs[2][1])
    assert (outs[1][1] == 7.0).all()


def test_attention_equals_the_uniform_paged_attention(kl):
    """A batch that both entry points take: within two bf16 roundings of weights and results of each other."""
    B, n, Hq, Hkv, bs = 5, 4, 8, 2, 16
    reqs = [(n, c) for c in (0, 5, 130, 700, 64)]
    rng, _, ctx, table, maxb, nb, kp, vp, cu, T = _step(6, reqs, Hkv, bs)
    q = _bf(rng, T, Hq, D)
    kp, vp = np.nan_to_num(kp), np.nan_to_num(vp)
    qd, kd, vd, td, cd, xd = _dev(q), _dev(kp), _dev(vp), _i(np.minimum(table, nb - 1)), _i(cu), _i(ctx)
    a, b = torch.empty_like(qd), torch.empty_like(qd)
    rc, pc = kl.RaggedCfg(B, T, bs, maxb, nb), kl.PagedCfg(B, n, bs, maxb, nb)
    ws = torch.empty(kl.kl_ragged_attention_ws_bytes(rc, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    w2 = torch.empty(max(256, kl.kl_paged_attention_ws_bytes(pc, Hq, Hkv, D)), dtype=torch.uint8, device="cuda")
    kl.kl_ragged_attention(rc, Hq, Hkv, D, kl.KL_BF16, qd.data_ptr(), kd.data_ptr(), vd.data_ptr(), td.data_ptr(), cd.data_ptr(), xd.data_ptr(), a.data_ptr(), 0,
                           ws.data_ptr(), ws.numel())
    kl.kl_paged_attention(pc, Hq, Hkv, D, kl.KL_BF16, qd.data_ptr(), kd.data_ptr(), vd.data_ptr(), td.data_ptr(), xd.data_ptr(), b.data_ptr(), 0, w2.data_ptr(), w2.numel())
    assert kl.kl_device_status() == 0
    _, _, A = O.ragged_attention(q, kp, vp, table, cu, ctx)
    assert (np.abs(_host(a) - _host(b)) <= 2 * (2.0 ** -8 + 2.0 ** -9) * A + 2 * 2.0 ** -8 * np.abs(_host(a))).all()


@pytest.mark.parametrize("bs", [16, 5])
def test_attention_reports_pages_outside_the_pool(kl, bs):
    """A bad table entry reads as zero keys and values and is reported; other requests are not touched by it."""
    reqs, Hq, Hkv = [(2, 60), (3, 300)], 8, 2
    rng, n, ctx, table, maxb, nb, kp, vp, cu, T = _step(7, reqs, Hkv, bs)
    q = _bf(rng, T, Hq, D)
    bad = table.copy()
    bad[0, 1] = -1
    bad[0, 2] = nb
    rc = kl.RaggedCfg(2, T, bs, maxb, nb)
    qd, kd, vd, td, cd, xd = _dev(q), _dev(kp), _dev(vp), _i(bad), _i(cu), _i(ctx)
    o = torch.empty_like(qd)
    ws = torch.empty(kl.kl_ragged_attention_ws_bytes(rc, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    kl.kl_ragged_attention(rc, Hq, Hkv, D, kl.KL_BF16, qd.data_ptr(), kd.data_ptr(), vd.data_ptr(), td.data_ptr(), cd.data_ptr(), xd.data_ptr(), o.data_ptr(), 0,
                           ws.data_ptr(), ws.numel())
    with pytest.raises(kl.KLError) as e:
        kl.kl_device_status()
    assert e.value.status == kl.KL_ERR_DEVICE and "0x8" in str(e.value)
    # the same as a pool with zero blocks there
    zk, zv = np.concatenate([kp, np.zeros((1,) + kp.shape[1:])]), np.concatenate([vp, np.zeros((1,) + vp.shape[1:])])
    z = np.where((bad < 0) | (bad == nb), nb, bad)
    want, _, A = O.ragged_attention(q, zk, zv, z, cu, ctx)
    tol = (2.0 ** -8 + 2.0 ** -9 + 2e-4) * A + 2.0 ** -8 * np.abs(want)
    assert (np.abs(_host(o) - want) <= tol).all()


def test_attention_does_not_depend_on_the_block_size(kl):
    """Runs of some fifty key tiles a CTA: the same cache in pages of 8 to 256 tokens and of sizes that are gathered row by row gives the same bits."""
    Hq, Hkv, reqs = 64, 8, [(1, 39990), (3, 40001), (1, 37777)]
    g = torch.Generator(device="cuda").manual_seed(9)
    q = torch.randn(5, Hq, D, generator=g, device="cuda").bfloat16()
    kv = [[torch.randn(a + c, Hkv, D, generator=g, device="cuda").bfloat16() for a, c in reqs] for _ in range(2)]
    cu, ctx = _i([0, 1, 4, 5]), _i([c for _, c in reqs])
    first = None
    for bs in (16, 8, 32, 40, 128, 256, 20, 1):
        per = [-(-(a + c) // bs) for a, c in reqs]
        maxb, nb = max(per) + 1, sum(per) + 2
        order = torch.randperm(nb, generator=g, device="cuda")
        table = torch.full((3, maxb), nb + 9, device="cuda")
        pools = [torch.full((nb * bs, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        at = 0
        for b, (a, c) in enumerate(reqs):
            table[b, :per[b]] = order[at:at + per[b]]
            at += per[b]
            pos = torch.arange(a + c, device="cuda")
            for pool, x in zip(pools, kv):
                pool[table[b, pos // bs] * bs + pos % bs] = x[b]
        td = table.to(torch.int32)
        rc = kl.RaggedCfg(3, 5, bs, maxb, nb)
        ws = torch.empty(kl.kl_ragged_attention_ws_bytes(rc, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
        o = torch.empty_like(q)
        kl.kl_ragged_attention(rc, Hq, Hkv, D, kl.KL_BF16, q.data_ptr(), pools[0].data_ptr(), pools[1].data_ptr(), td.data_ptr(), cu.data_ptr(), ctx.data_ptr(), o.data_ptr(),
                               0, ws.data_ptr(), ws.numel())
        assert kl.kl_device_status() == 0
        if first is None:
            first = o
        assert torch.equal(o, first), bs
    for b, (a, c) in enumerate(reqs):
        r0 = int(cu[b])
        for i in range(a):
            k, v = (x[b][:c + i + 1].double() for x in kv)
            qi = q[r0 + i].double().reshape(Hkv, Hq // Hkv, D)
            w = torch.softmax(torch.einsum("hgd,khd->hgk", qi, k) / D ** 0.5, -1)
            want, A = (torch.einsum("hgk,khd->hgd", w, x).reshape(Hq, D) for x in (v, v.abs()))
            # as in test_attention_matches_oracle, with running sums of up to 2^16 keys
            tol = (2.0 ** -8 + 2.0 ** -8 + 2e-4) * A + 2.0 ** -8 * want.abs()
            assert ((first[r0 + i].double() - want).abs() <= tol).all(), (b, i)


def test_attention_without_rows(kl):
    rc = kl.RaggedCfg(3, 4, 16, 2, 4)
    q = torch.randn(4, 8, D, device="cuda").bfloat16()
    pool = torch.randn(4, 16, 1, D, device="cuda").bfloat16()
    o = torch.full_like(q, 3.0)
    cu, ctx, table = _i([0, 0, 0, 0]), _i([5, 0, 9]), _i(np.zeros((3, 2)))
    ws = torch.empty(kl.kl_ragged_attention_ws_bytes(rc, 8, 1, D), dtype=torch.uint8, device="cuda")
    kl.kl_ragged_attention(rc, 8, 1, D, kl.KL_BF16, q.data_ptr(), pool.data_ptr(), pool.data_ptr(), table.data_ptr(), cu.data_ptr(), ctx.data_ptr(), o.data_ptr(), 0,
                           ws.data_ptr(), ws.numel())
    assert kl.kl_device_status() == 0
    assert (o == 3.0).all()


# ---------------------------------------------------------------------------
# norm, rotation, cache write
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("Hq,Hkv,bs,reqs,norm,inter,inplace", [
    (8, 1, 16, [(1, 0)], False, False, False),
    (64, 8, 16, [(1, 300), (5, 100000), (0, 7), (33, 64)], True, False, False),
    (12, 4, 5, [(3, 7), (2, 190)], True, True, True),
    (7, 7, 24, [(9, 23)], False, True, False),
    (128, 1, 8, [(2, 5)], True, False, True),
    # more rows than the GPU holds at once, more heads than a CTA holds at once
    (8, 1, 16, [(700, 3), (0, 1), (33, 64)], False, False, True),
    (10, 2, 16, [(1, 9), (900, 0), (310, 70000)], True, True, False),
    (40, 40, 32, [(650, 20)], True, False, False),
    (100, 100, 64, [(620, 1)], True, False, False),
])
def test_qkv_matches_oracle(kl, Hq, Hkv, bs, reqs, norm, inter, inplace):
    rng = np.random.default_rng(8)
    n, ctx = np.array([r[0] for r in reqs]), np.array([r[1] for r in reqs])
    T = int(n.sum())
    pos = np.concatenate([np.arange(c, c + k) for k, c in reqs])
    nb = T // bs + 4
    slots = rng.permutation(nb * bs)[:T]
    if T > 2:
        slots[1] = -1                            # a row without a block
    qp, kp_, v = _bf(rng, T + 2, Hq, D), _bf(rng, T + 2, Hkv, D), _bf(rng, T + 2, Hkv, D)
    gq, gk = synth.round_bf16(1 + 0.2 * rng.standard_normal(D)), synth.round_bf16(1 + 0.2 * rng.standard_normal(D))
    kp, vp = _bf(rng, nb, bs, Hkv, D), _bf(rng, nb, bs, Hkv, D)
    eps, base = 1e-6, 1e6

    def want(x, g):
        x = x[:T]
        if norm:
            x = O.rmsnorm_fwd(x, g, eps)[0]
        return O.rope_at(x, pos, base, inter), np.abs(x) + np.abs(O.rope_at(x, np.zeros(T), base, inter))

    (wq, _), (wk, _) = want(qp, gq), want(kp_, gk)
    rc = kl.RaggedCfg(len(reqs), T + 2, bs, 4, nb)
    qd, kd, vd, gqd, gkd, kpd, vpd = _dev(qp), _dev(kp_), _dev(v), _dev(gq), _dev(gk), _dev(kp), _dev(vp)
    out = qd if inplace else torch.full_like(qd, 7.0)
    cu, pd, sd = _i(np.concatenate([[0], np.cumsum(n)])), _i(np.concatenate([pos, [3, 4]])), _i(np.concatenate([slots, [0, 1]]))
    kl.kl_ragged_qkv_rope(rc, Hq, Hkv, D, kl.KL_BF16, qd.data_ptr(), kd.data_ptr(), vd.data_ptr(), gqd.data_ptr() if norm else 0, gkd.data_ptr() if norm else 0, eps, base,
                          int(inter), cu.data_ptr(), pd.data_ptr(), sd.data_ptr(), out.data_ptr(), kpd.data_ptr(), vpd.data_ptr())
    assert kl.kl_device_status() == 0
    kref, vref = kp.reshape(-1, Hkv, D).copy(), vp.reshape(-1, Hkv, D).copy()
    rows = slots >= 0
    kref[slots[rows]], vref[slots[rows]] = wk[rows], v[:T][rows]

    def close(got, ref, scale):
        # one rounding to bf16 (2^-8), and before it fp32: 128 squares (2^-18 of the root), a few products, an angle good to
        # 2^-22: below 2^-16 of the pair's size, which is at most the head's largest value times two
        tol = 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -7) + 2.0 ** -16 * 2 * scale
        assert (np.abs(got - ref) <= tol).all(), np.max(np.abs(got - ref) / tol)

    close(_host(out)[:T], wq, np.abs(wq).max(-1, keepdims=True))
    got_k, got_v = _host(kpd).reshape(-1, Hkv, D), _host(vpd).reshape(-1, Hkv, D)
    close(got_k[slots[rows]], kref[slots[rows]], np.abs(wk[rows]).max(-1, keepdims=True))
    untouched = np.setdiff1d(np.arange(nb * bs), slots[rows])
    assert (got_k[untouched] == kref[untouched]).all()
    assert (got_v == vref).all()
    # rows behind the last request stay as they were
    assert (_host(out)[T:] == (qp[T:] if inplace else 7.0)).all()


def test_qkv_reports_a_slot_past_the_pool(kl):
    rc = kl.RaggedCfg(1, 2, 16, 2, 2)
    q, k = torch.randn(2, 8, D, device="cuda").bfloat16(), torch.randn(2, 1, D, device="cuda").bfloat16()
    pool = torch.zeros(2, 16, 1, D, device="cuda", dtype=torch.bfloat16)
    cu, pos, slots = _i([0, 2]), _i([0, 1]), _i([32, 5])
    kl.kl_ragged_qkv_rope(rc, 8, 1, D, kl.KL_BF16, q.data_ptr(), k.data_ptr(), k.data_ptr(), 0, 0, 1e-6, 1e6, 0, cu.data_ptr(), pos.data_ptr(), slots.data_ptr(), q.data_ptr(),
                          pool.data_ptr(), pool.data_ptr())
    with pytest.raises(kl.KLError) as e:
        kl.kl_device_status()
    assert "0x8" in str(e.value)
    got = pool.view(32, D)
    assert (got[:5] == 0).all() and (got[6:] == 0).all()


# ---------------------------------------------------------------------------
# verify
# ---------------------------------------------------------------------------

def _verify(kl, p, q, tokens, cu, ua, us, ldp=None, ldq=None):
    T, V = p.shape
    cfg = kl.VerifyCfg(len(cu) - 1, T, V, kl.KL_F32 if p.dtype == torch.float32 else kl.KL_BF16)
    acc, nxt = _i(np.full(len(cu) - 1, -7)), _i(np.full(len(cu) - 1, -7))
    td, cd, uad, usd = _i(tokens), _i(cu), torch.as_tensor(ua).cuda(), torch.as_tensor(us).cuda()
    kl.kl_draft_verify(cfg, p.data_ptr(), ldp or V, kl.ptr(q), ldq or V, td.data_ptr(), cd.data_ptr(), uad.data_ptr(), usd.data_ptr(), acc.data_ptr(), nxt.data_ptr())
    torch.cuda.synchronize()
    return acc.cpu().numpy(), nxt.cpu().numpy()


@pytest.mark.parametrize("V,dtype,given_q,drafts", [
    (1, torch.float32, True, [1, 0]),
    (5, torch.bfloat16, False, [2, 0, 3]),
    (1000, torch.float32, True, [0, 1, 4, 40]),              # more drafts than a warp has lanes
    (32001, torch.bfloat16, True, [3, 7, 0, 1, 2, 4]),       # odd rows: every alignment of a 16-byte vector
    (32003, torch.float32, False, [3, 7, 1, 1, 2, 4]),
    (151936, torch.float32, True, [4] * 6),
    (151936, torch.bfloat16, False, [4] * 6),
])
def test_verify_matches_oracle(kl, V, dtype, given_q, drafts):
    g = torch.Generator(device="cuda").manual_seed(V)
    cu = np.concatenate([[0], np.cumsum([k + 1 for k in drafts])])
    T, B = int(cu[-1]), len(drafts)
    z = torch.randn(T, V, generator=g, device="cuda") * 2
    p = torch.softmax(z, 1).to(dtype)
    q = torch.softmax(z + 0.5 * torch.randn(T, V, generator=g, device="cuda"), 1).to(dtype)
    rng = np.random.default_rng(V)
    for rep in range(3):
        tokens = np.concatenate([[0], torch.multinomial(q.float(), 1, generator=g)[:-1, 0].cpu().numpy()])
        ua, us = rng.random(T).astype(np.float32), rng.random(B).astype(np.float32)
        if rep == 0:
            us[0], us[-1] = 0.0, np.float32(1 - 2.0 ** -24)
        if rep == 2:
            ua[:] = 0.0                                       # all accepted (every probability is above zero)
        got = _verify(kl, p, q if given_q else None, tokens, cu, ua, us)
        want = O.draft_verify(_host(p), _host(q) if given_q else None, tokens, cu, ua, us)
        np.testing.assert_array_equal(got[0], want[0])
        np.testing.assert_array_equal(got[1], want[1])
    assert kl.kl_device_status() == 0


def test_verify_strides_of_their_own(kl):
    """p and q as pieces of wider buffers with different row strides: rows that start at different places of a 16-byte vector."""
    T, V = 6, 997
    g = torch.Generator(device="cuda").manual_seed(3)
    P, Q = torch.rand(T, 1003, generator=g, device="cuda"), torch.rand(T, 1010, generator=g, device="cuda")
    tokens, cu = [0, 5, 700, 1, 996, 3], [0, 3, 6]
    ua, us = np.full(T, 0.9, np.float32), np.array([0.3, 0.8], np.float32)
    cfg = kl.VerifyCfg(2, T, V, kl.KL_F32)
    acc, nxt = _i([9, 9]), _i([9, 9])
    td, cd, uad, usd = _i(tokens), _i(cu), torch.as_tensor(ua).cuda(), torch.as_tensor(us).cuda()
    kl.kl_draft_verify(cfg, P.data_ptr(), 1003, Q.data_ptr(), 1010, td.data_ptr(), cd.data_ptr(), uad.data_ptr(), usd.data_ptr(), acc.data_ptr(), nxt.data_ptr())
    want = O.draft_verify(_host(P)[:, :V], _host(Q)[:, :V], tokens, cu, ua, us)
    assert kl.kl_device_status() == 0
    np.testing.assert_array_equal(acc.cpu().numpy(), want[0])
    np.testing.assert_array_equal(nxt.cpu().numpy(), want[1])


def test_verify_corners(kl):
    p = torch.tensor([[0.0, 0.5, 0.5], [0.2, 0.3, 0.5], [0.0, 0.0, 0.0], [float("nan"), 0.0, 1.0], [float("inf"), 0.0, 1.0]], device="cuda")
    f = np.float32
    one = lambda tokens, cu, ua, us, q=None: [list(x) for x in _verify(kl, p, q, tokens, cu, np.array(ua, f), np.array(us, f))]  # noqa: E731
    z = [0.0] * 5
    assert one([0, 0, 0, 0, 0], [0, 2, 2], z, [0.0, 0.0]) == [[0, 0], [1, -1]]           # probability zero; a request without rows
    assert one([0, 1, 0, 0, 0], [0, 2], [1.0] + z[1:], [0.4], p) == [[0], [1]]           # p = q and the test fails: p itself
    assert one([0, 1, 0, 0, 0], [2, 3], z, [0.5]) == [[0], [-1]]                         # no weight at all
    assert one([0, 1, 0, 0, 0], [3, 4], z, [0.5]) == [[0], [2]]                          # a NaN counts as zero
    assert one([0, 1, 0, 0, 0], [4, 5], z, [0.5]) == [[0], [-1]]                         # no finite sum
    assert kl.kl_device_status() == 0
    assert one([0, 3, 0, 0, 0], [0, 2], z, [0.0]) == [[0], [1]]                          # a draft outside the vocabulary
    with pytest.raises(kl.KLError) as e:
        kl.kl_device_status()
    assert "0x2" in str(e.value)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify_answers_do_not_depend_on_the_batch(kl, dtype):
    """Three requests alone, and repeated in batches up to 7, 14 and more (each served by another split of the row)."""
    V, g = 5001, torch.Generator(device="cuda").manual_seed(8)
    p = torch.softmax(2 * torch.randn(9, V, generator=g, device="cuda"), 1).to(dtype)
    q = torch.softmax(2 * torch.randn(9, V, generator=g, device="cuda"), 1).to(dtype)
    tokens = np.concatenate([[0], torch.multinomial(q.float(), 1, generator=g)[:-1, 0].cpu().numpy()])
    rng = np.random.default_rng(8)
    ua, us = rng.random(9).astype(np.float32), rng.random(3).astype(np.float32)
    want = O.draft_verify(_host(p), _host(q), tokens, [0, 4, 5, 9], ua, us)
    for times in (1, 2, 4, 5, 7):
        B = 3 * times
        cu = np.concatenate([[0], (9 * np.arange(times)[:, None] + [4, 5, 9]).reshape(-1)])
        got = _verify(kl, p.repeat(times, 1), q.repeat(times, 1), np.tile(tokens, times), cu, np.tile(ua, times), np.tile(us, times))
        assert len(got[0]) == B
        np.testing.assert_array_equal(got[0], np.tile(want[0], times))
        np.testing.assert_array_equal(got[1], np.tile(want[1], times))
    assert kl.kl_device_status() == 0


@pytest.mark.parametrize("B", [3, 9, 20])
def test_verify_a_sum_that_meets_its_mark(kl, B):
    """4096 equal weights and u = k / 4096: the sum of k weights is exactly u times the total, which the token after it exceeds first."""
    p = torch.full((B, 4096), 2.0 ** -12, device="cuda")
    k = np.linspace(0, 4095, B).astype(np.int64)
    got = _verify(kl, p, None, np.zeros(B, np.int64), np.arange(B + 1), np.zeros(B, np.float32), (k / 4096).astype(np.float32))
    np.testing.assert_array_equal(got[1], k)
    assert kl.kl_device_status() == 0


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def test_layer_forward_matches_oracle_and_the_paged_layer(kl):
    H, Hq, Hkv, I, bs = 256, 4, 2, 512, 16
    reqs = [(1, 20), (20, 0), (0, 9), (3, 45)]
    for qk_norm, inter in ((False, False), (True, True)):
        rng, n, ctx, table, maxb, nb, kp, vp, cu, T = _step(21, reqs, Hkv, bs)
        kp, vp = np.nan_to_num(kp), np.nan_to_num(vp)
        w = synth.layer_weights(21, H, Hq, Hkv, D, I, bf16=True, qk_norm=qk_norm)
        X = synth.layer_inputs(21, T, H, bf16=True)["X"]
        want, kref, vref = np.zeros((T, H)), kp, vp
        for b in range(len(reqs)):
            if n[b]:
                oc = O.LayerConfig(B=1, S=int(n[b]), H=H, Hq=Hq, Hkv=Hkv, d=D, I=I, qk_norm=qk_norm, rope_interleaved=inter)
                want[cu[b]:cu[b + 1]], kref, vref, _ = O.layer_forward_paged(oc, w, X[cu[b]:cu[b + 1]], kref, vref, table[b:b + 1], ctx[b:b + 1], int(n[b]))
        cfg = L.make_cfg(1, T, H, Hq, Hkv, D, I, dtype=kl.KL_BF16, qk_norm=qk_norm, rope_interleaved=inter)
        rc = kl.RaggedCfg(len(reqs), T, bs, maxb, nb)
        wd = {k: L.to_device(w[L.SYNTH_NAMES[k]], kl.KL_BF16, "cuda") for k in L.weight_fields(cfg)}
        pos = np.concatenate([np.arange(c, c + k) for k, c in reqs])
        req = np.repeat(np.arange(len(reqs)), n)
        slots = table[req, pos // bs] * bs + pos % bs
        kd, vd, Xd, td, cd, xd, pd, sd = _dev(kp), _dev(vp), _dev(X), _i(table), _i(cu), _i(ctx), _i(pos), _i(slots)
        ws = torch.empty(kl.kl_layer_forward_ragged_ws_bytes(cfg, rc), dtype=torch.uint8, device="cuda")
        Y = torch.empty_like(Xd)
        kl.kl_layer_forward_ragged(cfg, rc, L.weights_struct(wd), Xd.data_ptr(), Y.data_ptr(), kd.data_ptr(), vd.data_ptr(), td.data_ptr(), cd.data_ptr(), xd.data_ptr(),
                                   pd.data_ptr(), sd.data_ptr(), ws.data_ptr(), ws.numel())
        assert kl.kl_device_status() == 0
        assert_rel(_host(Y), want, TOL_BF16, "Y")
        assert_rel(_host(kd), kref, TOL_BF16, "k pool")
        assert_rel(_host(vd), vref, TOL_BF16, "v pool")


def test_a_captured_serving_loop(kl):
    """plan -> norm, rotation and cache write -> attention -> verify captured once and replayed over steps of different
    lengths (a prompt, drafts, rejected ones, an ended request and its successor), on a stream of its own, each checked against
    the oracle; the graph's lengths, contexts and random numbers are only ever changed on the device."""
    B, T, bs, maxb, nb, Hq, Hkv, V = 3, 64, 8, 16, 40, 8, 2, 50
    rng = np.random.default_rng(31)
    s = Planner(kl, B, T, bs, maxb, nb, rng.permutation(nb), nb)
    bf = torch.bfloat16
    q, k, v = (torch.zeros(T, h, D, dtype=bf, device="cuda") for h in (Hq, Hkv, Hkv))
    qr, o = torch.zeros_like(q), torch.zeros_like(q)
    kp, vp = (torch.full((nb, bs, Hkv, D), float("nan"), dtype=bf, device="cuda") for _ in range(2))
    P, Q = torch.zeros(T, V, device="cuda"), torch.zeros(T, V, device="cuda")
    tokens, ua, us = _i(np.zeros(T)), torch.zeros(T, device="cuda"), torch.zeros(B, device="cuda")
    acc, nxt = _i(np.zeros(B)), _i(np.zeros(B))
    ws = torch.empty(kl.kl_ragged_attention_ws_bytes(s.rc, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    vc = kl.VerifyCfg(B, T, V, kl.KL_F32)

    def body():
        s.launch()
        kl.kl_ragged_qkv_rope(s.rc, Hq, Hkv, D, kl.KL_BF16, q.data_ptr(), k.data_ptr(), v.data_ptr(), 0, 0, 1e-6, 1e4, 0, s.cu.data_ptr(), s.pos.data_ptr(), s.slots.data_ptr(),
                              qr.data_ptr(), kp.data_ptr(), vp.data_ptr())
        kl.kl_ragged_attention(s.rc, Hq, Hkv, D, kl.KL_BF16, qr.data_ptr(), kp.data_ptr(), vp.data_ptr(), s.d["table"].data_ptr(), s.cu.data_ptr(), s.ctx.data_ptr(), o.data_ptr(),
                               0, ws.data_ptr(), ws.numel())
        kl.kl_draft_verify(vc, P.data_ptr(), V, Q.data_ptr(), V, tokens.data_ptr(), s.cu.data_ptr(), ua.data_ptr(), us.data_ptr(), acc.data_ptr(), nxt.data_ptr())

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        body()                                   # the first call outside the capture (an empty step)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        body()
    ctx = np.zeros(B, int)
    K, VV = [np.zeros((0, Hkv, D)) for _ in range(B)], [np.zeros((0, Hkv, D)) for _ in range(B)]
    for step in range(8):
        n = [[30, 1, 0], [3, 4, 17], [1, 1, 1], [4, -1, 2], [2, 9, 4], [0, 1, 5], [5, 5, 5], [1, 2, 0]][step]
        for t in (q, k, v):
            t.copy_(torch.as_tensor(_bf(rng, *t.shape)))
        P.copy_(torch.as_tensor(rng.dirichlet(np.ones(V), T)))
        Q.copy_(torch.as_tensor(rng.dirichlet(np.ones(V), T)))
        tokens.copy_(_i(rng.integers(0, V, T)))
        ua.copy_(torch.as_tensor(rng.random(T)))
        us.copy_(torch.as_tensor(rng.random(B)))
        torch.cuda.synchronize()

        def replay():
            with torch.cuda.stream(side):
                graph.replay()

        r = s.step(n, ctx, replay)
        assert kl.kl_device_status(side) == 0 and r["missing"] == 0
        cu, rows = r["cu"], int(r["cu"][-1])
        pos = r["pos"]
        kr, got_q = O.rope_at(_host(k)[:rows], pos, 1e4), _host(qr)
        want_acc, want_nxt = O.draft_verify(_host(P), _host(Q), tokens.cpu().numpy(), cu, ua.cpu().numpy(), us.cpu().numpy())
        np.testing.assert_array_equal(acc.cpu().numpy(), want_acc)
        np.testing.assert_array_equal(nxt.cpu().numpy(), want_nxt)
        for b in range(B):
            if n[b] < 0:
                ctx[b], K[b], VV[b] = 0, K[b][:0], VV[b][:0]
                continue
            x = slice(int(cu[b]), int(cu[b + 1]))
            K[b], VV[b] = np.concatenate([K[b][:ctx[b]], kr[x]]), np.concatenate([VV[b][:ctx[b]], _host(v)[x]])
            if n[b]:
                pages = np.arange(len(K[b])).reshape(-1, 1)
                want, _, _ = O.ragged_attention(got_q[x], K[b][:, None], VV[b][:, None], pages.T, [0, n[b]], [ctx[b]])
                assert_rel(_host(o)[x], want, TOL_BF16, f"step {step} request {b}")
                ctx[b] += int(want_acc[b]) + 1    # the rejected drafts' rows are fed again


def test_attention_of_many_requests(kl):
    """More requests than a CTA has threads, most of them idle."""
    Hq, Hkv, bs = 8, 2, 8
    rng = np.random.default_rng(41)
    reqs = [(int(a), int(c)) for a, c in zip(rng.choice([0, 0, 0, 1, 3], 1500), rng.integers(0, 200, 1500))]
    rng, n, ctx, table, maxb, nb, kp, vp, cu, T = _step(42, reqs, Hkv, bs)
    q = _bf(rng, T, Hq, D)
    rc = kl.RaggedCfg(len(reqs), T, bs, maxb, nb)
    qd, kd, vd, td, cd, xd = _dev(q), _dev(kp), _dev(vp), _i(table), _i(cu), _i(ctx)
    ws = torch.empty(kl.kl_ragged_attention_ws_bytes(rc, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    o = torch.empty_like(qd)
    kl.kl_ragged_attention(rc, Hq, Hkv, D, kl.KL_BF16, qd.data_ptr(), kd.data_ptr(), vd.data_ptr(), td.data_ptr(), cd.data_ptr(), xd.data_ptr(), o.data_ptr(), 0,
                           ws.data_ptr(), ws.numel())
    assert kl.kl_device_status() == 0
    want, _, A = O.ragged_attention(q, kp, vp, table, cu, ctx)
    assert (np.abs(_host(o) - want) <= (2.0 ** -8 + 2.0 ** -9 + 2e-4) * A + 2.0 ** -8 * np.abs(want)).all()


def test_two_streams_at_once(kl):
    """The same operators on two streams at the same time, a workspace each: the bits of one after the other."""
    Hq, Hkv, bs = 64, 8, 16
    sets = []
    for seed, reqs in ((51, [(1, 3000), (40, 100), (7, 0)]), (52, [(300, 700), (1, 5)])):
        rng, n, ctx, table, maxb, nb, kp, vp, cu, T = _step(seed, reqs, Hkv, bs)
        rc = kl.RaggedCfg(len(reqs), T, bs, maxb, nb)
        t = dict(q=_dev(_bf(rng, T, Hq, D)), k=_dev(kp), v=_dev(vp), t=_i(table), c=_i(cu), x=_i(ctx),
                 ws=torch.empty(kl.kl_ragged_attention_ws_bytes(rc, Hq, Hkv, D), dtype=torch.uint8, device="cuda"))
        t["outs"] = [torch.empty_like(t["q"]) for _ in range(21)]
        sets.append((rc, t, torch.cuda.Stream()))

    def call(rc, t, o, st):
        kl.kl_ragged_attention(rc, Hq, Hkv, D, kl.KL_BF16, t["q"].data_ptr(), t["k"].data_ptr(), t["v"].data_ptr(), t["t"].data_ptr(), t["c"].data_ptr(), t["x"].data_ptr(),
                               o.data_ptr(), 0, t["ws"].data_ptr(), t["ws"].numel(), st)

    for rc, t, st in sets:
        call(rc, t, t["outs"][0], None)
    torch.cuda.synchronize()
    for i in range(1, 21):
        for rc, t, st in sets:
            call(rc, t, t["outs"][i], st)
    assert kl.kl_device_status(sets[0][2]) == 0 and kl.kl_device_status(sets[1][2]) == 0
    for rc, t, st in sets:
        assert all(torch.equal(o, t["outs"][0]) for o in t["outs"][1:])


def test_offsets_past_32_bits(kl):
    """Pools of more than 2^31 elements and probability rows past 2^31: what lies at their ends is found."""
    Hq, Hkv, bs, nb = 64, 8, 16, 140000                       # 2.3e9 elements a pool
    kp, vp = (torch.empty(nb, bs, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rng = np.random.default_rng(61)
    n, ctx = 3, 90
    table = np.array([[nb - 1, nb - 7, 5, nb - 3, 0, nb - 2]])
    pos = np.arange(ctx + n)
    slots = table[0][pos // bs] * bs + pos % bs
    T = n + ctx
    q, k, v = _bf(rng, T, Hq, D), _bf(rng, T, Hkv, D), _bf(rng, T, Hkv, D)
    rc = kl.RaggedCfg(1, T, bs, table.shape[1], nb)
    qd, kd, vd, cu, pd, sd = _dev(q), _dev(k), _dev(v), _i([0, T]), _i(np.zeros(T)), _i(slots)
    kl.kl_ragged_qkv_rope(rc, Hq, Hkv, D, kl.KL_BF16, qd.data_ptr(), kd.data_ptr(), vd.data_ptr(), 0, 0, 1e-6, 1e6, 0, cu.data_ptr(), pd.data_ptr(), sd.data_ptr(),
                          qd.data_ptr(), kp.data_ptr(), vp.data_ptr())      # position zero: no rotation
    sl = torch.as_tensor(slots, device="cuda")
    assert torch.equal(kp.view(-1, Hkv, D)[sl], kd) and torch.equal(vp.view(-1, Hkv, D)[sl], vd)
    o = torch.empty(n, Hq, D, dtype=torch.bfloat16, device="cuda")
    rc2 = kl.RaggedCfg(1, n, bs, table.shape[1], nb)
    ws = torch.empty(kl.kl_ragged_attention_ws_bytes(rc2, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    qn, td, c2, xd = qd[ctx:].contiguous(), _i(table), _i([0, n]), _i([ctx])
    kl.kl_ragged_attention(rc2, Hq, Hkv, D, kl.KL_BF16, qn.data_ptr(), kp.data_ptr(), vp.data_ptr(), td.data_ptr(), c2.data_ptr(), xd.data_ptr(), o.data_ptr(), 0, ws.data_ptr(),
                           ws.numel())
    assert kl.kl_device_status() == 0
    want, _, A = O.ragged_attention(q[ctx:], k[:, None], v[:, None], np.arange(T)[None], [0, n], [ctx])
    assert (np.abs(_host(o) - want) <= (2.0 ** -8 + 2.0 ** -9 + 2e-4) * A + 2.0 ** -8 * np.abs(want)).all()
    del kp, vp
    T, V = 15000, 151936                                      # 2.3e9 probabilities
    p = torch.empty(T, V, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(62)
    p[T - 2:] = torch.softmax(torch.randn(2, V, generator=g, device="cuda"), 1)
    p[0] = torch.softmax(torch.randn(V, generator=g, device="cuda"), 0)
    p[0, 7] = 0.0
    tokens = np.full(T, 7)
    tokens[T - 1] = 11
    ua, us = np.zeros(T, np.float32), np.array([0.37, 0.61], np.float32)
    acc, nxt = _verify(kl, p, None, tokens, [0, T - 2, T], ua, us)   # request 0's first draft has probability zero
    rows = _host(p[[0, T - 2, T - 1]])
    want = O.draft_verify(rows, None, [7, 7, 11], [0, 1, 3], [0.0, 0.0, 0.0], us)
    w0 = np.searchsorted(np.cumsum(rows[0]), float(us[0]) * rows[0].sum(), side="right")   # p without the draft, whose weight is zero
    assert list(acc) == [0, want[0][1]] and list(nxt) == [w0, want[1][1]]


def test_a_copy_of_the_rows_in_the_wrong_places_is_left_alone(kl):
    """cu_rows that run past the tensors or backwards: brought into range, nothing outside is touched."""
    Hq, Hkv, bs = 8, 1, 16
    rng, n, ctx, table, maxb, nb, kp, vp, cu, T = _step(71, [(4, 20), (3, 10)], Hkv, bs)
    q = _dev(_bf(rng, T, Hq, D))
    rc = kl.RaggedCfg(2, T, bs, maxb, nb)
    guard = torch.full((T + 8, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(kl.kl_ragged_attention_ws_bytes(rc, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    kd, vd, td, xd = _dev(np.nan_to_num(kp)), _dev(np.nan_to_num(vp)), _i(np.clip(table, 0, nb - 1)), _i([20, 10])
    for bad in ([0, 4, 100], [-3, 4, 7], [4, 2, 7]):
        cd = _i(bad)
        kl.kl_ragged_attention(rc, Hq, Hkv, D, kl.KL_BF16, q.data_ptr(), kd.data_ptr(), vd.data_ptr(), td.data_ptr(), cd.data_ptr(), xd.data_ptr(), guard[4:].data_ptr(), 0,
                               ws.data_ptr(), ws.numel())
        torch.cuda.synchronize()
        assert (guard[:4] == 5.0).all() and (guard[4 + T:] == 5.0).all()
    try:
        kl.kl_device_status()          # positions past the table may have been reported
    except kl.KLError as e:
        assert e.status == kl.KL_ERR_DEVICE
