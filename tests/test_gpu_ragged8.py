"""The ragged step over a cache held in 8 bits through the C ABI against the fp64 oracle: append (codes and scales), attention,
the layer, and a captured serving loop that fills, rejects and refills pages."""
import numpy as np
import pytest
import torch

import oracle as O
from bwd_qwen3_layer_gb300 import layer as L
from bwd_qwen3_layer_gb300 import synth
from _parity import TOL_BF16, assert_rel
from test_gpu_ragged import ATTENTION, D, Planner, _bf, _dev, _host, _i, _step

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def _codes(values):
    """e4m3 values on the host -> codes on the device."""
    return torch.as_tensor(np.asarray(values, np.float32)).to(E4M3).cuda()


def _f(a):
    return torch.as_tensor(np.ascontiguousarray(a, np.float32)).cuda()


def _step8(seed, reqs, Hkv, bs, extra_rows=0, any_scale=False):
    """_step with its pools in 8 bits: pages of different sizes, NaN codes in every slot behind a request's end, NaN scales in the
    blocks that nobody has. any_scale: scales that are no powers of two."""
    rng, n, ctx, table, maxb, nb, kp, vp, cu, T = _step(seed, reqs, Hkv, bs, extra_rows)
    r2 = np.random.default_rng(seed + 1000)
    out = []
    for x in (kp, vp):
        x = x * np.exp2(r2.integers(-2, 3, (nb, 1, Hkv, 1)))
        a = np.nanmax(np.abs(np.where(np.isnan(x), 0.0, x)), (1, 3))
        s = O.scale_for(a)
        if any_scale:
            s = (s * r2.uniform(1.0, 1.9, s.shape)).astype(np.float32).astype(np.float64)
        c = O.e4m3_round(np.clip(x / s[:, None, :, None], -448, 448))
        s[np.isnan(x).all((1, 2, 3))] = np.nan
        out += [c, s]
    return rng, n, ctx, table, maxb, nb, out, cu, T


def _attention_tol(q, kc, ks, vc, vs, table, cu, ctx, want, A):
    """The bound on |o - oracle| of a weight that is a sum of two e4m3 numbers, elementwise, and the one on lse.
    Queries: two e4m3 pieces hold a bf16 number's 8 bits; below 2^-10 of the row's largest one they are off by 2^-10 at a largest of
    128 or more: 2^-17 of it. Weights: f16 (2^-11) cut to 4 bits, the rest, below 2^-3 of the weight's power of two, rounded to
    4: 2^-8 of it; codes below 2^-6 are off by 2^-10 instead, in both parts, where the row's largest weight times scale is held as
    2^4 or more: 2^-13 of that weight, in units of the scale. fp32 sums as in the bf16 test: 2^-24 x 128 x sum |q k| / sqrt(d) of a
    score and 2^-9 A of the running sums; the result is rounded to bf16, 2^-8 |o|."""
    T, Hq, d = q.shape
    bs, Hkv = kc.shape[1], kc.shape[2]
    tol, ltol = np.zeros_like(want), np.zeros((T, Hq))
    for b in range(len(ctx)):
        n = int(cu[b + 1] - cu[b])
        L_ = int(ctx[b]) + n
        p = np.arange(L_)
        at = np.asarray(table[b])[p // bs]
        for i in range(n):
            r, end = int(cu[b]) + i, int(ctx[b]) + i + 1
            for h in range(Hq):
                g = h // (Hq // Hkv)
                kb, vb = ks[at[:end], g], vs[at[:end], g]
                k, v = kc[at[:end], p[:end] % bs, g], vc[at[:end], p[:end] % bs, g]
                z = k @ q[r, h] * kb / np.sqrt(d)
                w = np.exp(z - z.max())
                w /= w.sum()
                mag = np.abs(k).sum(1) * kb / np.sqrt(d)
                dz = 2.0 ** -17 * np.abs(q[r, h]).max() * mag.max() + 2.0 ** -17 * (np.abs(k) @ np.abs(q[r, h]) * kb).max() / np.sqrt(d)
                ltol[r, h] = dz + 1e-6 * abs(z).max() + L_ * 2.0 ** -24 + 1e-6
                tol[r, h] = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -9 + 2 * dz) * A[r, h] + 2.0 ** -8 * np.abs(want[r, h]) + 2.0 ** -13 * (w * vb).max() * np.abs(v).sum(0)
    return tol, ltol


def _attend(kl, rc, Hq, Hkv, q, kc, ks, vc, vs, table, cu, ctx, lse=True, ws=None, stream=None, o=None):
    o = torch.full_like(q, 7.0) if o is None else o
    ls = torch.full(q.shape[:2], 7.0, device="cuda")
    if ws is None:
        ws = torch.empty(kl.kl_ragged_attention8_ws_bytes(rc, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    kl.kl_ragged_attention8(rc, Hq, Hkv, D, kl.KL_BF16, q.data_ptr(), kc.data_ptr(), vc.data_ptr(), ks.data_ptr(), vs.data_ptr(), table.data_ptr(), cu.data_ptr(),
                            ctx.data_ptr(), o.data_ptr(), ls.data_ptr() if lse else 0, ws.data_ptr(), ws.numel(), stream)
    return o, ls


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("any_scale", [False, True])
@pytest.mark.parametrize("Hq,Hkv,bs,reqs", ATTENTION)
def test_attention_matches_oracle(kl, Hq, Hkv, bs, reqs, any_scale):
    rng, n, ctx, table, maxb, nb, (kc, ks, vc, vs), cu, T = _step8(5, reqs, Hkv, bs, 3, any_scale)
    q = _bf(rng, T, Hq, D)
    want, want_lse, A = O.ragged_attention(q[:T - 3], O.dequantised(kc, ks), O.dequantised(vc, vs), table, cu, ctx)
    rc = kl.RaggedCfg(len(reqs), T, bs, maxb, nb)
    a = [_dev(q), _codes(kc), _f(ks), _codes(vc), _f(vs), _i(table), _i(cu), _i(ctx)]
    outs = [_attend(kl, rc, Hq, Hkv, *a, lse=x) for x in (True, False, True)]
    assert kl.kl_device_status() == 0
    got, got_lse = _host(outs[0][0]), _host(outs[0][1])
    tol, ltol = _attention_tol(q[:T - 3], kc, ks, vc, vs, table, cu, ctx, want, A)
    assert (np.abs(got[:T - 3] - want) <= tol).all(), np.max(np.abs(got[:T - 3] - want) / tol)
    assert_rel(got[:T - 3], want, 2.0 ** -7, "O")
    assert (np.abs(got_lse[:T - 3] - want_lse) <= ltol).all(), np.max(np.abs(got_lse[:T - 3] - want_lse) / ltol)
    # rows behind the last request stay as they were; the same bits again, with and without lse
    assert (got[T - 3:] == 7.0).all() and (got_lse[T - 3:] == 7.0).all()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][0], outs[2][0]) and torch.equal(outs[0][1], outs[2][1])
    assert (outs[1][1] == 7.0).all()


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -20, 2.0 ** 20, 2.0 ** 100])
def test_attention_of_queries_of_any_size(kl, size):
    """Queries of one size and keys of the other's inverse: the same scores, so nearly the same result."""
    Hq, Hkv, bs, reqs = 8, 2, 16, [(5, 300), (1, 17)]
    rng, n, ctx, table, maxb, nb, (kc, ks, vc, vs), cu, T = _step8(6, reqs, Hkv, bs)
    q = _bf(rng, T, Hq, D)
    rc = kl.RaggedCfg(len(reqs), T, bs, maxb, nb)
    rest = [_codes(vc), _f(vs), _i(table), _i(cu), _i(ctx)]
    o, lse = _attend(kl, rc, Hq, Hkv, _dev(q), _codes(kc), _f(ks), *rest)
    o2, lse2 = _attend(kl, rc, Hq, Hkv, _dev(q * size), _codes(kc), _f(ks / size), *rest)
    assert kl.kl_device_status() == 0
    # powers of two: every product the same, the factors of a score multiply in another order
    assert (_host(lse) - _host(lse2) == 0).all() or np.max(np.abs(_host(lse) - _host(lse2))) < 2e-5
    assert_rel(_host(o2), _host(o), 2.0 ** -8, "O")


def test_attention_of_values_of_any_size(kl):
    """Pages whose value scales lie 2^80 apart: the small ones' values vanish, the sums stay right."""
    Hq, Hkv, bs, reqs = 8, 1, 16, [(3, 200), (1, 700), (40, 30)]
    rng, n, ctx, table, maxb, nb, (kc, ks, vc, vs), cu, T = _step8(7, reqs, Hkv, bs)
    vs = vs * 2.0 ** rng.choice([-60, -20, 0, 20], vs.shape)
    q = _bf(rng, T, Hq, D)
    want, want_lse, A = O.ragged_attention(q, O.dequantised(kc, ks), O.dequantised(vc, vs), table, cu, ctx)
    rc = kl.RaggedCfg(len(reqs), T, bs, maxb, nb)
    o, lse = _attend(kl, rc, Hq, Hkv, _dev(q), _codes(kc), _f(ks), _codes(vc), _f(vs), _i(table), _i(cu), _i(ctx))
    assert kl.kl_device_status() == 0
    tol, ltol = _attention_tol(q, kc, ks, vc, vs, table, cu, ctx, want, A)
    assert (np.abs(_host(o) - want) <= tol).all()
    assert (np.abs(_host(lse) - want_lse) <= ltol).all()


@pytest.mark.parametrize("k", [-60, 20, 100])
def test_attention_scales_with_its_values(kl, k):
    """All value scales times 2^k: the result times 2^k. The scores' logarithms are formed around k, off by 2^-17 there at most: 2^-17 of
    a weight, beside the 2^-8 of its parts and the result's rounding of the one call and of the other; lse is a number of that size."""
    Hq, Hkv, bs, reqs = 8, 2, 16, [(5, 300), (1, 1700), (40, 30)]
    rng, n, ctx, table, maxb, nb, (kc, ks, vc, vs), cu, T = _step8(9, reqs, Hkv, bs)
    vs = np.nan_to_num(vs, nan=1.0)
    vs[vs * 2.0 ** k < 2.0 ** -64] = 2.0 ** (-64 - min(k, 0))
    q = _dev(_bf(rng, T, Hq, D))
    rc = kl.RaggedCfg(len(reqs), T, bs, maxb, nb)
    tail = [_i(table), _i(cu), _i(ctx)]
    o, lse = _attend(kl, rc, Hq, Hkv, q, _codes(kc), _f(ks), _codes(vc), _f(vs), *tail)
    o2, lse2 = _attend(kl, rc, Hq, Hkv, q, _codes(kc), _f(ks), _codes(vc), _f(vs * 2.0 ** k), *tail)
    assert kl.kl_device_status() == 0
    A = O.ragged_attention(_host(q), O.dequantised(kc, ks), O.dequantised(vc, vs), table, cu, ctx)[2]
    assert (np.abs(_host(o2) * 2.0 ** -k - _host(o)) <= (2.0 ** -7 + 2.0 ** -15) * A + 2.0 ** -7 * np.abs(_host(o))).all()
    assert np.abs(_host(lse2) - _host(lse)).max() <= 1e-4


@pytest.mark.parametrize("bs", [16, 5])
def test_attention_reports_pages_outside_the_pool(kl, bs):
    """A bad table entry reads as zero keys and values and is reported; other requests are not touched by it."""
    reqs, Hq, Hkv = [(2, 60), (3, 300)], 8, 2
    rng, n, ctx, table, maxb, nb, (kc, ks, vc, vs), cu, T = _step8(7, reqs, Hkv, bs)
    q = _bf(rng, T, Hq, D)
    bad = table.copy()
    bad[0, 1] = -1
    bad[0, 2] = nb
    rc = kl.RaggedCfg(2, T, bs, maxb, nb)
    o, _ = _attend(kl, rc, Hq, Hkv, _dev(q), _codes(kc), _f(ks), _codes(vc), _f(vs), _i(bad), _i(cu), _i(ctx))
    with pytest.raises(kl.KLError) as e:
        kl.kl_device_status()
    assert e.value.status == kl.KL_ERR_DEVICE and "0x8" in str(e.value)
    # the same as a pool with zero blocks there
    zero = np.zeros((1,) + kc.shape[1:])
    kc, vc, ks, vs = np.concatenate([kc, zero]), np.concatenate([vc, zero]), np.concatenate([ks, np.ones((1, Hkv))]), np.concatenate([vs, np.ones((1, Hkv))])
    z = np.where((bad < 0) | (bad == nb), nb, bad)
    want, _, A = O.ragged_attention(q, O.dequantised(kc, ks), O.dequantised(vc, vs), z, cu, ctx)
    tol, _ = _attention_tol(q, kc, ks, vc, vs, z, cu, ctx, want, A)
    assert (np.abs(_host(o) - want) <= tol).all()


@pytest.mark.parametrize("bs", [16, 5])
def test_attention_nonfinite(kl, bs):
    """A NaN or an infinity in a query, a NaN in a key that a row sees or in the scale of its block: the row's o and lse are NaN, the
    others' as they were. A NaN in a key behind the rows that see it is not met."""
    Hq, Hkv, reqs = 4, 2, [(30, 100), (1, 50), (2, 1000)]
    rng, n, ctx, table, maxb, nb, (kc, ks, vc, vs), cu, T = _step8(8, reqs, Hkv, bs)
    q = _bf(rng, T, Hq, D)
    rc = kl.RaggedCfg(3, T, bs, maxb, nb)
    tail = [_i(table), _i(cu), _i(ctx)]
    base, blse = _attend(kl, rc, Hq, Hkv, _dev(q), _codes(kc), _f(ks), _codes(vc), _f(vs), *tail)

    def check(bad, *args):
        o, lse = _attend(kl, rc, Hq, Hkv, *args, *tail)
        bad = torch.as_tensor(bad).cuda()
        assert torch.isnan(o[bad]).all() and torch.isnan(lse[bad]).all()
        assert torch.equal(o[~bad], base[~bad]) and torch.equal(lse[~bad], blse[~bad])

    for x in (np.nan, np.inf, -np.inf):
        q2 = q.copy()
        q2[3, 1, 77] = x
        bad = np.zeros((T, Hq), bool)
        bad[3, 1] = True
        check(bad, _dev(q2), _codes(kc), _f(ks), _codes(vc), _f(vs))
    # request 0's key at position 110 (its rows from 10 on see it), head 1
    k2 = kc.copy()
    k2[table[0, 110 // bs], 110 % bs, 1, 5] = np.nan
    bad = np.zeros((T, Hq), bool)
    bad[10:30, 2:] = True
    check(bad, _dev(q), _codes(k2), _f(ks), _codes(vc), _f(vs))
    # scales of a block of request 2 that both its rows see
    for which in (0, 1):
        s2 = [ks.copy(), vs.copy()]
        s2[which][table[2, 333 // bs], 0] = np.nan
        bad = np.zeros((T, Hq), bool)
        bad[31:, :2] = True
        check(bad, _dev(q), _codes(kc), _f(s2[0]), _codes(vc), _f(s2[1]))
    assert kl.kl_device_status() == 0


def test_attention_without_rows(kl):
    rc = kl.RaggedCfg(3, 4, 16, 2, 4)
    q = torch.randn(4, 8, D, device="cuda").bfloat16()
    pool, scale = torch.zeros(4, 16, 1, D, device="cuda").to(E4M3), torch.ones(4, 1, device="cuda")
    o, lse = _attend(kl, rc, 8, 1, q, pool, scale, pool, scale, _i(np.zeros((3, 2))), _i([0, 0, 0, 0]), _i([5, 0, 9]))
    assert kl.kl_device_status() == 0
    assert (o == 7.0).all() and (lse == 7.0).all()


def test_attention_of_many_requests(kl):
    """More requests than a CTA has threads, most of them idle."""
    Hq, Hkv, bs = 8, 2, 8
    rng = np.random.default_rng(41)
    reqs = [(int(a), int(c)) for a, c in zip(rng.choice([0, 0, 0, 1, 3], 1500), rng.integers(0, 200, 1500))]
    rng, n, ctx, table, maxb, nb, (kc, ks, vc, vs), cu, T = _step8(42, reqs, Hkv, bs)
    q = _bf(rng, T, Hq, D)
    rc = kl.RaggedCfg(len(reqs), T, bs, maxb, nb)
    o, _ = _attend(kl, rc, Hq, Hkv, _dev(q), _codes(kc), _f(ks), _codes(vc), _f(vs), _i(table), _i(cu), _i(ctx))
    assert kl.kl_device_status() == 0
    want, _, A = O.ragged_attention(q, O.dequantised(kc, ks), O.dequantised(vc, vs), table, cu, ctx)
    tol, _ = _attention_tol(q, kc, ks, vc, vs, table, cu, ctx, want, A)
    assert (np.abs(_host(o) - want) <= tol).all()


def test_cu_rows_in_the_wrong_places(kl):
    """cu_rows that run past the tensors or backwards: brought into range, nothing outside is touched."""
    Hq, Hkv, bs = 8, 1, 16
    rng, n, ctx, table, maxb, nb, (kc, ks, vc, vs), cu, T = _step8(71, [(4, 20), (3, 10)], Hkv, bs)
    q = _dev(_bf(rng, T, Hq, D))
    rc = kl.RaggedCfg(2, T, bs, maxb, nb)
    guard = torch.full((T + 8, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda")
    a = [_codes(np.nan_to_num(kc)), _f(np.nan_to_num(ks)), _codes(np.nan_to_num(vc)), _f(np.nan_to_num(vs)), _i(np.clip(table, 0, nb - 1))]
    for bad in ([0, 4, 100], [-3, 4, 7], [4, 2, 7]):
        _attend(kl, rc, Hq, Hkv, q, *a, _i(bad), _i([20, 10]), o=guard[4:4 + T])
        torch.cuda.synchronize()
        assert (guard[:4] == 5.0).all() and (guard[4 + T:] == 5.0).all()
    try:
        kl.kl_device_status()          # positions past the table may have been reported
    except kl.KLError as e:
        assert e.status == kl.KL_ERR_DEVICE


def test_two_streams_at_once(kl):
    """The same operators on two streams at the same time, a workspace each: the bits of one after the other."""
    Hq, Hkv, bs = 64, 8, 16
    sets = []
    for seed, reqs in ((51, [(1, 3000), (40, 100), (7, 0)]), (52, [(300, 700), (1, 5)])):
        rng, n, ctx, table, maxb, nb, (kc, ks, vc, vs), cu, T = _step8(seed, reqs, Hkv, bs)
        rc = kl.RaggedCfg(len(reqs), T, bs, maxb, nb)
        a = [_dev(_bf(rng, T, Hq, D)), _codes(kc), _f(ks), _codes(vc), _f(vs), _i(table), _i(cu), _i(ctx)]
        ws = torch.empty(kl.kl_ragged_attention8_ws_bytes(rc, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
        sets.append((rc, a, ws, torch.cuda.Stream(), [torch.empty_like(a[0]) for _ in range(21)]))
    for rc, a, ws, st, outs in sets:
        _attend(kl, rc, Hq, Hkv, *a, lse=False, ws=ws, o=outs[0])
    torch.cuda.synchronize()
    for i in range(1, 21):
        for rc, a, ws, st, outs in sets:
            _attend(kl, rc, Hq, Hkv, *a, lse=False, ws=ws, o=outs[i], stream=st)
    assert kl.kl_device_status(sets[0][3]) == 0 and kl.kl_device_status(sets[1][3]) == 0
    for *_, outs in sets:
        assert all(torch.equal(o, outs[0]) for o in outs[1:])


def test_attention_offsets_past_32_bits(kl):
    """Pools of more than 2^32 bytes: what lies at their ends is found."""
    Hq, Hkv, nb = 64, 8, 270000
    for bs in (16, 15):
        kp, vp = (torch.empty(nb, bs, Hkv, D, dtype=torch.uint8, device="cuda") for _ in range(2))
        ks, vs = (torch.empty(nb, Hkv, device="cuda") for _ in range(2))
        table = np.array([[nb - 1, nb - 7, 5, nb - 3, 0, nb - 2, 9]])
        rng, n, ctx, small, maxb, _, (kc, ksc, vc, vsc), cu, T = _step8(61, [(3, 90)], Hkv, bs)
        held = -(-93 // bs)
        for i in range(held):
            kp[table[0, i]], vp[table[0, i]] = _codes(kc[small[0, i]]).view(torch.uint8), _codes(vc[small[0, i]]).view(torch.uint8)
            ks[table[0, i]], vs[table[0, i]] = _f(ksc[small[0, i]]), _f(vsc[small[0, i]])
        q = _bf(rng, T, Hq, D)
        rc = kl.RaggedCfg(1, T, bs, table.shape[1], nb)
        o, _ = _attend(kl, rc, Hq, Hkv, _dev(q), kp, ks, vp, vs, _i(table), _i(cu), _i(ctx))
        assert kl.kl_device_status() == 0
        want, _, A = O.ragged_attention(q, O.dequantised(kc, ksc), O.dequantised(vc, vsc), small, cu, ctx)
        tol, _ = _attention_tol(q, kc, ksc, vc, vsc, small, cu, ctx, want, A)
        assert (np.abs(_host(o) - want) <= tol).all()
        del kp, vp


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def _append_case(seed, reqs, Hq, Hkv, bs, extra=2):
    """Rows, slots and pools with held pages: every request's earlier tokens are in its pages, with the scales they ask for."""
    rng = np.random.default_rng(seed)
    n, ctx = np.array([r[0] for r in reqs]), np.array([r[1] for r in reqs])
    blocks = -(-(n + ctx) // bs)
    nb = int(blocks.sum()) + 3
    order = rng.permutation(nb)
    T = int(n.sum())
    # only the pages that a request writes, and the one before, lie in the test's pool: far positions need no far pages
    slots, pos, at = [], [], 0
    for (k, c), m in zip(reqs, blocks):
        page = order[at:at + m]
        at += m
        p = np.arange(c, c + k)
        pos += list(p)
        slots += list(page[p // bs] * bs + p % bs)
    y0 = rng.standard_normal((nb, bs, Hkv, D)) * np.exp(rng.standard_normal((nb, 1, Hkv, 1)))
    pools = []
    for x in (y0, y0[::-1] * 0.7):
        s = O.scale_for(np.abs(x).max((1, 3)))
        pools += [O.e4m3_round(x / s[:, None, :, None]), s]
    x = [_bf(rng, T + extra, h, D) for h in (Hq, Hkv, Hkv)]
    return rng, T, np.array(pos, np.int64), np.array(slots, np.int64), nb, pools, x, np.concatenate([[0], np.cumsum(n)])


def _check_append(y, mag, slots, before, got_pool, got_scale, exact=False):
    """y: the rows in 64 bits, off by at most mag 2^-16 in fp32 (the bf16 append's bound). Scales: those of some y that near. Codes:
    within half a step, and that, of y / scale; older ones of growing pages exactly e4m3(code * old / new); all else as it was."""
    pool, scale = before
    bs = pool.shape[1]
    off = 0.0 if exact else 2.0 ** -16
    rows = np.nonzero(slots >= 0)[0]
    new = np.zeros(pool.shape[:2], bool)
    new.reshape(-1)[slots[rows]] = True
    for blk in range(pool.shape[0]):
        r = rows[slots[rows] // bs == blk]
        if not len(r):
            np.testing.assert_array_equal(got_scale[blk], scale[blk])
            np.testing.assert_array_equal(got_pool[blk], pool[blk])
            continue
        first = int(slots[r].min() % bs)
        for h in range(pool.shape[2]):
            x, d = y[r, h], mag[r, h] * off
            fin = np.isfinite(x)
            a, da = np.abs(np.where(fin, x, 0.0)).max(), d.max()
            w = [float(O.scale_for(max(0.0, v))) for v in (a - da, a, a + da)]
            if first > 0:
                w = [max(v, scale[blk, h]) for v in w]
            assert got_scale[blk, h] in w, (blk, h)
            s = got_scale[blk, h]
            if first > 0:
                old = pool[blk, :first, h]
                np.testing.assert_array_equal(got_pool[blk, :first, h], O.e4m3_round(old * (scale[blk, h] / s)) if s > scale[blk, h] else old)
            got = got_pool[blk, slots[r] % bs, h]
            assert np.isnan(got[~fin]).all()
            t = np.where(fin, x, 0.0) / s
            err = np.abs(np.where(fin, got - t, 0.0))
            assert (err <= np.where(fin, O.e4m3_half_step(np.abs(t) + d / s), 0.0) + d / s).all()
            if exact:
                np.testing.assert_array_equal(got[fin], O.e4m3_round(t)[fin])
            behind = np.setdiff1d(np.arange(first, bs), slots[r] % bs)
            np.testing.assert_array_equal(got_pool[blk, behind, h], pool[blk, behind, h])


@pytest.mark.parametrize("Hq,Hkv,bs,reqs,norm,inter,inplace", [
    (8, 1, 16, [(1, 0)], False, False, False),
    (64, 8, 16, [(1, 300), (5, 1000), (0, 7), (33, 64)], True, False, False),
    (12, 4, 5, [(3, 7), (2, 190), (11, 0)], True, True, True),
    (7, 7, 24, [(9, 23), (40, 5)], False, True, False),
    (128, 1, 8, [(2, 5)], True, False, True),
    (8, 1, 1, [(5, 3), (1, 0)], False, False, False),                # pages of one token
    (8, 2, 128, [(300, 100), (1, 127), (129, 0)], True, False, True),   # pages longer than a CTA's rows in flight
    (4, 2, 300, [(290, 250)], True, True, False),
    (8, 1, 16, [(700, 3), (0, 1), (33, 64)], False, False, True),
    (100, 100, 64, [(130, 1)], True, False, False),
    (64, 8, 16, [(1, 13 * i) for i in range(64)], True, False, False),
])
def test_append_matches_oracle(kl, Hq, Hkv, bs, reqs, norm, inter, inplace):
    rng, T, pos, slots, nb, (kc, ks, vc, vs), (qp, kp, v), cu = _append_case(8, reqs, Hq, Hkv, bs)
    if T > 2:
        slots[T // 2] = -1                           # a row without a block
        if (T // 2 + 1 < T) and slots[T // 2 + 1] % bs and slots[T // 2 + 1] == slots[T // 2 - 1] + 2:
            slots[T // 2 + 1:][slots[T // 2 + 1:] // bs == slots[T // 2 - 1] // bs] = -1    # the rest of its page: rows of a page are consecutive
    gq, gk = synth.round_bf16(1 + 0.2 * rng.standard_normal(D)), synth.round_bf16(1 + 0.2 * rng.standard_normal(D))
    eps, base = 1e-6, 1e6
    rc = kl.RaggedCfg(len(reqs), T + 2, bs, 4, nb)
    qd, kd, vd, gqd, gkd = _dev(qp), _dev(kp), _dev(v), _dev(gq), _dev(gk)
    kpd, vpd, ksd, vsd = _codes(kc), _codes(vc), _f(ks), _f(vs)
    out = qd if inplace else torch.full_like(qd, 7.0)
    cud, pd, sd = _i(cu), _i(np.concatenate([pos, [3, 4]])), _i(np.concatenate([slots, [0, 1]]))

    def call():
        kl.kl_ragged_qkv_rope8(rc, Hq, Hkv, D, kl.KL_BF16, qd.data_ptr(), kd.data_ptr(), vd.data_ptr(), gqd.data_ptr() if norm else 0, gkd.data_ptr() if norm else 0, eps, base,
                               int(inter), cud.data_ptr(), pd.data_ptr(), sd.data_ptr(), out.data_ptr(), kpd.data_ptr(), vpd.data_ptr(), ksd.data_ptr(), vsd.data_ptr())

    call()
    assert kl.kl_device_status() == 0

    def want(x, g):
        x = x[:T]
        if norm:
            x = O.rmsnorm_fwd(x, g, eps)[0]
        y = O.rope_at(x, pos, base, inter)
        return y, np.broadcast_to(2 * np.abs(x).max(-1, keepdims=True), x.shape)

    yq, mq = want(qp, gq)
    yk, mk = want(kp, gk)
    got_q = _host(out)
    assert (np.abs(got_q[:T] - yq) <= 2.0 ** -8 * np.abs(yq) * (1 + 2.0 ** -7) + 2.0 ** -16 * mq).all()
    assert (got_q[T:] == (qp[T:] if inplace else 7.0)).all()
    after = [_host(t) for t in (kpd, ksd, vpd, vsd)]
    _check_append(yk, mk, slots, (kc, ks), after[0], after[1])
    _check_append(v[:T], np.zeros_like(yk), slots, (vc, vs), after[2], after[3], exact=True)
    if not inplace:
        # the same step again changes nothing: the scales have grown already
        call()
        assert kl.kl_device_status() == 0
        for t, w in zip((kpd, ksd, vpd, vsd), after):
            np.testing.assert_array_equal(_host(t), w)


def _append(kl, rc, Hq, Hkv, q, k, v, cu, pos, slots, pools, out=None, stream=None, gains=(0, 0), inter=0):
    out = torch.full_like(q, 7.0) if out is None else out
    kl.kl_ragged_qkv_rope8(rc, Hq, Hkv, D, kl.KL_BF16, q.data_ptr(), k.data_ptr(), v.data_ptr(), *gains, 1e-6, 1e6, inter, cu.data_ptr(), pos.data_ptr(), slots.data_ptr(),
                           out.data_ptr(), *[t.data_ptr() for t in pools], stream)
    return out


@pytest.mark.parametrize("Hq,Hkv,bs,n_max,B", [(1, 1, 16, 40, 60), (8, 2, 17, 40, 60), (6, 3, 16, 3, 200), (4, 1, 18, 50, 40), (2, 2, 32, 90, 30), (2, 1, 16, 9800, 1), (16, 8, 16, 1, 700)])
def test_append_of_many_runs(kl, Hq, Hkv, bs, n_max, B):
    """Runs of all lengths and beginnings, within a CTA's rows and across their ends; requests appended together or one after the other
    leave the same bits."""
    rng = np.random.default_rng(B + bs)
    reqs = [(int(n), int(c)) for n, c in zip(rng.integers(min(n_max, 9800 if B == 1 else 1), n_max + 1, B), rng.integers(0, 3 * bs, B))]
    rng, T, pos, slots, nb, (kc, ks, vc, vs), (qp, kp, v), cu = _append_case(B, reqs, Hq, Hkv, bs)
    rc = kl.RaggedCfg(B, T + 2, bs, 4, nb)
    x = [_dev(qp), _dev(kp), _dev(v)]
    pools = [_codes(kc), _codes(vc), _f(ks), _f(vs)]
    alone = [t.clone() for t in pools]
    pd, sd = _i(np.concatenate([pos, [3, 4]])), _i(np.concatenate([slots, [0, 1]]))
    out = _append(kl, rc, Hq, Hkv, *x, _i(cu), pd, sd, pools)
    assert kl.kl_device_status() == 0
    yq, yk = O.rope_at(qp[:T], pos, 1e6, False), O.rope_at(kp[:T], pos, 1e6, False)
    mq, mk = (np.broadcast_to(2 * np.abs(t[:T]).max(-1, keepdims=True), t[:T].shape) for t in (qp, kp))
    got_q = _host(out)
    assert (np.abs(got_q[:T] - yq) <= 2.0 ** -8 * np.abs(yq) * (1 + 2.0 ** -7) + 2.0 ** -16 * mq).all() and (got_q[T:] == 7.0).all()
    after = [_host(t) for t in pools]
    _check_append(yk, mk, slots, (kc, ks), after[0], after[2])
    _check_append(v[:T], np.zeros_like(yk), slots, (vc, vs), after[1], after[3], exact=True)
    apart = torch.full_like(out, 7.0)
    for b in range(min(B, 40)):
        r = slice(int(cu[b]), int(cu[b + 1]))
        rows = int(cu[b + 1] - cu[b])
        _append(kl, kl.RaggedCfg(1, rows, bs, 4, nb), Hq, Hkv, *[t[r].contiguous() for t in x], _i([0, rows]), _i(pos[r]), _i(slots[r]), alone, apart[r])
    assert kl.kl_device_status() == 0
    done = np.unique(slots[:int(cu[min(B, 40)])] // bs)
    assert torch.equal(apart[:int(cu[min(B, 40)])], out[:int(cu[min(B, 40)])])
    for a, b in zip(alone, pools):
        assert torch.equal(a[done].view(torch.uint8), b[done].view(torch.uint8))


def test_append_in_two_graphs_and_on_two_streams(kl):
    """Two captured appends, each with pools of its own, replayed at the same time on two streams: the bits of eager calls."""
    sets = []
    for seed, bs, reqs in ((71, 16, [(40, 5), (1, 77), (300, 30)]), (72, 24, [(1, 24 * i + 7) for i in range(50)])):
        rng, T, pos, slots, nb, (kc, ks, vc, vs), (qp, kp, v), cu = _append_case(seed, reqs, 16, 4, bs)
        rc = kl.RaggedCfg(len(reqs), T + 2, bs, 4, nb)
        args = [_dev(qp), _dev(kp), _dev(v), _i(cu), _i(np.concatenate([pos, [0, 0]])), _i(np.concatenate([slots, [-1, -1]]))]
        start = [_codes(kc), _codes(vc), _f(ks), _f(vs)]
        eager, pools = [t.clone() for t in start], [t.clone() for t in start]
        want = _append(kl, rc, 16, 4, *args, eager)
        torch.cuda.synchronize()
        st, out = torch.cuda.Stream(), torch.full_like(want, 7.0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            for p_, s_ in zip(pools, start):
                p_.view(torch.uint8).copy_(s_.view(torch.uint8))
            _append(kl, rc, 16, 4, *args, pools, out, stream=st)
        sets.append((graph, st, pools, eager, out, want, args, start))      # the graph reads the inputs
    for _ in range(10):
        for graph, st, *_ in sets:
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    assert kl.kl_device_status() == 0
    for graph, st, pools, eager, out, want, *_ in sets:
        assert torch.equal(out, want) and all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(pools, eager))


def test_append_nonfinite_and_zeros(kl):
    """Infinities and NaN are held as NaN and do not count for the scale; a page of zeros has the least scale; a scale that a begun
    page had before is forgotten, a NaN among them."""
    Hq, Hkv, bs, T = 8, 2, 16, 40
    rng = np.random.default_rng(9)
    q, k, v = (_bf(rng, T, h, D) for h in (Hq, Hkv, Hkv))
    k[3, 0, 5], k[9, 1, 100], v[20, 0, 7], v[21, 1, :] = np.inf, np.nan, -np.inf, np.nan
    k[16:32, 1], v[32:40, 0] = 0.0, 0.0
    rc = kl.RaggedCfg(1, T, bs, 4, 4)
    slots = np.concatenate([np.arange(32, 64), np.arange(8)])
    pools = [np.zeros((4, bs, Hkv, D)), np.full((4, Hkv), np.nan)]
    qd, kd, vd = (torch.as_tensor(x).to(torch.bfloat16).cuda() for x in (q, k, v))
    kpd, ksd, vpd, vsd = _codes(pools[0]), _f(pools[1]), _codes(pools[0]), _f(pools[1])
    cu, pd, sd = _i([0, T]), _i(np.zeros(T)), _i(slots)
    kl.kl_ragged_qkv_rope8(rc, Hq, Hkv, D, kl.KL_BF16, qd.data_ptr(), kd.data_ptr(), vd.data_ptr(), 0, 0, 1e-6, 1e6, 0, cu.data_ptr(), pd.data_ptr(), sd.data_ptr(),
                           qd.data_ptr(), kpd.data_ptr(), vpd.data_ptr(), ksd.data_ptr(), vsd.data_ptr())
    assert kl.kl_device_status() == 0
    # position zero: no rotation. The partner of an infinity is inf * 0 = NaN after the rotation, as 1 * x - 0 * inf is.
    k = np.where(np.isfinite(k), k, np.nan)
    for j in (0, 1):
        part = np.concatenate([k[:, j, D // 2:], k[:, j, :D // 2]], -1)
        k[:, j] = np.where(np.isnan(part), np.nan, k[:, j])
    want = O.cache8_append(k, slots, *[np.nan_to_num(x) for x in pools]), O.cache8_append(v, slots, *[np.nan_to_num(x) for x in pools])
    for (p, s), gp, gs in zip(want, (kpd, vpd), (ksd, vsd)):
        np.testing.assert_array_equal(_host(gp)[[0, 2, 3]], p[[0, 2, 3]])
        np.testing.assert_array_equal(_host(gs)[[0, 2, 3]], s[[0, 2, 3]])
        assert torch.isnan(gs[1]).all()                     # a block that the step does not touch
    assert float(vsd[0, 0]) == 2.0 ** -64 and float(ksd[3, 1]) == 2.0 ** -64


def test_append_reports_a_slot_past_the_pool(kl):
    rc = kl.RaggedCfg(1, 3, 16, 2, 2)
    q, k = torch.randn(3, 8, D, device="cuda").bfloat16(), torch.randn(3, 1, D, device="cuda").bfloat16()
    guard = torch.zeros(3, 16, 1, D, device="cuda", dtype=torch.uint8)
    scale = torch.zeros(3, 1, device="cuda")
    cu, pos, slots = _i([0, 3]), _i([0, 1, 2]), _i([32, 33, 5])
    g2, s2 = guard.clone(), scale.clone()
    kl.kl_ragged_qkv_rope8(rc, 8, 1, D, kl.KL_BF16, q.data_ptr(), k.data_ptr(), k.data_ptr(), 0, 0, 1e-6, 1e6, 0, cu.data_ptr(), pos.data_ptr(), slots.data_ptr(), q.data_ptr(),
                           guard.data_ptr(), g2.data_ptr(), scale.data_ptr(), s2.data_ptr())
    with pytest.raises(kl.KLError) as e:
        kl.kl_device_status()
    assert "0x8" in str(e.value)
    for g in (guard, g2):
        got = g.view(48, D)
        assert (got[:5] == 0).all() and (got[5] != 0).any() and (got[6:] == 0).all()
    assert (scale[1:] == 0).all() and (scale[0] > 0).all()


def test_append_offsets_past_32_bits(kl):
    Hq, Hkv, bs, nb = 8, 8, 16, 270000
    kp, vp = (torch.zeros(nb, bs, Hkv, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(nb, Hkv, device="cuda") for _ in range(2))
    rng = np.random.default_rng(62)
    T = 20
    slots = np.concatenate([np.arange((nb - 1) * bs + 5, nb * bs), np.arange(7 * bs, 7 * bs + 9)])
    q, k, v = _bf(rng, T, Hq, D), _bf(rng, T, Hkv, D), _bf(rng, T, Hkv, D)
    kp[nb - 1, :5] = vp[nb - 1, :5] = 0x38       # ones
    rc = kl.RaggedCfg(1, T, bs, 4, nb)
    qd, kd, vd, cu, pd, sd = _dev(q), _dev(k), _dev(v), _i([0, T]), _i(np.zeros(T)), _i(slots)
    ks[nb - 1] = vs[nb - 1] = 2.0 ** -20
    kl.kl_ragged_qkv_rope8(rc, Hq, Hkv, D, kl.KL_BF16, qd.data_ptr(), kd.data_ptr(), vd.data_ptr(), 0, 0, 1e-6, 1e6, 0, cu.data_ptr(), pd.data_ptr(), sd.data_ptr(),
                           qd.data_ptr(), kp.data_ptr(), vp.data_ptr(), ks.data_ptr(), vs.data_ptr())
    assert kl.kl_device_status() == 0
    for x, pool, scale in ((k, kp, ks), (v, vp, vs)):
        small, s0 = np.zeros((2, bs, Hkv, D)), np.full((2, Hkv), 2.0 ** -20)
        small[0, :5] = 1.0
        p, s = O.cache8_append(x, np.where(slots >= 8 * bs, slots - (nb - 1) * bs, slots - 6 * bs), small, s0)
        np.testing.assert_array_equal(_host(pool[[nb - 1, 7]].view(E4M3)), p)
        np.testing.assert_array_equal(_host(scale[[nb - 1, 7]]), s)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("qk_norm,inter", [(False, False), (True, True)])
def test_layer_forward(kl, qk_norm, inter):
    """The layer over 8-bit pages against the parts it is made of, and within the cache's rounding of the bf16 layer."""
    H, Hq, Hkv, I, bs = 256, 4, 2, 512, 16
    reqs = [(1, 20), (20, 0), (0, 9), (3, 45), (70, 100)]
    rng, n, ctx, table, maxb, nb, (kc, ks, vc, vs), cu, T = _step8(21, reqs, Hkv, bs)
    ks, vs = np.nan_to_num(ks, nan=1.0), np.nan_to_num(vs, nan=1.0)
    kc, vc = np.nan_to_num(kc), np.nan_to_num(vc)
    w = synth.layer_weights(21, H, Hq, Hkv, D, I, bf16=True, qk_norm=qk_norm)
    cfg = L.make_cfg(1, T, H, Hq, Hkv, D, I, dtype=kl.KL_BF16, qk_norm=qk_norm, rope_interleaved=inter)
    rc = kl.RaggedCfg(len(reqs), T, bs, maxb, nb)
    wd = {k: L.to_device(w[L.SYNTH_NAMES[k]], kl.KL_BF16, "cuda") for k in L.weight_fields(cfg)}
    X = _dev(synth.layer_inputs(21, T, H, bf16=True)["X"])
    pos = np.concatenate([np.arange(c, c + k) for k, c in reqs])
    req = np.repeat(np.arange(len(reqs)), n)
    slots = table[req, pos // bs] * bs + pos % bs
    td, cd, xd, pd, sd = _i(table), _i(cu), _i(ctx), _i(pos), _i(slots)
    p8 = [_codes(kc), _codes(vc), _f(ks), _f(vs)]
    ws = torch.empty(kl.kl_layer_forward_ragged8_ws_bytes(cfg, rc), dtype=torch.uint8, device="cuda")
    Y = torch.empty_like(X)
    kl.kl_layer_forward_ragged8(cfg, rc, L.weights_struct(wd), X.data_ptr(), Y.data_ptr(), *[t.data_ptr() for t in p8], td.data_ptr(), cd.data_ptr(), xd.data_ptr(),
                                pd.data_ptr(), sd.data_ptr(), ws.data_ptr(), ws.numel())
    assert kl.kl_device_status() == 0
    # the bf16 layer over the dequantised pages: its new keys and values are not rounded to 8 bits
    k16, v16 = _dev(O.dequantised(kc, ks)), _dev(O.dequantised(vc, vs))
    Y16 = torch.empty_like(X)
    w2 = torch.empty(kl.kl_layer_forward_ragged_ws_bytes(cfg, rc), dtype=torch.uint8, device="cuda")
    kl.kl_layer_forward_ragged(cfg, rc, L.weights_struct(wd), X.data_ptr(), Y16.data_ptr(), k16.data_ptr(), v16.data_ptr(), td.data_ptr(), cd.data_ptr(), xd.data_ptr(),
                               pd.data_ptr(), sd.data_ptr(), w2.data_ptr(), w2.numel())
    assert kl.kl_device_status() == 0
    # e4m3 is off by 2^-4 at most, about 2^-5.6 on average, of each key and value: the residual stream dilutes it
    assert_rel(_host(Y), _host(Y16), 2.0 ** -4, "Y")
    # the pages: the bf16 layer's keys and values are the same projections' (bf16), so the codes are within half a step of them
    for c8, s8, x16, old in ((p8[0], p8[2], k16, ks), (p8[1], p8[3], v16, vs)):
        got, s = _host(c8).reshape(-1, Hkv, D)[slots], _host(s8)
        y = _host(x16).reshape(-1, Hkv, D)[slots]
        sc = s[slots // bs][..., None]
        # bf16 keys are off by 2^-9 of themselves before, the fp32 ones behind these codes not
        assert (np.abs(got * sc - y) <= O.e4m3_half_step(np.abs(y / sc) * (1 + 2.0 ** -8)) * sc + 2.0 ** -8 * np.abs(y)).all()
        assert (s >= old * (s == old)).all()
    # a second call of the same step: same bits, the pages as they are
    again = [t.clone() for t in p8]
    Y2 = torch.empty_like(X)
    kl.kl_layer_forward_ragged8(cfg, rc, L.weights_struct(wd), X.data_ptr(), Y2.data_ptr(), *[t.data_ptr() for t in again], td.data_ptr(), cd.data_ptr(), xd.data_ptr(),
                                pd.data_ptr(), sd.data_ptr(), ws.data_ptr(), ws.numel())
    assert torch.equal(Y, Y2) and all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(p8, again))


def test_a_captured_serving_loop(kl):
    """plan -> append -> attention -> log probabilities captured once and replayed over steps of different lengths (a prompt, rejected
    drafts, an ended request and its successor), each checked against the oracle's pages."""
    B, T, bs, maxb, nb, Hq, Hkv, V = 3, 64, 8, 16, 40, 8, 2, 50
    rng = np.random.default_rng(31)
    s = Planner(kl, B, T, bs, maxb, nb, rng.permutation(nb), nb)
    bf = torch.bfloat16
    q, k, v = (torch.zeros(T, h, D, dtype=bf, device="cuda") for h in (Hq, Hkv, Hkv))
    qr, o = torch.zeros_like(q), torch.zeros_like(q)
    kp, vp = (torch.full((nb, bs, Hkv, D), float("nan"), device="cuda").to(E4M3) for _ in range(2))
    ks, vs = (torch.full((nb, Hkv), float("nan"), device="cuda") for _ in range(2))
    z, tok = torch.zeros(T, V, device="cuda"), _i(np.zeros(T))
    lp, ent = torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda")
    ti, tl = _i(np.zeros((T, 4))), torch.zeros(T, 4, device="cuda")
    ws = torch.empty(kl.kl_ragged_attention8_ws_bytes(s.rc, Hq, Hkv, D), dtype=torch.uint8, device="cuda")

    def body():
        s.launch()
        kl.kl_ragged_qkv_rope8(s.rc, Hq, Hkv, D, kl.KL_BF16, q.data_ptr(), k.data_ptr(), v.data_ptr(), 0, 0, 1e-6, 1e4, 0, s.cu.data_ptr(), s.pos.data_ptr(), s.slots.data_ptr(),
                               qr.data_ptr(), kp.data_ptr(), vp.data_ptr(), ks.data_ptr(), vs.data_ptr())
        _attend_into(kl, s, Hq, Hkv, qr, kp, ks, vp, vs, o, ws)
        kl.kl_token_logprobs(T, V, kl.KL_F32, z.data_ptr(), V, tok.data_ptr(), 4, lp.data_ptr(), ent.data_ptr(), 0, ti.data_ptr(), tl.data_ptr())

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        body()                                   # the first call outside the capture (an empty step)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        body()
    ctx = np.zeros(B, int)
    for step in range(8):
        n = [[30, 1, 0], [3, 4, 17], [1, 1, 1], [4, -1, 2], [2, 9, 4], [0, 1, 5], [5, 5, 5], [1, 2, 0]][step]
        for t in (q, k, v):
            t.copy_(torch.as_tensor(_bf(rng, *t.shape) * 2.0 ** (step - 3)))
        z.copy_(torch.as_tensor(rng.standard_normal((T, V))))
        tok.copy_(_i(rng.integers(-1, V, T)))
        before = [_host(t) for t in (kp, ks, vp, vs)]
        torch.cuda.synchronize()

        def replay():
            with torch.cuda.stream(side):
                graph.replay()

        r = s.step(n, ctx, replay)
        assert kl.kl_device_status(side) == 0 and r["missing"] == 0
        cu, rows = r["cu"], int(r["cu"][-1])
        after = [_host(t) for t in (kp, ks, vp, vs)]
        y = O.rope_at(_host(k)[:rows], r["pos"], 1e4)
        mag = np.broadcast_to(2 * np.abs(_host(k)[:rows]).max(-1, keepdims=True), y.shape)
        _check_append(y, mag, r["slots"], before[:2], *after[:2])
        _check_append(_host(v)[:rows], mag, r["slots"], before[2:], *after[2:], exact=True)
        lens = np.diff(cu)
        want, _, A = O.ragged_attention(_host(qr)[:rows], O.dequantised(after[0], after[1]), O.dequantised(after[2], after[3]), s.table, cu, np.where(lens > 0, ctx, 0))
        tol, _ = _attention_tol(_host(qr)[:rows], *after, s.table, cu, np.where(lens > 0, ctx, 0), want, A)
        assert (np.abs(_host(o)[:rows] - want) <= tol).all(), step
        w = O.token_logprobs(_host(z), tok.cpu().numpy(), 4)
        assert np.abs(_host(lp) - w["logprob"]).max() < 2e-6 and (ti.cpu().numpy() == w["top_id"]).all()
        for b in range(B):
            ctx[b] = 0 if n[b] < 0 else ctx[b] + (n[b] if step != 1 else (n[b] + 1) // 2)      # step 1: half the drafts are rejected


def _attend_into(kl, s, Hq, Hkv, q, kp, ks, vp, vs, o, ws):
    kl.kl_ragged_attention8(s.rc, Hq, Hkv, D, kl.KL_BF16, q.data_ptr(), kp.data_ptr(), vp.data_ptr(), ks.data_ptr(), vs.data_ptr(), s.d["table"].data_ptr(), s.cu.data_ptr(),
                            s.ctx.data_ptr(), o.data_ptr(), 0, ws.data_ptr(), ws.numel())
