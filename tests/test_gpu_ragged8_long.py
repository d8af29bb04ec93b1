"""Attention over long 8-bit caches, where the copies keep HBM busy and pieces have many key tiles: against a reference in 64 bits
on the device, and the same bits from run to run."""
import math

import numpy as np
import pytest
import torch

from test_gpu_ragged import D, _i
from test_gpu_ragged8 import E4M3, _attend

pytestmark = pytest.mark.gpu


class Cache:
    """Pages of positive values (so that no key's share is lost in a sum of both signs) and small scores, on the device; NaN codes in
    every slot behind a request's end and in the blocks that nobody has. reqs: (new, cached) tokens."""

    def __init__(self, seed, reqs, Hq, Hkv, bs):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.reqs, self.Hq, self.Hkv, self.bs = reqs, Hq, Hkv, bs
        held = [-(-(n + c) // bs) for n, c in reqs]
        self.nb, self.maxb = sum(held) + 3, max(held) + 1
        order, at = torch.randperm(self.nb, generator=self.gen, device="cuda"), 0
        self.table = torch.full((len(reqs), self.maxb), self.nb + 5, device="cuda")
        there = torch.zeros(self.nb * bs, dtype=torch.bool, device="cuda")
        for b, (n, c) in enumerate(reqs):
            self.table[b, :held[b]] = order[at:at + held[b]]
            at += held[b]
            p = torch.arange(n + c, device="cuda")
            there[self.table[b, p // bs] * bs + p % bs] = True
        self.cu = np.concatenate([[0], np.cumsum([n for n, _ in reqs])])
        self.q = 0.3 * self.rand(int(self.cu[-1]), Hq, D)
        self.k, self.v = (self.rand(self.nb, bs, Hkv, D) for _ in range(2))
        self.v = self.v.abs()
        self.there = there.view(self.nb, bs, 1, 1)

    def rand(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda")

    def codes(self):
        """The pools as codes and scales, and the call's arguments."""
        out = []
        for x in (self.k, self.v):
            m, e = torch.frexp(torch.where(self.there, x, 0.0).abs().amax((1, 3)))
            s = torch.ldexp(torch.ones_like(m), torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-64))
            c = torch.where(self.there, x / s[:, None, :, None], float("nan")).to(E4M3)
            out += [c, s]
        self.kc, self.ks, self.vc, self.vs = out
        self.q = self.q.to(torch.bfloat16)
        self.args = [self.q, *out, self.table.to(torch.int32).contiguous(), _i(self.cu), _i([c for _, c in self.reqs])]
        return self

    def cfg(self, kl):
        return kl.RaggedCfg(len(self.reqs), int(self.cu[-1]), self.bs, self.maxb, self.nb)

    def exact(self, rows=None):
        """(row, o, sum of weights times |values|, largest weight times value scale, sum of the values' codes, bound on a score's error) for
        each row of `rows` (all of a step's, if None) by request and kv head: o and the rest [rows, G, D] or [rows, G, 1], in 64 bits."""
        G = self.Hq // self.Hkv
        for b, (n, c) in enumerate(self.reqs):
            mine = [r for r in (range(int(self.cu[b]), int(self.cu[b + 1])) if rows is None else rows) if self.cu[b] <= r < self.cu[b + 1]]
            p = torch.arange(n + c, device="cuda")
            page, place = self.table[b, p // self.bs], p % self.bs
            for g in range(self.Hkv) if mine else ():
                kc, vc = self.kc[page, place, g].double(), self.vc[page, place, g].double()
                ks, vs = self.ks[page, g].double(), self.vs[page, g].double()
                for i0 in range(0, len(mine), 64):
                    r = mine[i0:i0 + 64]
                    q = self.q[r, g * G:(g + 1) * G].double()
                    z = torch.einsum("rhd,jd->rhj", q, kc) * (ks / math.sqrt(D))
                    seen = p[None, :] <= torch.tensor([c + x - int(self.cu[b]) for x in r], device="cuda")[:, None]
                    w = torch.softmax(z.masked_fill(~seen[:, None, :], -math.inf), -1)
                    wb = w * vs
                    dz = 2.0 ** -16 * q.abs().amax(-1, keepdim=True) * (kc.abs().sum(1) * ks).max() / math.sqrt(D)
                    codes = torch.where(seen[:, None, :], 1.0, 0.0).double() @ vc.abs()
                    yield r, slice(g * G, (g + 1) * G), wb @ vc, wb @ vc.abs(), wb.amax(-1, keepdim=True), codes, dz


def _check(cache, o, rows=None):
    """The bound of tests/test_gpu_ragged8.py: a weight off by 2^-8 and 2^-11 of itself and by 2^-13 of the row's largest, in units of the
    value scale; the queries' two parts; 2^-9 for the running sums; the result rounded to bf16."""
    for r, h, want, size, top, codes, dz in cache.exact(rows):
        tol = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -9 + 2 * dz) * size + 2.0 ** -8 * want.abs() + 2.0 ** -13 * top * codes
        err = (o[r, h].double() - want).abs()
        assert (err <= tol).all(), (r[0], h, float((err / tol).max()))


@pytest.mark.parametrize("reqs", [
    # decoding requests, the last key tile with 1 to 40 keys: a tile that loses its other values is off by 2 % of the whole
    [(1, 128 * (28 + b % 8) + b * 39 // 63) for b in range(64)],
    [(1, 128 * (28 + b % 8) + b * 127 // 63) for b in range(64)],
    [(1500, 9007)], [(1, 32790)], [(3, 700 * b + 5) for b in range(12)] + [(700, 5000)],
], ids=["decode", "decode_any", "chunk", "long", "mixed"])
def test_attention_of_long_caches(kl, reqs):
    """Hundreds of runs: the same bits, and the first one's right."""
    cache = Cache(len(reqs) + reqs[0][1], reqs, 64, 8, 16).codes()
    rc = cache.cfg(kl)
    ws = torch.empty(kl.kl_ragged_attention8_ws_bytes(rc, 64, 8, D), dtype=torch.uint8, device="cuda")
    first, lse = _attend(kl, rc, 64, 8, *cache.args, ws=ws)
    rows = None if len(first) < 100 else sorted(set(np.random.default_rng(1).integers(0, len(first), 150).tolist()) | {0, len(first) - 1})
    _check(cache, first, rows)
    different = torch.zeros((), dtype=torch.int64, device="cuda")
    o = torch.empty_like(first)
    for _ in range(300):
        o.fill_(7.0)
        _attend(kl, rc, 64, 8, *cache.args, lse=False, ws=ws, o=o)
        different += (o.view(torch.int16) != first.view(torch.int16)).any()
    assert kl.kl_device_status() == 0
    assert int(different) == 0 and not bool(torch.isnan(first).any())


def _sink(cache, mass, lift=1.0):
    """Each request's first key takes `mass` of its rows' weight and has a small value; the rest is spread evenly over the other keys. lift:
    the second value's size, which says how coarse the first page's scale is."""
    u = cache.rand(D).sign() * 0.5
    cache.q = u + 0.05 * cache.rand(int(cache.cu[-1]), cache.Hq, D)
    cache.k *= 0.05
    for b, (n, c) in enumerate(cache.reqs):
        page = int(cache.table[b, 0])
        score = math.log(mass / (1 - mass) * (n + c))
        cache.k[page, 0] = u * (score * math.sqrt(D) / float(u @ u))
        cache.v[page, 0] = 0.01 * cache.v[page, 0]
        if cache.bs > 1:
            cache.v[page, 1] *= lift
    return cache.codes()


def _check_relative(cache, o, rows=None):
    """All values positive: the result is off by what a weight is, 2^-9 and 2^-11 of itself, by twice what a score is (below 2^-10), the
    running sums' 2^-9, the rounding to bf16, 2^-8: below 2^-6.2 of it in all. And for each key by half of 2^-16, the least step of the weights'
    parts, where the row's largest weight times scale is held as 2^11 or more: 2^-28 of that, times the key's code."""
    for r, h, want, size, top, codes, dz in cache.exact(rows):
        assert float(dz.max()) < 2.0 ** -10
        err = (o[r, h].double() - want).abs()
        tol = 2.0 ** -6 * want + 2.0 ** -28 * top * codes
        assert (err <= tol).all(), (r[0], h, float((err / tol).max()))


@pytest.mark.parametrize("mass,lift", [(0.3, 1.0), (0.5, 64.0), (0.9, 1.0), (0.95, 8.0)])
@pytest.mark.parametrize("Hq,Hkv,bs,reqs", [
    (64, 8, 16, [(1, 32768), (1, 8191), (1, 2000)]),
    (10, 1, 16, [(1, 9000)]), (11, 1, 16, [(1, 9000)]), (16, 1, 16, [(1, 30000), (1, 700)]),       # 10 rows, 11, 16
    (16, 2, 5, [(1, 8192), (9, 3000)]),
    (64, 8, 16, [(300, 8000)]), (16, 2, 24, [(40, 2000), (1, 17000), (3, 5000)]),
])
def test_attention_with_a_key_that_outweighs_the_others(kl, Hq, Hkv, bs, reqs, mass, lift):
    """What the many small weights add up to is there, in whatever pieces a request is cut: alone, and in a batch."""
    cache = _sink(Cache(len(reqs) + reqs[0][1], reqs, Hq, Hkv, bs), mass, lift)
    rc = cache.cfg(kl)
    o, _ = _attend(kl, rc, Hq, Hkv, *cache.args)
    assert kl.kl_device_status() == 0
    rows = sorted(set(np.random.default_rng(1).integers(0, len(o), 60).tolist()) | set(int(c) for c in cache.cu[:-1]))
    _check_relative(cache, o, rows)
    # the first request alone, and beside 39 others: cut in other places
    n, c = reqs[0]
    q, kc, ks, vc, vs, table, cu, ctx = cache.args
    one = kl.RaggedCfg(1, n, bs, cache.maxb, cache.nb)
    o1, _ = _attend(kl, one, Hq, Hkv, q[:n].contiguous(), kc, ks, vc, vs, table[:1].contiguous(), _i([0, n]), _i([c]))
    many = kl.RaggedCfg(40, 40 * n, bs, cache.maxb, cache.nb)
    o40, _ = _attend(kl, many, Hq, Hkv, q[:n].repeat(40, 1, 1), kc, ks, vc, vs, table[:1].repeat(40, 1), _i(np.arange(41) * n), _i([c] * 40))
    assert kl.kl_device_status() == 0
    _check_relative(cache, o1, [r for r in rows if r < n])
    for b in (0, 17, 39):
        _check_relative(cache, o40[b * n:(b + 1) * n], [r for r in rows if r < n])


@pytest.mark.parametrize("which", ["key", "value"])
@pytest.mark.parametrize("bs", [16, 5])
def test_attention_of_a_block_without_a_scale(kl, bs, which):
    """A NaN scale of a block that only a request's last rows see: these are NaN, the rows of other query tiles, heads and requests as they
    were. (Rows of the same tile before the block may be NaN, too.)"""
    reqs, Hq, Hkv = [(100, 60), (3, 400), (9, 0)], 4, 2          # two heads a group: tiles of 64 tokens
    cache = Cache(3, reqs, Hq, Hkv, bs).codes()
    rc = cache.cfg(kl)
    base, blse = _attend(kl, rc, Hq, Hkv, *cache.args)
    first = 145 // bs * bs                                       # rows from here on see the block: in the second tile
    (cache.ks if which == "key" else cache.vs)[cache.table[0, first // bs], 1] = float("nan")
    o, lse = _attend(kl, rc, Hq, Hkv, *cache.args)
    assert kl.kl_device_status() == 0
    assert torch.isnan(o[first - 60:100, 2:]).all() and torch.isnan(lse[first - 60:100, 2:]).all()
    for a, b in ((o, base), (lse, blse)):
        assert torch.equal(a[:64], b[:64]) and torch.equal(a[100:], b[100:]) and torch.equal(a[:, :2], b[:, :2])


@pytest.mark.parametrize("k", [-60, 0, 60, 110])
def test_lse_beside_value_scales_of_any_size(kl, k):
    """lse does not depend on the value scales but for rounding: 2^-21 of their largest |log2|, beside what a score is off by, the sum's
    2^-24 a key and 2^-22 of the result."""
    reqs, Hq, Hkv, bs = [(3, 500), (40, 100), (1, 2000)], 8, 2, 16
    cache = Cache(5, reqs, Hq, Hkv, bs).codes()
    cache.vs *= 2.0 ** k * (1 + 0.9 * torch.rand(cache.vs.shape, generator=cache.gen, device="cuda"))
    o, lse = _attend(kl, cache.cfg(kl), Hq, Hkv, *cache.args)
    assert kl.kl_device_status() == 0
    for r, h, want, size, top, codes, dz in cache.exact():
        b = int(np.searchsorted(cache.cu, r[0], side="right")) - 1
        p = torch.arange(sum(reqs[b]), device="cuda")
        page, g = cache.table[b, p // bs], h.start // (Hq // Hkv)
        keys = cache.kc[page, p % bs, g].double() * cache.ks[page, g].double()[:, None] / math.sqrt(D)
        z = cache.q[r, h].double() @ keys.T
        seen = p[None, :] <= torch.tensor([reqs[b][1] + x - int(cache.cu[b]) for x in r], device="cuda")[:, None]
        exact = torch.logsumexp(z.masked_fill(~seen[:, None, :], -math.inf), -1)
        tol = dz[..., 0] + 2.0 ** -22 * exact.abs() + len(p) * 2.0 ** -24 + 2.0 ** -21 * cache.vs[page, g].log2().abs().max().double() + 1e-6
        assert ((lse[r, h].double() - exact).abs() <= tol).all()
