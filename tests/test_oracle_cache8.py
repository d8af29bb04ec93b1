"""The oracle of the 8-bit cache and of the token log probabilities pinned by definitions, brute force and differences, and the
refusals of their entry points. CPU only."""
import ctypes
import os

import numpy as np
import pytest
import torch

import bwd_qwen3_layer_gb300 as K
import oracle as O


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(K.LIB_PATH):
        import __graft_entry__ as g
        g.build()
    return K.load()


def test_codes_are_those_of_e4m3():
    want = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(O.e4m3_values(), want)


def test_rounding_is_to_the_nearest_code():
    v = O.e4m3_values()
    pos = np.sort(np.unique(v[np.isfinite(v) & (v >= 0)]))
    mid = (pos[1:] + pos[:-1]) / 2
    even = np.where(np.searchsorted(pos, pos[:-1]) % 2 == 0, pos[:-1], pos[1:])      # codes count up with the values
    np.testing.assert_array_equal(O.e4m3_round(mid), even)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-448, 448, 2000), rng.uniform(-0.05, 0.05, 2000)])
    near = pos[np.abs(np.abs(x)[:, None] - pos[None]).argmin(1)] * np.sign(x)
    np.testing.assert_array_equal(O.e4m3_round(x), near)
    assert (np.abs(O.e4m3_round(x) - x) <= O.e4m3_half_step(x)).all()
    assert np.isnan(O.e4m3_round([np.inf, -np.inf, np.nan])).all()


def test_scales():
    for a, w in ((0.0, 2.0 ** -64), (448.0, 1.0), (448.01, 2.0), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8), (1.76, 2.0 ** -7), (1e-30, 2.0 ** -64), (3e38, 2.0 ** 120)):
        assert float(O.scale_for(a)) == w
        assert a / w <= 448 and (w == 2.0 ** -64 or a / (w / 2) > 448)


def test_filling_a_block_in_any_steps_gives_the_codes_of_its_last_scale():
    """Scales are powers of two: a block filled a token at a time holds what one filled at once does, but for subnormal codes."""
    rng = np.random.default_rng(1)
    y = rng.standard_normal((16, 2, 128)) * np.exp(rng.standard_normal((16, 1, 1)))
    slots = np.arange(32, 48)
    pool, scale = np.zeros((4, 16, 2, 128)), np.full((4, 2), np.nan)
    once = O.cache8_append(y, slots, pool, scale)
    p, s = pool, scale
    for i in range(16):
        p, s = O.cache8_append(y[i:i + 1], slots[i:i + 1], p, s)
    np.testing.assert_array_equal(once[1][2], s[2])
    a, b = once[0][2], p[2]
    normal = np.abs(a) >= 2.0 ** -5          # a code of half that size may have been rounded as a subnormal one
    np.testing.assert_array_equal(a[normal], b[normal])
    # each of at most 16 growths rounds by half of 2^-9 of its scale, at least halved by each later one
    assert (np.abs(a - b) <= 2.0 ** -9 + 1e-12).all()


def test_logprobs_by_brute_force():
    rng = np.random.default_rng(2)
    z = rng.standard_normal((6, 40)) * 3
    z[1, 5:] = -np.inf
    z[2] = -np.inf
    z[3, 7] = z[3, 3] = z[3].max() + 1
    tok = np.array([3, 0, 4, 7, -1, 39])
    r = O.token_logprobs(z, tok, 6)
    for n in (0, 1, 3, 5):
        p = torch.softmax(torch.as_tensor(z[n]), 0)
        assert abs(r["logprob"][n] - float(torch.log(p[tok[n]]))) < 1e-12
        assert abs(r["entropy"][n] + float(torch.xlogy(p, p).sum())) < 1e-12
        assert abs(r["norm"][n].sum() - float(torch.logsumexp(torch.as_tensor(z[n]), 0))) < 1e-12
    assert list(r["top_id"][3][:2]) == [3, 7]
    assert list(r["top_id"][1][5:]) == [-1] and (r["top_id"][2] == -1).all()
    assert r["logprob"][2] == -np.inf and r["entropy"][2] == 0 and r["logprob"][4] == 0


def test_logprobs_gradient_by_differences():
    rng = np.random.default_rng(3)
    z = rng.standard_normal((4, 12))
    z[1, 4:9] = -np.inf
    tok = np.array([3, 0, -1, 11])
    a, b = rng.standard_normal(4), rng.standard_normal(4)

    def f(z):
        r = O.token_logprobs(z, tok, 0)
        return np.sum(a * r["logprob"] * (tok >= 0) + b * r["entropy"])

    dz = O.token_logprobs_bwd(z, tok, a, b)
    for n in range(4):
        for j in range(12):
            if z[n, j] == -np.inf:
                assert dz[n, j] == 0
                continue
            up, dn = z.copy(), z.copy()
            up[n, j] += 1e-5
            dn[n, j] -= 1e-5
            assert abs((f(up) - f(dn)) / 2e-5 - dz[n, j]) < 1e-8     # a third derivative of order one times 1e-10, rounding 1e-16 / 1e-5


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def _rc(**kw):
    base = dict(B=3, T=64, block_size=16, max_blocks=8, n_blocks=24)
    base.update(kw)
    return K.RaggedCfg(**base)


def test_append_refusals(lib):
    def call(rc=None, Hq=64, Hkv=8, d=128, dtype=K.KL_BF16, eps=1e-6, base=1e6, inter=0, **ptr):
        a = dict(q=0x1000, k=0x2000, v=0x3000, gq=None, gk=None)
        b = dict(cu=0x4004, pos=0x5004, slots=0x6004, out=0x7000, kp=0x8000, vp=0x9000, ks=0xa004, vs=0xb004)
        for d_ in (a, b):
            d_.update({n: x for n, x in ptr.items() if n in d_})
        return lib.kl_ragged_qkv_rope8(ctypes.byref(rc or _rc()), Hq, Hkv, d, dtype, *a.values(), eps, base, inter, *b.values(), None)

    assert call(d=64) == K.KL_ERR_UNSUPPORTED
    assert call(dtype=K.KL_F32) == K.KL_ERR_UNSUPPORTED
    assert call(rc=_rc(T=(1 << 24) + 1)) == K.KL_ERR_UNSUPPORTED
    for bad in (dict(Hq=6, Hkv=4), dict(rc=_rc(T=0)), dict(base=0.5), dict(eps=-1.0), dict(inter=2), dict(gq=0x1000)):
        assert call(**bad) == K.KL_ERR_INVALID_ARG, bad
    for n in ("q", "k", "v", "out", "kp", "vp"):
        assert call(**{n: None}) == K.KL_ERR_INVALID_ARG
        assert call(**{n: 0x1008}) == K.KL_ERR_INVALID_ARG
    for n in ("cu", "pos", "slots", "ks", "vs"):
        assert call(**{n: None}) == K.KL_ERR_INVALID_ARG
        assert call(**{n: 0x1002}) == K.KL_ERR_INVALID_ARG


def test_attention_refusals(lib):
    def call(Hq=64, Hkv=8, d=128, dtype=K.KL_BF16, lse=0x9004, ws=0x10000, nb=1 << 40, **ptr):
        a = dict(q=0x1000, kp=0x2000, vp=0x3000, ks=0x4004, vs=0x5004, table=0x6004, cu=0x7004, ctx=0x8004, o=0xa000)
        a.update(ptr)
        return lib.kl_ragged_attention8(ctypes.byref(_rc()), Hq, Hkv, d, dtype, *a.values(), lse, ws, nb, None)

    assert K.kl_ragged_attention8_ws_bytes(_rc(), 64, 8, 128) > 0
    assert K.kl_ragged_attention8_ws_bytes(_rc(), 64, 8, 64) == 0
    assert call(Hq=6, Hkv=4) == K.KL_ERR_INVALID_ARG
    assert call(d=64) == K.KL_ERR_UNSUPPORTED
    assert call(dtype=K.KL_F32) == K.KL_ERR_UNSUPPORTED
    assert call(Hq=258, Hkv=2) == K.KL_ERR_UNSUPPORTED
    assert call(lse=0x1002) == K.KL_ERR_INVALID_ARG
    for n in ("q", "kp", "vp", "o"):
        assert call(**{n: None}) == K.KL_ERR_INVALID_ARG
        assert call(**{n: 0x1008}) == K.KL_ERR_INVALID_ARG
    for n in ("ks", "vs", "table", "cu", "ctx"):
        assert call(**{n: None}) == K.KL_ERR_INVALID_ARG
        assert call(**{n: 0x1002}) == K.KL_ERR_INVALID_ARG
    assert call(o=0x7010) == K.KL_ERR_INVALID_ARG
    assert call(ws=None) == K.KL_ERR_NO_MEMORY
    assert call(ws=0x10080) == K.KL_ERR_NO_MEMORY
    assert call(nb=16) == K.KL_ERR_NO_MEMORY


def test_layer_refusals(lib):
    cfg = K.LayerCfg(1, 64, 256, 4, 2, 128, 512, 1e-6, 1e6, K.KL_BF16, 0, 0)
    w = K.LayerWeights(*([0x1000] * 9))
    assert K.kl_layer_forward_ragged8_ws_bytes(cfg, _rc()) > 0
    assert K.kl_layer_forward_ragged8_ws_bytes(cfg, _rc(T=63)) == 0

    def call(ws=0x10000, nb=1 << 40, **ptr):
        a = dict(X=0x1000, Y=0x2000, kp=0x3000, vp=0x4000, ks=0x5004, vs=0x6004, table=0x5004, cu=0x6004, ctx=0x7004, pos=0x8004, slots=0x9004)
        a.update(ptr)
        return lib.kl_layer_forward_ragged8(ctypes.byref(cfg), ctypes.byref(_rc()), ctypes.byref(w), *a.values(), ws, nb, None)

    assert call(ws=None) == K.KL_ERR_NO_MEMORY
    assert call(nb=1024) == K.KL_ERR_NO_MEMORY
    for n in ("X", "Y", "kp", "vp", "ks", "vs", "table", "cu", "ctx", "pos", "slots"):
        assert call(**{n: None}) == K.KL_ERR_INVALID_ARG


def test_logprobs_refusals(lib):
    def call(N=4, V=100, dtype=K.KL_F32, z=0x1000, ldz=100, tok=0x2004, top=5, lp=0x3004, ent=0x4004, norm=0x5004, ti=0x6004, tl=0x7004):
        return lib.kl_token_logprobs(N, V, dtype, z, ldz, tok, top, lp, ent, norm, ti, tl, None)

    for bad in (dict(N=0), dict(V=0), dict(ldz=99), dict(dtype=7), dict(z=None), dict(z=0x1008), dict(tok=None), dict(tok=0x2002), dict(top=-1), dict(top=33), dict(lp=None),
                dict(lp=0x3001), dict(ent=0x4002), dict(norm=0x5002), dict(ti=None), dict(tl=None), dict(ti=0x6001)):
        assert call(**bad) == K.KL_ERR_INVALID_ARG, bad
    assert call(N=(1 << 24) + 1) == K.KL_ERR_UNSUPPORTED
    assert call(V=(1 << 30) + 1, ldz=1 << 31) == K.KL_ERR_UNSUPPORTED

    def grad(N=4, V=100, dtype=K.KL_F32, z=0x10000, ldz=100, tok=0x2004, norm=0x3004, ent=0x4004, dlp=0x5004, dent=0x6004, dt=K.KL_F32, dz=0x20000, lddz=100):
        return lib.kl_token_logprobs_bwd(N, V, dtype, z, ldz, tok, norm, ent, dlp, dent, dt, dz, lddz, None)

    for bad in (dict(N=0), dict(V=0), dict(ldz=99), dict(lddz=99), dict(dtype=7), dict(dt=7), dict(z=None), dict(dz=None), dict(dz=0x20004), dict(tok=None), dict(norm=None),
                dict(norm=0x3001), dict(ent=None), dict(dlp=0x5001), dict(dent=0x6001),
                dict(dz=0x10010), dict(dz=0x10000, lddz=104), dict(dz=0x10000, dt=K.KL_BF16), dict(z=0x1ff00)):       # overlaps that are not in place
        assert grad(**bad) == K.KL_ERR_INVALID_ARG, bad
    assert grad(N=(1 << 24) + 1) == K.KL_ERR_UNSUPPORTED
