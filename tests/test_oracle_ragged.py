"""Pins of the ragged step's oracle and the refusals of its entry points (CPU only: no call here launches a kernel)."""
import ctypes
import os

import numpy as np
import pytest

import bwd_qwen3_layer_gb300 as K
import oracle as O


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(K.LIB_PATH):
        import __graft_entry__ as g
        g.build()
    return K.load()


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------

def test_plan_keeps_every_block_exactly_once():
    """Over a random run of steps no block is lost or given twice, and every row's slot lies in its request's own blocks."""
    rng = np.random.default_rng(0)
    B, bs, maxb, nb = 6, 4, 8, 30
    table, held, ctx = np.full((B, maxb), -1), np.zeros(B, int), np.zeros(B, int)
    free, n_free = rng.permutation(nb), nb
    seen_missing = False
    for _ in range(200):
        n = np.where(rng.random(B) < 0.15, -1, np.minimum(rng.integers(0, 6, B), maxb * bs - ctx))
        r = O.ragged_plan(n, ctx, table, held, free, n_free, bs, 100)
        table, held, free, n_free = r["table"], r["held"], r["free_list"], r["n_free"]
        owned = [int(table[b, i]) for b in range(B) for i in range(held[b])]
        assert sorted(owned + list(free[:n_free])) == list(range(nb))
        for b in range(B):
            s = r["slots"][r["cu"][b]:r["cu"][b + 1]]
            assert all(x < 0 or x // bs in table[b, :held[b]] for x in s)
            if r["missing"] == 0:
                assert (s >= 0).all()
        seen_missing |= r["missing"] > 0
        got = np.array([(r["slots"][r["cu"][b]:r["cu"][b + 1]] >= 0).all() for b in range(B)])
        ctx = np.where(n < 0, 0, np.where(got, ctx + np.maximum(n, 0), ctx))
    assert seen_missing


def test_attention_equals_the_paged_oracle():
    rng = np.random.default_rng(1)
    ctx, n, bs = [3, 0, 9], 2, 4
    kp, vp = rng.standard_normal((12, bs, 2, 8)), rng.standard_normal((12, bs, 2, 8))
    table = rng.permutation(12).reshape(3, 4)
    q = rng.standard_normal((6, 4, 8))
    want, lse = O.paged_attention(q, kp, vp, table, ctx, n)
    got, glse, A = O.ragged_attention(q, kp, vp, table, [0, 2, 4, 6], ctx)
    np.testing.assert_allclose(got, want, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(glse.reshape(3, n, 4).transpose(0, 2, 1), lse, rtol=1e-12)
    assert (A >= np.abs(got) - 1e-12).all()


def test_verify_draws_from_the_target():
    """The tokens that come out follow the target's distribution, whatever the draft's is (10^5 trials, 4 classes: each
    frequency has a standard deviation of at most 0.0016; 6 of them are allowed)."""
    rng = np.random.default_rng(2)
    p, q = np.array([0.1, 0.2, 0.3, 0.4]), np.array([0.5, 0.1, 0.25, 0.15])
    N = 100000
    t = rng.choice(4, N, p=q)
    tokens = np.stack([np.zeros(N, int), t], 1).reshape(-1)
    P, Q = np.tile(p, (2 * N, 1)), np.tile(q, (2 * N, 1))
    acc, nxt = O.draft_verify(P, Q, tokens, np.arange(0, 2 * N + 1, 2), rng.random(2 * N), rng.random(N))
    first = np.where(acc == 1, t, nxt)
    np.testing.assert_allclose(np.bincount(first, minlength=4) / N, p, atol=0.01)
    # without draft probabilities, the same with a fixed draft
    tokens = np.tile([0, 2], N)
    acc, nxt = O.draft_verify(P, None, tokens, np.arange(0, 2 * N + 1, 2), rng.random(2 * N), rng.random(N))
    np.testing.assert_allclose(np.bincount(np.where(acc == 1, 2, nxt), minlength=4) / N, p, atol=0.01)


def test_verify_corners():
    p = np.array([[0.0, 0.5, 0.5], [0.2, 0.3, 0.5]])
    # a draft of probability zero is never accepted, u = 0 gives the first class with a weight
    assert [int(x[0]) for x in O.draft_verify(p, None, [0, 0], [0, 2], [0.0, 0.0], [0.0])] == [0, 1]
    # p = q everywhere: accepted; if the test still fails (u q < p is strict at u = 1), p itself is drawn from
    assert [int(x[0]) for x in O.draft_verify(p, p, [0, 1], [0, 2], [1.0, 0.0], [0.4])] == [0, 1]
    assert [int(x[0]) for x in O.draft_verify(p, p, [0, 1], [0, 2], [0.9, 0.0], [0.4])] == [1, 1]
    assert [list(x) for x in O.draft_verify(p, None, [0, 1], [0, 0, 2], [0.9, 0.0], [0.4, 0.0])] == [[0, 0], [-1, 2]]


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

RC = dict(B=4, T=64, block_size=16, max_blocks=8, n_blocks=64)


def _rc(**kw):
    return K.RaggedCfg(**{**RC, **kw})


def test_plan_refusals(lib):
    def call(rc, ptrs):
        return lib.kl_ragged_plan(None if rc is None else ctypes.byref(rc), *ptrs, None)

    good = [0x1000 + 4 * i for i in range(10)]
    assert call(None, good) == K.KL_ERR_INVALID_ARG
    for bad in (dict(B=0), dict(T=0), dict(block_size=0), dict(max_blocks=-1), dict(n_blocks=0)):
        assert call(_rc(**bad), good) == K.KL_ERR_INVALID_ARG, bad
    assert call(_rc(T=(1 << 24) + 1), good) == K.KL_ERR_UNSUPPORTED
    assert call(_rc(n_blocks=1 << 28), good) == K.KL_ERR_UNSUPPORTED        # slots beyond int32
    for i in range(10):
        assert call(_rc(), good[:i] + [None] + good[i + 1:]) == K.KL_ERR_INVALID_ARG
        assert call(_rc(), good[:i] + [0x1002] + good[i + 1:]) == K.KL_ERR_INVALID_ARG
        assert "aligned" in K.last_error()


def test_qkv_refusals(lib):
    def call(Hq=8, Hkv=2, d=128, dtype=K.KL_BF16, rc=None, base=1e6, eps=1e-6, inter=0, gq=None, gk=None, **ptr):
        a = dict(q=0x1000, k=0x2000, v=0x3000, cu=0x4004, pos=0x5004, slots=0x6004, qo=0x7000, kp=0x8000, vp=0x9000)
        a.update(ptr)
        return lib.kl_ragged_qkv_rope(ctypes.byref(rc or _rc()), Hq, Hkv, d, dtype, a["q"], a["k"], a["v"], gq, gk, eps, base, inter,
                                      a["cu"], a["pos"], a["slots"], a["qo"], a["kp"], a["vp"], None)

    assert call(Hq=6, Hkv=4) == K.KL_ERR_INVALID_ARG
    assert call(Hq=129, Hkv=1) == K.KL_ERR_UNSUPPORTED
    assert call(d=64) == K.KL_ERR_UNSUPPORTED
    assert call(dtype=K.KL_F32) == K.KL_ERR_UNSUPPORTED
    assert call(rc=_rc(n_blocks=1 << 26)) == K.KL_ERR_UNSUPPORTED           # 2^30 rows x 2 heads
    assert call(gq=0x1000) == K.KL_ERR_INVALID_ARG                          # one gain without the other
    assert call(gq=0x1008, gk=0x1000) == K.KL_ERR_INVALID_ARG
    assert call(base=0.5) == K.KL_ERR_INVALID_ARG
    assert call(base=float("nan")) == K.KL_ERR_INVALID_ARG
    assert call(eps=-1.0) == K.KL_ERR_INVALID_ARG
    assert call(inter=2) == K.KL_ERR_INVALID_ARG
    for n in ("q", "k", "v", "qo", "kp", "vp"):
        assert call(**{n: None}) == K.KL_ERR_INVALID_ARG
        assert call(**{n: 0x1008}) == K.KL_ERR_INVALID_ARG
    for n in ("cu", "pos", "slots"):
        assert call(**{n: None}) == K.KL_ERR_INVALID_ARG
        assert call(**{n: 0x1002}) == K.KL_ERR_INVALID_ARG


def test_attention_refusals(lib):
    big = 1 << 30

    def call(Hq=8, Hkv=2, d=128, dtype=K.KL_BF16, rc=None, lse=None, ws=0x10000, nb=big, **ptr):
        a = dict(q=0x1000, kp=0x2000, vp=0x3000, table=0x4004, cu=0x5004, ctx=0x6004, o=0x7000)
        a.update(ptr)
        return lib.kl_ragged_attention(ctypes.byref(rc or _rc()), Hq, Hkv, d, dtype, a["q"], a["kp"], a["vp"], a["table"], a["cu"], a["ctx"],
                                       a["o"], lse, ws, nb, None)

    assert K.kl_ragged_attention_ws_bytes(_rc(), 64, 8, 128) > 0
    assert K.kl_ragged_attention_ws_bytes(_rc(), 64, 8, 64) == 0
    assert K.kl_ragged_attention_ws_bytes(_rc(B=0), 64, 8, 128) == 0
    assert call(Hq=6, Hkv=4) == K.KL_ERR_INVALID_ARG
    assert call(d=64) == K.KL_ERR_UNSUPPORTED
    assert call(dtype=K.KL_F32) == K.KL_ERR_UNSUPPORTED
    assert call(Hq=258, Hkv=2) == K.KL_ERR_UNSUPPORTED
    assert call(lse=0x1002) == K.KL_ERR_INVALID_ARG
    for n in ("q", "kp", "vp", "o"):
        assert call(**{n: None}) == K.KL_ERR_INVALID_ARG
        assert call(**{n: 0x1008}) == K.KL_ERR_INVALID_ARG
    for n in ("table", "cu", "ctx"):
        assert call(**{n: None}) == K.KL_ERR_INVALID_ARG
    assert call(o=0x7010) == K.KL_ERR_INVALID_ARG                           # written in 32-byte sectors
    assert "32-byte" in K.last_error()
    assert call(ws=None) == K.KL_ERR_NO_MEMORY
    assert call(ws=0x10080) == K.KL_ERR_NO_MEMORY
    assert call(nb=1024) == K.KL_ERR_NO_MEMORY


def test_verify_refusals(lib):
    def call(B=2, T=6, V=100, dtype=K.KL_F32, p=0x1000, ldp=100, q=0x2000, ldq=100, **ptr):
        a = dict(tok=0x3004, cu=0x4004, ua=0x5004, us=0x6004, acc=0x7004, nxt=0x8004)
        a.update(ptr)
        return lib.kl_draft_verify(ctypes.byref(K.VerifyCfg(B, T, V, dtype)), p, ldp, q, ldq, a["tok"], a["cu"], a["ua"], a["us"], a["acc"],
                                   a["nxt"], None)

    assert lib.kl_draft_verify(None, *([0x1000, 1] * 2), *([0x1000] * 6), None) == K.KL_ERR_INVALID_ARG
    for bad in (dict(B=0), dict(T=0), dict(V=0), dict(ldp=99), dict(ldq=99), dict(dtype=9), dict(p=None), dict(p=0x1008), dict(q=0x1008)):
        assert call(**bad) == K.KL_ERR_INVALID_ARG, bad
    assert call(B=(1 << 24) + 1) == K.KL_ERR_UNSUPPORTED
    for n in ("tok", "cu", "ua", "us", "acc", "nxt"):
        assert call(**{n: None}) == K.KL_ERR_INVALID_ARG
        assert call(**{n: 0x1001}) == K.KL_ERR_INVALID_ARG


def test_sizes_past_32_bit_counting_are_refused(lib):
    """Loops over requests and classes step by up to 32768 in 32 bits."""
    p = [0x1000] * 10
    assert lib.kl_ragged_plan(ctypes.byref(_rc(B=(1 << 24) + 1)), *p, None) == K.KL_ERR_UNSUPPORTED
    v = K.VerifyCfg(1, 1, (1 << 30) + 1, K.KL_BF16)
    assert lib.kl_draft_verify(ctypes.byref(v), 0x1000, 1 << 31, None, 0, *p[:6], None) == K.KL_ERR_UNSUPPORTED


def test_layer_refusals(lib):
    def cfg(**kw):
        base = dict(B=1, S=64, H=256, Hq=4, Hkv=2, d=128, I=512, eps=1e-6, rope_base=1e6, dtype=K.KL_BF16)
        base.update(kw)
        return K.LayerCfg(**base)

    assert K.kl_layer_forward_ragged_ws_bytes(cfg(), _rc()) > 0
    assert K.kl_layer_forward_ragged_ws_bytes(cfg(S=63), _rc()) == 0        # S is the step's rows
    assert K.kl_layer_forward_ragged_ws_bytes(cfg(B=2, S=32), _rc()) == 0
    assert K.kl_layer_forward_ragged_ws_bytes(cfg(dtype=K.KL_F32), _rc()) == 0
    assert K.kl_layer_forward_ragged_ws_bytes(cfg(rope_base=0.5), _rc()) == 0
    w = K.LayerWeights(*([0x1000] * 9))

    def call(c=None, w=w, ws=0x10000, nb=1 << 40, **ptr):
        a = dict(X=0x1000, Y=0x2000, kp=0x3000, vp=0x4000, table=0x5004, cu=0x6004, ctx=0x7004, pos=0x8004, slots=0x9004)
        a.update(ptr)
        return lib.kl_layer_forward_ragged(ctypes.byref(c or cfg()), ctypes.byref(_rc()), None if w is None else ctypes.byref(w), *a.values(),
                                           ws, nb, None)

    assert call(w=None) == K.KL_ERR_INVALID_ARG
    assert call(cfg(qk_norm=1)) == K.KL_ERR_INVALID_ARG                     # gains missing
    assert call(ws=None) == K.KL_ERR_NO_MEMORY
    assert call(nb=1024) == K.KL_ERR_NO_MEMORY
    for n in ("X", "Y", "kp", "vp", "table", "cu", "ctx", "pos", "slots"):
        assert call(**{n: None}) == K.KL_ERR_INVALID_ARG
