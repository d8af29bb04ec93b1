"""Log probabilities of given tokens, entropies, alternatives and their gradient through the C ABI against the fp64 oracle."""
import numpy as np
import pytest
import torch

import oracle as O
from bwd_qwen3_layer_gb300 import synth

pytestmark = pytest.mark.gpu


def _i(a):
    return torch.as_tensor(np.ascontiguousarray(a).astype(np.int32)).cuda()


def _host(t):
    return t.double().cpu().numpy()


def _logits(rng, N, V, dtype, kind):
    z = rng.standard_normal((N, V)) * 3
    if kind == "masked":
        keep = 10.0 ** -rng.uniform(0, np.log10(V), (N, 1))
        z[rng.random((N, V)) >= keep] = -np.inf
        z[N // 2] = -np.inf
    elif kind == "lowest":                          # masks of the type's lowest value
        z[rng.random((N, V)) < 0.9] = -3.3e38
        z[N // 2] = -3.3e38
    elif kind == "ties":
        z = np.round(z)
        z[N // 2] = 1.5
    elif kind == "rising":                          # the largest are the last, in order
        z = np.sort(z, 1)
    elif kind == "large":
        z = z * 30 + 10000
    elif kind == "peaked":
        z[np.arange(N), rng.integers(0, V, N)] += 200
    z = torch.as_tensor(z, dtype=torch.float32).to(dtype)
    return z


def _forward(kl, z, tok, top, stride=None, stream=None, parts=True):
    N, V = z.shape
    ld = stride or V
    buf = torch.full((N, ld), float("nan"), dtype=z.dtype, device="cuda")
    buf[:, :V] = z
    lp, ent, norm = (torch.full(s, 7.0, device="cuda") for s in ((N,), (N,), (N, 2)))
    ti, tl = torch.full((N, top), -7, dtype=torch.int32, device="cuda"), torch.full((N, top), 7.0, device="cuda")
    kl.kl_token_logprobs(N, V, kl.KL_F32 if z.dtype == torch.float32 else kl.KL_BF16, buf.data_ptr(), ld, tok.data_ptr(), top, lp.data_ptr(), ent.data_ptr() if parts else 0,
                         norm.data_ptr() if parts else 0, ti.data_ptr() if top else 0, tl.data_ptr() if top else 0, stream)
    return lp, ent, norm, ti, tl


def _check(r, w, V):
    lp, ent, norm, ti, tl = (_host(t) for t in r)
    # fp32: z - m is off by 2^-24 of itself, a sum of V positive terms in groups of at most a few hundred by 2^-24 x 300, its logarithm by
    # that; an exponential by 2^-22 of itself and 2^-24 |z - m| of its argument
    fin = np.isfinite(w["logprob"])
    assert (lp[~fin] == w["logprob"][~fin]).all()
    size = np.abs(w["logprob"][fin])
    assert (np.abs(lp[fin] - w["logprob"][fin]) <= 2.0 ** -23 * size + 4e-5).all(), np.abs(lp[fin] - w["logprob"][fin]).max()
    assert (np.abs(ent - w["entropy"]) <= 1e-4).all(), np.abs(ent - w["entropy"]).max()
    np.testing.assert_array_equal(norm[:, 0], w["norm"][:, 0])
    f = np.isfinite(w["norm"][:, 1])
    assert (norm[~f, 1] == w["norm"][~f, 1]).all() and (np.abs(norm[f, 1] - w["norm"][f, 1]) <= 4e-5).all()
    np.testing.assert_array_equal(ti, w["top_id"])
    f = np.isfinite(w["top_logprob"])
    assert (tl[~f] == w["top_logprob"][~f]).all()
    assert (np.abs(tl[f] - w["top_logprob"][f]) <= 2.0 ** -23 * np.abs(w["top_logprob"][f]) + 4e-5).all()


CASES = [
    (1, 1, 0, "plain"), (1, 1, 3, "plain"), (3, 2, 2, "plain"), (5, 7, 32, "plain"), (2, 33, 32, "ties"), (4, 1000, 5, "masked"), (4, 1000, 32, "rising"),
    (3, 4095, 8, "ties"), (7, 4097, 20, "lowest"), (9, 5001, 1, "large"), (2, 8193, 32, "peaked"), (3, 32001, 32, "ties"), (3, 32001, 20, "masked"), (2, 50000, 32, "rising"),
    (2, 151936, 20, "plain"), (40, 30011, 8, "plain"), (1, 300007, 32, "plain"), (2, 1200011, 32, "masked"), (160, 2049, 5, "masked"), (700, 513, 3, "plain"), (1, 2000000, 32, "rising"),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V,top,kind", CASES)
def test_forward_matches_oracle(kl, N, V, top, kind, dtype):
    rng = np.random.default_rng(N + V + top)
    z = _logits(rng, N, V, dtype, kind)
    tok = rng.integers(0, V, N)
    tok[N // 3] = -1 if N > 2 else tok[N // 3]
    zd, td = z.cuda(), _i(tok)
    w = O.token_logprobs(_host(z), tok, top)
    r = _forward(kl, zd, td, top)
    assert kl.kl_device_status() == 0
    _check(r, w, V)
    # rows of any stride and alignment (which says in what groups a row is summed), NaN between them
    for ld in (V + 1, V + 5, (V + 15) // 16 * 16 + 16):
        _check(_forward(kl, zd, td, top, ld), w, V)
    # again, and without entropy and norm: the same bits
    assert all(torch.equal(a, b) for a, b in zip(r, _forward(kl, zd, td, top)))
    r3 = _forward(kl, zd, td, top, parts=False)
    assert torch.equal(r[0], r3[0]) and torch.equal(r[3], r3[3]) and torch.equal(r[4], r3[4]) and (r3[1] == 7.0).all() and (r3[2] == 7.0).all()
    assert kl.kl_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V,top,stride", [(1, 151936, 32, None), (3, 151936, 5, None), (4, 30011, 20, 30013), (700, 9001, 32, 9002), (900, 5003, 1, None)])
def test_alternatives_among_equal_logits(kl, N, V, top, stride, dtype):
    """More equal logits than a list holds: the alternatives are the better ones and the first of the equal ones, wherever these lie."""
    rng = np.random.default_rng(V + top)
    z = np.full((N, V), -3.3e38)
    for n in range(N):
        z[n, rng.choice(V, [0, 3, top - 1, top, 40][n % 5], replace=False)] = rng.standard_normal([0, 3, top - 1, top, 40][n % 5])
        if n % 3 == 1:                              # the equal ones only behind most of the row, but for the row's first class
            z[n, 1:V * 7 // 8] = -np.inf
        elif n % 3 == 2:                            # or the row's last
            z[n, V // 16:V - 2] = -np.inf
    z = torch.as_tensor(z, dtype=torch.float32).to(dtype)
    tok = rng.integers(0, V, N)
    w = O.token_logprobs(z.double().numpy(), tok, top)
    _check(_forward(kl, z.cuda(), _i(tok), top, stride), w, V)
    assert kl.kl_device_status() == 0


@pytest.mark.parametrize("V,top", [(700, 5), (40000, 20)])
def test_forward_nonfinite(kl, V, top):
    rng = np.random.default_rng(1)
    z = rng.standard_normal((6, V)).astype(np.float32)
    z[1, V // 2], z[3, V - 1], z[4, 0] = np.nan, np.inf, -np.inf
    z[5, 3:] = -np.inf
    z[5, 2] = np.nan
    tok = np.array([1, 2, 3, 4, 5, -1])
    lp, ent, norm, ti, tl = _forward(kl, torch.as_tensor(z).cuda(), _i(tok), top)
    assert kl.kl_device_status() == 0
    for n in (1, 3):
        assert torch.isnan(lp[n]) and torch.isnan(ent[n]) and torch.isnan(norm[n, 1])
    assert float(lp[5]) == 0.0 and torch.isnan(ent[5]) and torch.isnan(norm[5, 1])
    w = O.token_logprobs(z[[0, 2, 4]], tok[[0, 2, 4]], top)
    _check([t[[0, 2, 4]] for t in (lp, ent, norm, ti, tl)], w, V)


def test_bad_tokens_are_reported(kl):
    z = torch.randn(4, 100, device="cuda")
    good = _forward(kl, z, _i([5, 6, 7, -1]), 2)
    assert kl.kl_device_status() == 0
    for bad in (100, -2, 1 << 30):
        lp, *rest = _forward(kl, z, _i([5, 6, bad, -1]), 2)
        with pytest.raises(kl.KLError) as e:
            kl.kl_device_status()
        assert e.value.status == kl.KL_ERR_DEVICE and "0x2" in str(e.value)
        assert float(lp[2]) == 0.0 and torch.equal(lp[:2], good[0][:2]) and all(torch.equal(a, b) for a, b in zip(rest, good[1:]))
        dz = torch.full_like(z, 7.0)
        a = torch.ones(4, device="cuda")
        tk = _i([5, 6, bad, -1])
        kl.kl_token_logprobs_bwd(4, 100, kl.KL_F32, z.data_ptr(), 100, tk.data_ptr(), good[2].data_ptr(), 0, a.data_ptr(), 0, kl.KL_F32, dz.data_ptr(), 100)
        with pytest.raises(kl.KLError) as e:
            kl.kl_device_status()
        assert "0x2" in str(e.value)
        assert (dz[2:] == 0).all() and (dz[:2] != 0).any()


def _backward(kl, z, tok, norm, ent, a, b, dt, ld=None, ldd=None, inplace=False):
    N, V = z.shape
    ld = ld or V
    buf = torch.full((N, ld), float("nan"), dtype=z.dtype, device="cuda")
    buf[:, :V] = z
    ldd = ld if inplace else ldd or V
    dz = buf if inplace else torch.full((N, ldd), 7.0, dtype=dt, device="cuda")
    D = lambda t: kl.KL_F32 if t == torch.float32 else kl.KL_BF16  # noqa: E731
    kl.kl_token_logprobs_bwd(N, V, D(z.dtype), buf.data_ptr(), ld, tok.data_ptr(), norm.data_ptr(), kl.ptr(ent), kl.ptr(a), kl.ptr(b), D(dz.dtype), dz.data_ptr(), ldd)
    if ldd > V:
        gap = dz[:, V:]
        assert torch.isnan(gap).all() if inplace else (gap == 7.0).all()      # what lies between the rows stays
    return dz[:, :V]


@pytest.mark.parametrize("dtype,dz_dtype", [(torch.float32, torch.float32), (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("N,V,kind", [(1, 1, "plain"), (3, 2, "plain"), (4, 1000, "masked"), (7, 4097, "lowest"), (3, 8191, "large"), (2, 32001, "peaked"), (5, 33003, "masked"),
                                      (2, 151936, "plain"), (300, 515, "ties")])
def test_backward_matches_oracle(kl, N, V, kind, dtype, dz_dtype):
    rng = np.random.default_rng(V)
    z = _logits(rng, N, V, dtype, kind)
    tok = rng.integers(0, V, N)
    tok[N // 3] = -1 if N > 2 else tok[N // 3]
    if N > 3:
        tok[0] = int(np.argmax(_host(z)[0]))
    a, b = rng.standard_normal(N).astype(np.float32), rng.standard_normal(N).astype(np.float32)
    zd, td, ad, bd = z.cuda(), _i(tok), torch.as_tensor(a).cuda(), torch.as_tensor(b).cuda()
    _, ent, norm, _, _ = _forward(kl, zd, td, 0)
    for use_a, use_b in ((True, True), (True, False), (False, True)):
        want = O.token_logprobs_bwd(_host(z), tok, a * use_a, b * use_b)
        got = _backward(kl, zd, td, norm, ent if use_b else None, ad if use_a else None, bd if use_b else None, dz_dtype)
        assert kl.kl_device_status() == 0
        # p is off by 2^-22 and 2^-24 |log p| of itself and by the norm's error (4e-5, as for the forward), the entropy by 1e-4; with |a|, |b| below 5:
        # 2e-4 p (1 + |log p| + H), which is below 6e-4 sqrt(p) for any p, and half a step of the result's type
        p = np.exp(np.maximum(_host(z) - np.where(np.isfinite(_host(z).max(1)), _host(z).max(1), 0)[:, None], -745))
        p /= np.maximum(p.sum(1, keepdims=True), 1e-300)
        half = torch.finfo(dz_dtype).eps / 2
        # one minus p at the token: the difference is off by what p is
        tol = half * np.abs(want) * 1.01 + 5e-4 * p * (1 + np.abs(np.log(np.maximum(p, 1e-300))) + np.log(V)) + 1e-30
        assert (np.abs(_host(got) - want) <= tol).all(), np.max(np.abs(_host(got) - want) / tol)
    base = _backward(kl, zd, td, norm, ent, ad, bd, dz_dtype)
    for ld, ldd in ((V + 1, V + 3), (V + 8, V + 8), (V + 3, V)):
        assert torch.equal(_backward(kl, zd, td, norm, ent, ad, bd, dz_dtype, ld, ldd), base)
    if dtype == dz_dtype:
        for ld in (V, V + 3):
            assert torch.equal(_backward(kl, zd, td, norm, ent, ad, bd, dz_dtype, ld, inplace=True), base)
    assert kl.kl_device_status() == 0


def test_backward_by_differences(kl):
    """The gradient against differences of the forward's own outputs, along random directions."""
    rng = np.random.default_rng(4)
    N, V = 6, 3001
    z = (rng.standard_normal((N, V)) * 2).astype(np.float32)
    tok = rng.integers(0, V, N)
    a, b = rng.standard_normal(N).astype(np.float32), rng.standard_normal(N).astype(np.float32)
    td = _i(tok)

    def f(z):
        lp, ent, *_ = _forward(kl, torch.as_tensor(z, dtype=torch.float32).cuda(), td, 0)
        return float(np.sum(a * _host(lp) + b * _host(ent)))

    _, ent, norm, _, _ = _forward(kl, torch.as_tensor(z).cuda(), td, 0)
    dz = _host(_backward(kl, torch.as_tensor(z).cuda(), td, norm, ent, torch.as_tensor(a).cuda(), torch.as_tensor(b).cuda(), torch.float32))
    for seed in range(4):
        d = np.random.default_rng(seed).standard_normal((N, V))
        d[np.arange(N), tok] *= 3
        h = 2.0 ** -5
        # second differences of order h^2, the forward's rounding (12 numbers, 4e-5 each at most) over 2 h
        assert abs((f(z + h * d) - f(z - h * d)) / (2 * h) - np.sum(dz * d)) < 12 * 4e-5 / h + 30 * h * h


def test_captured_and_two_streams(kl):
    """A forward and a backward captured into a graph while the same call runs on another stream: the bits of one after the other."""
    rng = np.random.default_rng(5)
    N, V, top = 12, 20011, 20
    zs = [torch.as_tensor(rng.standard_normal((N, V)) * 3, dtype=torch.float32).cuda() for _ in range(3)]
    tok = _i(rng.integers(0, V, N))
    a, b = torch.randn(N, device="cuda"), torch.randn(N, device="cuda")

    def bufs():
        return [torch.zeros(N, V, device="cuda"), torch.zeros(N, device="cuda"), torch.zeros(N, device="cuda"), torch.zeros(N, 2, device="cuda"),
                torch.zeros(N, top, dtype=torch.int32, device="cuda"), torch.zeros(N, top, device="cuda"), torch.zeros(N, V, device="cuda")]

    def call(t, st=None):
        kl.kl_token_logprobs(N, V, kl.KL_F32, t[0].data_ptr(), V, tok.data_ptr(), top, *[x.data_ptr() for x in t[1:6]], st)
        kl.kl_token_logprobs_bwd(N, V, kl.KL_F32, t[0].data_ptr(), V, tok.data_ptr(), t[3].data_ptr(), t[2].data_ptr(), a.data_ptr(), b.data_ptr(), kl.KL_F32, t[6].data_ptr(), V, st)

    alone = []
    for z in zs:
        t = bufs()
        t[0].copy_(z)
        call(t)
        torch.cuda.synchronize()
        alone.append(t)
    g, e = bufs(), bufs()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s1):
        call(g)
    for i in range(6):
        g[0].copy_(zs[i % 3])
        e[0].copy_(zs[(i + 1) % 3])
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            graph.replay()
        call(e, s2)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(g, alone[i % 3])) and all(torch.equal(x, y) for x, y in zip(e, alone[(i + 1) % 3]))
    assert kl.kl_device_status() == 0


def test_offsets_past_32_bits(kl):
    """Logits past 2^31 elements: the rows at their end."""
    N, V = 15000, 151936
    z = torch.zeros(N, V, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    z[-2:] = 3 * torch.randn(2, V, generator=g, device="cuda")
    tok = torch.full((N,), 7, dtype=torch.int32, device="cuda")
    lp, ent, norm = torch.empty(N, device="cuda"), torch.empty(N, device="cuda"), torch.empty(N, 2, device="cuda")
    ti, tl = torch.empty(N, 3, dtype=torch.int32, device="cuda"), torch.empty(N, 3, device="cuda")
    kl.kl_token_logprobs(N, V, kl.KL_BF16, z.data_ptr(), V, tok.data_ptr(), 3, lp.data_ptr(), ent.data_ptr(), norm.data_ptr(), ti.data_ptr(), tl.data_ptr())
    assert kl.kl_device_status() == 0
    rows = _host(z[-2:])
    w = O.token_logprobs(rows, [7, 7], 3)
    _check([t[-2:] for t in (lp, ent, norm, ti, tl)], w, V)
    assert (ti[:-2] == torch.arange(3, device="cuda")).all() and (lp[:-2] + float(np.log(V))).abs().max() < 4e-5
    a = torch.randn(N, device="cuda")
    kl.kl_token_logprobs_bwd(N, V, kl.KL_BF16, z.data_ptr(), V, tok.data_ptr(), norm.data_ptr(), ent.data_ptr(), a.data_ptr(), a.data_ptr(), kl.KL_BF16, z.data_ptr(), V)
    assert kl.kl_device_status() == 0
    want = O.token_logprobs_bwd(rows, [7, 7], _host(a[-2:]), _host(a[-2:]))
    assert np.linalg.norm(_host(z[-2:]) - want) <= 2.0 ** -8 * np.linalg.norm(want)


@pytest.mark.parametrize("first", ["z", "dz"])
def test_backward_side_by_side(kl, first):
    """The gradient in the other half of the logits' rows: no overlap. Four columns further in is one."""
    rng = np.random.default_rng(8)
    N, V = 5, 1004
    buf = torch.full((N, 2 * V), 7.0, device="cuda")
    z, dz = (buf[:, :V], buf[:, V:]) if first == "z" else (buf[:, V:], buf[:, :V])
    z.copy_(_logits(rng, N, V, torch.float32, "plain"))
    tok = _i(rng.integers(0, V, N))
    lp, ent, norm, _, _ = _forward(kl, z, tok, 0)
    a, b = torch.randn(N, device="cuda"), torch.randn(N, device="cuda")
    call = lambda g, ld, at: kl.kl_token_logprobs_bwd(N, V, kl.KL_F32, z.data_ptr(), 2 * V, tok.data_ptr(), norm.data_ptr(), ent.data_ptr(), a.data_ptr(), b.data_ptr(),
                                                      kl.KL_F32, at, ld, None)
    apart = torch.empty(N, V, device="cuda")
    before = z.clone()
    call(apart, V, apart.data_ptr())
    call(dz, 2 * V, dz.data_ptr())
    assert kl.kl_device_status() == 0
    assert torch.equal(dz, apart) and torch.equal(z, before)
    with pytest.raises(kl.KLError, match="overlaps"):
        call(dz, 2 * V, dz.data_ptr() + (-16 if first == "z" else 16))
    assert torch.equal(z, before)
