"""The ragged step's operators together, in the ways a server runs them: a pool that runs short, room for more rows than a
step has, a captured layer, streams side by side."""
import numpy as np
import pytest
import torch

import oracle as O
from bwd_qwen3_layer_gb300 import layer as L
from bwd_qwen3_layer_gb300 import synth
from _parity import TOL_BF16, assert_rel
from test_gpu_ragged import D, Planner, _bf, _dev, _host, _i, _step

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


# ---------------------------------------------------------------------------
# the layer
# ---------------------------------------------------------------------------

class Layer:
    def __init__(self, kl, seed, reqs, T, H, Hq, Hkv, I, bs, qk_norm):
        self.kl = kl
        self.rng, n, ctx, table, maxb, nb, kp, vp, cu, self.rows = _step(seed, reqs, Hkv, bs)
        self.n, self.ctx, self.table, self.T = n, ctx, table, T
        w = synth.layer_weights(seed, H, Hq, Hkv, D, I, bf16=True, qk_norm=qk_norm)
        self.cfg = L.make_cfg(1, T, H, Hq, Hkv, D, I, dtype=kl.KL_BF16, qk_norm=qk_norm)
        self.rc = kl.RaggedCfg(len(reqs), T, bs, maxb, nb)
        self.w = {k: L.to_device(w[L.SYNTH_NAMES[k]], kl.KL_BF16, "cuda") for k in L.weight_fields(self.cfg)}
        pos = np.concatenate([np.arange(c, c + k) for k, c in reqs])
        req = np.repeat(np.arange(len(reqs)), n)
        # what lies behind the step's rows in the arrays is no position and no slot
        junk = np.full(T - self.rows, 1 << 30)
        self.kp, self.vp, self.td, self.cd, self.xd = _dev(kp), _dev(vp), _i(table), _i(cu), _i(ctx)
        self.pd, self.sd = _i(np.concatenate([pos, junk])), _i(np.concatenate([table[req, pos // bs] * bs + pos % bs, junk]))
        self.X = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.X[:self.rows] = L.to_device(synth.layer_inputs(seed, self.rows, H, bf16=True)["X"], kl.KL_BF16, "cuda")
        self.Y = torch.zeros_like(self.X)
        nbytes = kl.kl_layer_forward_ragged_ws_bytes(self.cfg, self.rc)
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")

    def call(self, X=None, kp=None, vp=None, Y=None, stream=None):
        t = [self.X if X is None else X, self.Y if Y is None else Y, self.kp if kp is None else kp, self.vp if vp is None else vp]
        self.kl.kl_layer_forward_ragged(self.cfg, self.rc, L.weights_struct(self.w), *[x.data_ptr() for x in t], self.td.data_ptr(), self.cd.data_ptr(), self.xd.data_ptr(),
                                        self.pd.data_ptr(), self.sd.data_ptr(), self.ws.data_ptr(), self.ws.numel(), stream)
        return t


@pytest.mark.parametrize("T,reqs", [
    (29, [(1, 20), (20, 0), (0, 9), (3, 45)]),                       # the few-rows products, five rows of room
    (333, [(1, 20), (200, 3), (0, 9), (64, 45), (1, 500)]),          # the tiled products
])
@pytest.mark.parametrize("qk_norm", [False, True])
def test_rows_behind_the_last_request_reach_no_other(kl, T, reqs, qk_norm):
    """NaN in X's rows behind the requests' and in the whole workspace: the bits of the same call with zeros there."""
    a = Layer(kl, 5, reqs, T, 512, 8, 2, 768, 16, qk_norm)
    pools = [torch.nan_to_num(a.kp), torch.nan_to_num(a.vp)]
    outs = []
    for fill, X in ((0x00, torch.nan_to_num(a.X)), (0xff, a.X)):     # 0xffff is a NaN in bf16, 0xffffffff in fp32
        a.ws.fill_(fill)
        kp, vp, Y = pools[0].clone(), pools[1].clone(), torch.zeros_like(a.X)
        a.call(X=X, kp=kp, vp=vp, Y=Y)
        assert kl.kl_device_status() == 0
        assert torch.isfinite(Y[:a.rows]).all()
        outs.append((Y[:a.rows], kp, vp))
    assert all(torch.equal(x, y) for x, y in zip(*outs))


def test_a_uniform_step_equals_the_paged_layer(kl):
    """A step that both layer forwards take: within the layer tests' bound of each other, as each is of the oracle."""
    B, n, H, Hq, Hkv, I, bs = 4, 3, 512, 8, 2, 768, 16
    a = Layer(kl, 6, [(n, c) for c in (0, 17, 300, 64)], B * n, H, Hq, Hkv, I, bs, True)
    kp, vp = torch.nan_to_num(a.kp), torch.nan_to_num(a.vp)
    k2, v2, Y2 = kp.clone(), vp.clone(), torch.zeros_like(a.X)
    a.call(kp=kp, vp=vp)
    cfg = L.make_cfg(B, n, H, Hq, Hkv, D, I, dtype=kl.KL_BF16, qk_norm=True)
    pc = kl.PagedCfg(B, n, bs, a.rc.max_blocks, a.rc.n_blocks)
    ws = torch.empty(kl.kl_layer_forward_paged_ws_bytes(cfg, pc), dtype=torch.uint8, device="cuda")
    td = a.td.clamp(max=a.rc.n_blocks - 1)
    kl.kl_layer_forward_paged(cfg, pc, L.weights_struct(a.w), a.X.data_ptr(), Y2.data_ptr(), k2.data_ptr(), v2.data_ptr(), td.data_ptr(), a.xd.data_ptr(), ws.data_ptr(), ws.numel())
    assert kl.kl_device_status() == 0
    assert_rel(_host(a.Y), _host(Y2), TOL_BF16, "Y")
    assert_rel(_host(kp), _host(k2), TOL_BF16, "k pool")
    assert torch.equal(vp, v2)


def test_a_captured_layer_serves_later_steps(kl):
    """The layer captured on a stream of its own and replayed after the lengths, rows and tables were changed on the device."""
    a = Layer(kl, 7, [(3, 40), (30, 0), (1, 200)], 40, 256, 4, 2, 512, 16, True)
    a.kp, a.vp = torch.nan_to_num(a.kp), torch.nan_to_num(a.vp)
    a.X.nan_to_num_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        a.call()
    for new in ([1, 1, 1], [0, 25, 8], [8, 0, 0], [3, 30, 1]):
        cu = np.concatenate([[0], np.cumsum(new)])
        pos = np.concatenate([np.arange(c, c + k) for k, c in zip(new, a.ctx)])
        req = np.repeat(np.arange(3), new)
        slots = a.table[req, pos // 16] * 16 + pos % 16
        a.cd.copy_(_i(cu))
        a.pd[:len(pos)] = _i(pos)
        a.sd[:len(pos)] = _i(slots)
        X = torch.randn(a.X.shape, device="cuda").bfloat16()
        kp, vp = a.kp.clone(), a.vp.clone()
        a.X.copy_(X)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        want = torch.zeros_like(a.X)
        a.call(X=X, kp=kp, vp=vp, Y=want)
        assert kl.kl_device_status() == 0
        rows = int(cu[-1])
        assert torch.equal(a.Y[:rows], want[:rows]) and torch.equal(a.kp, kp) and torch.equal(a.vp, vp)


# ---------------------------------------------------------------------------
# streams side by side
# ---------------------------------------------------------------------------

def test_plan_and_verify_on_two_streams_at_once(kl):
    """Two servers' plans and verifications in flight together: each gives what it gives alone."""
    g = torch.Generator(device="cuda").manual_seed(9)
    jobs = []
    for B, V, dt in ((64, 30000, torch.float32), (3, 50001, torch.bfloat16)):
        rng = np.random.default_rng(B)
        T, bs, maxb, nb = 5 * B, 16, 8, 8 * B
        p = torch.softmax(2 * torch.randn(T, V, generator=g, device="cuda"), 1).to(dt)
        q = torch.softmax(2 * torch.randn(T, V, generator=g, device="cuda"), 1).to(dt)
        jobs.append(dict(
            st=torch.cuda.Stream(), rc=kl.RaggedCfg(B, T, bs, maxb, nb), vc=kl.VerifyCfg(B, T, V, kl.KL_F32 if dt == torch.float32 else kl.KL_BF16), p=p, q=q, V=V,
            new=_i(np.full(B, 5)), ctx=_i(rng.integers(0, 60, B)), tok=torch.multinomial(q.float(), 1, generator=g)[:, 0].to(torch.int32),
            ua=torch.rand(T, generator=g, device="cuda"), us=torch.rand(B, generator=g, device="cuda"), free=_i(rng.permutation(nb)), B=B, T=T, maxb=maxb))

    def state(j):
        return [torch.full((j["B"], j["maxb"]), -1, dtype=torch.int32, device="cuda"), _i(np.zeros(j["B"])), j["free"].clone(), _i([len(j["free"])]),
                _i(np.zeros(j["B"] + 1)), _i(np.zeros(j["T"])), _i(np.zeros(j["T"])), _i([0]), _i(np.zeros(j["B"])), _i(np.zeros(j["B"]))]

    def call(j, t, st):
        kl.kl_ragged_plan(j["rc"], j["new"].data_ptr(), j["ctx"].data_ptr(), *[x.data_ptr() for x in t[:8]], st)
        kl.kl_draft_verify(j["vc"], j["p"].data_ptr(), j["V"], j["q"].data_ptr(), j["V"], j["tok"].data_ptr(), t[4].data_ptr(), j["ua"].data_ptr(), j["us"].data_ptr(),
                           t[8].data_ptr(), t[9].data_ptr(), st)

    alone = []
    for j in jobs:
        t = state(j)
        call(j, t, None)
        torch.cuda.synchronize()
        alone.append(t)
    rounds = [[state(j) for j in jobs] for _ in range(20)]
    torch.cuda.synchronize()
    for r in rounds:
        for j, t in zip(jobs, r):
            call(j, t, j["st"])
    assert kl.kl_device_status(jobs[0]["st"]) == 0 and kl.kl_device_status(jobs[1]["st"]) == 0
    for r in rounds:
        for t, want in zip(r, alone):
            assert all(torch.equal(x, y) for x, y in zip(t, want))
