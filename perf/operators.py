"""The operators of a ragged serving step: what is measured, their plain forms and their definitions.

  plan       block tables, positions and cache slots of a step from the requests' lengths
  qkv        per-head norm and rotation of the new queries and keys, keys and values into their cache slots
  attention  attention of each request's new tokens over its paged cache
  verify     drafted tokens accepted or replaced from the target's probabilities and given random numbers

Head counts, widths and the vocabulary are those of the benchmark's layer (64 query heads, 8 key/value heads of 128,
151936 classes, pages of 16 tokens) or the tests' smaller ones.
"""
import math
import random

import numpy as np
import torch

own = False

D = 128


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # the step of 64 decoding requests: the smallest call of a server's loop
        dict(name="plan_decode_64", op="plan", B=64, new_lo=1, new_hi=1, ctx_lo=3800, ctx_hi=4300, block=16, ended=0.0, short=False, lens=1),
        # a large admission step: 700 requests of very different lengths, some of them ended
        dict(name="plan_admit_700", op="plan", B=700, new_lo=1, new_hi=400, ctx_lo=0, ctx_hi=8000, block=16, ended=0.1, short=False, lens=2),
        # the new tokens of 64 decoding requests, without the per-head norm
        dict(name="qkv_decode_64", op="qkv", B=64, Hq=64, Hkv=8, new_lo=1, new_hi=1, ctx_lo=3800, ctx_hi=4300, block=16, norm=False, inter=False, lens=3),
        # prompts of odd lengths far into long contexts, with the norm
        dict(name="qkv_prompts_9000", op="qkv", B=9, Hq=64, Hkv=8, new_lo=700, new_hi=1300, ctx_lo=0, ctx_hi=100000, block=16, norm=True, inter=False, lens=4),
        # one request decoding at a long context: latency
        dict(name="attn_decode_1x32768", op="attention", B=1, Hq=64, Hkv=8, new_lo=1, new_hi=1, ctx_lo=32768, ctx_hi=32768, block=16, lens=5),
        # the benchmark's decode step, contexts around 4096
        dict(name="attn_decode_64x4096", op="attention", B=64, Hq=64, Hkv=8, new_lo=1, new_hi=1, ctx_lo=3600, ctx_hi=4600, block=16, lens=6),
        # four drafted tokens and the last one for 24 requests, pages of 32
        dict(name="attn_drafts_24x5", op="attention", B=24, Hq=64, Hkv=8, new_lo=5, new_hi=5, ctx_lo=500, ctx_hi=8000, block=32, lens=7),
        # decoding requests beside chunks of prompts, few heads, pages that end inside a key tile
        dict(name="attn_mixed_20", op="attention", B=20, Hq=16, Hkv=2, new_lo=1, new_hi=600, ctx_lo=0, ctx_hi=6000, block=24, lens=8),
        # a chunk of a long prompt over what is cached already: the tensor-core end
        dict(name="attn_chunk_4096_of_16384", op="attention", B=1, Hq=64, Hkv=8, new_lo=4095, new_hi=4095, ctx_lo=12288, ctx_hi=12288, block=16, lens=9),
        # one request's four drafted tokens: latency
        dict(name="verify_1x4", op="verify", B=1, k_lo=4, k_hi=4, V=151936, dtype="fp32", given_q=True, lens=10),
        # 64 requests
        dict(name="verify_64x4", op="verify", B=64, k_lo=4, k_hi=4, V=151936, dtype="fp32", given_q=True, lens=11),
        # drafts without probabilities of their own (a lookup), an odd vocabulary in 16 bits, some requests without drafts
        dict(name="verify_lookup_24", op="verify", B=24, k_lo=0, k_hi=7, V=32001, dtype="bf16", given_q=False, lens=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "qkv", "attention", "attention", "attention", "verify"])
    lens = rng.randrange(1 << 30)
    block = rng.choice([5, 8, 16, 16, 24, 32, 64, 128])
    heads = rng.choice([(64, 8), (64, 8), (8, 1), (4, 2), (16, 2), (12, 4), (64, 8), (8, 8)])
    if op == "plan":
        return dict(op=op, B=_log(rng, 1, 800), new_lo=rng.choice([0, 1]), new_hi=_log(rng, 1, 400), ctx_lo=0, ctx_hi=_log(rng, 16, 8000), block=block,
                    ended=rng.choice([0.0, 0.05, 0.3]), short=rng.choice([False, False, True]), lens=lens)
    if op == "qkv":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, Hq=heads[0], Hkv=heads[1], new_lo=1, new_hi=_log(rng, 1, max(1, 9000 // B)), ctx_lo=0, ctx_hi=_log(rng, 64, 100000), block=block,
                    norm=rng.choice([False, True]), inter=rng.choice([False, False, True]), lens=lens)
    if op == "verify":
        k = _log(rng, 1, 8)
        return dict(op=op, B=_log(rng, 1, 64), k_lo=rng.choice([0, k]), k_hi=k, V=_log(rng, 1000, 151936), dtype=rng.choice(["fp32", "bf16"]), given_q=rng.choice([True, True, False]), lens=lens)
    while True:
        B, n, ctx = _log(rng, 1, 96), rng.choice([1, 1, _log(rng, 2, 9), _log(rng, 10, 4096)]), _log(rng, 16, 32768)
        lo = 1 if rng.random() < 0.5 else n
        # the plain form holds the scores of the whole padded batch
        if B * heads[0] * n * (ctx + n) <= 4.0e9 and B * heads[1] * (ctx + n) <= 2.2e6:
            break
    return dict(op="attention", B=B, Hq=heads[0], Hkv=heads[1], new_lo=lo, new_hi=n, ctx_lo=0, ctx_hi=ctx, block=block, lens=lens)


def _lengths(case):
    """Each request's new tokens (-1: the request has ended) and cached tokens: part of the case, not of the seed."""
    r = random.Random(case["lens"])
    lo, hi = case["new_lo"], case["new_hi"]
    # a wide range holds single tokens beside chunks: even over the logarithm
    new = [_log(r, lo, hi) if lo >= 1 and hi >= 16 * lo else r.randint(lo, hi) for _ in range(case["B"])]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    if case.get("ended"):
        new = [-1 if r.random() < case["ended"] else n for n in new]
    return new, ctx


def _drafts(case):
    r = random.Random(case["lens"])
    return [r.randint(case["k_lo"], case["k_hi"]) for _ in range(case["B"])]


def _up(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------

def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(values):
    cu = [0]
    for v in values:
        cu.append(cu[-1] + max(0, v))
    return cu


class State:
    pass


def _pages(case, new, ctx, gen, pools):
    """A step's lengths, tables over a shuffled pool, and (with `pools`) pools that hold values in every slot."""
    s = State()
    s.case, s.B, s.block = case, case["B"], case["block"]
    s.max_blocks = max(1, max(_up(c + max(n, 0), s.block) for n, c in zip(new, ctx)))
    held = [_up(c + max(n, 0), s.block) for n, c in zip(new, ctx)]
    s.n_blocks = sum(held) + 7
    order = torch.randperm(s.n_blocks, generator=gen, device="cuda", dtype=torch.int32)
    lb = torch.arange(s.max_blocks, device="cuda")
    first = torch.tensor(_cu(held)[:-1], device="cuda")
    at = (first[:, None] + lb[None, :]).clamp(max=s.n_blocks - 1)
    s.table = order[at].where(lb[None, :] < torch.tensor(held, device="cuda")[:, None], -1).contiguous()
    s.new, s.ctx, s.cu = _int(new), _int(ctx), _int(_cu(new))
    s.T, s.longest, s.deepest = _cu(new)[-1], max(new), max(n + c for n, c in zip(new, ctx))
    if pools:
        shape = (s.n_blocks, s.block, case["Hkv"], D)
        s.k_pool = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
        s.v_pool = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "verify":
        return _prepare_verify(case, gen)
    new, ctx = _lengths(case)
    if op == "plan":
        return _prepare_plan(case, new, ctx, gen)
    s = _pages(case, new, ctx, gen, True)
    s.op = op
    Hq, Hkv = case["Hq"], case["Hkv"]
    rnd = lambda *shape: torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    if op == "qkv":
        s.q_pre, s.k_pre, s.v = rnd(s.T, Hq, D), rnd(s.T, Hkv, D), rnd(s.T, Hkv, D)
        s.gq = s.gk = None
        if case["norm"]:
            s.gq, s.gk = (1 + 0.1 * rnd(D)).to(torch.bfloat16), (1 + 0.1 * rnd(D)).to(torch.bfloat16)
        req = torch.repeat_interleave(torch.arange(s.B, device="cuda"), s.new.long())
        s.pos = (s.ctx[req] + torch.arange(s.T, device="cuda") - s.cu[req]).to(torch.int32)
        s.slots = (s.table[req, (s.pos // s.block).long()] * s.block + s.pos % s.block).to(torch.int32)
        s.q_out = torch.empty_like(s.q_pre)
    else:
        s.q = rnd(s.T, Hq, D)
        s.o = torch.empty_like(s.q)
        s.lse = torch.empty(s.T, Hq, device="cuda")
    if own:
        import bwd_qwen3_layer_gb300 as K
        s.cfg = K.RaggedCfg(s.B, s.T, s.block, s.max_blocks, s.n_blocks)
        if op == "attention":
            s.ws = torch.empty(max(256, K.kl_ragged_attention_ws_bytes(s.cfg, Hq, Hkv, D)), dtype=torch.uint8, device="cuda")
    return s


def _prepare_plan(case, new, ctx, gen):
    s = _pages(case, new, ctx, gen, False)
    s.op = "plan"
    # the requests hold the blocks of their cached tokens; the rest of the pool is the free list
    bs = s.block
    held = torch.tensor([_up(c, bs) for c in ctx], dtype=torch.int32, device="cuda")
    lb = torch.arange(s.max_blocks, device="cuda")
    mine = lb[None, :] < held[:, None]
    used = torch.zeros(s.n_blocks, dtype=torch.bool, device="cuda")
    used[s.table[mine].long()] = True
    free = torch.arange(s.n_blocks, device="cuda", dtype=torch.int32)[~used]
    free = free[torch.randperm(free.numel(), generator=gen, device="cuda")]
    n_free = free.numel() // 2 if case["short"] else free.numel()  # a pool that runs out, or one that does not
    # all that a step changes lies in one buffer, so that a pass starts from the same state
    parts = [s.table.where(mine, -1).reshape(-1), held, torch.cat([free, torch.full((s.n_blocks - free.numel(),), -1, dtype=torch.int32, device="cuda")]), _int([n_free])]
    s.start = torch.cat(parts)
    s.state = s.start.clone()
    s.table, s.held, s.free_list, s.n_free = s.state.split([p.numel() for p in parts])
    s.table = s.table.view(s.B, s.max_blocks)
    s.cu_out = torch.empty(s.B + 1, dtype=torch.int32, device="cuda")
    s.pos, s.slots = torch.empty(max(1, s.T), dtype=torch.int32, device="cuda"), torch.empty(max(1, s.T), dtype=torch.int32, device="cuda")
    s.pos.zero_(), s.slots.zero_()
    s.missing = torch.empty(1, dtype=torch.int32, device="cuda")
    if own:
        import bwd_qwen3_layer_gb300 as K
        s.cfg = K.RaggedCfg(s.B, max(1, s.T), s.block, s.max_blocks, s.n_blocks)
    return s


def _prepare_verify(case, gen):
    s = State()
    s.op, s.case, s.B, s.V = "verify", case, case["B"], case["V"]
    k = _drafts(case)
    cu = _cu([n + 1 for n in k])
    s.T, s.cu, s.given_q = cu[-1], _int(cu), case["given_q"]
    dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    z = torch.randn(s.T, s.V, generator=gen, device="cuda") * 2.5
    s.p = torch.softmax(z, 1).to(dt)
    zq = z + 0.7 * torch.randn(s.T, s.V, generator=gen, device="cuda")
    s.q = torch.softmax(zq, 1).to(dt) if s.given_q else None
    # each row's draft is drawn from the row's draft probabilities; it is the token that the next row was fed
    pick = (zq - torch.log(-torch.log(torch.rand(s.T, s.V, generator=gen, device="cuda").clamp(1e-7, 1 - 1e-7)))).argmax(1)
    s.tokens = torch.cat([torch.randint(0, s.V, (1,), generator=gen, device="cuda"), pick[:-1]]).to(torch.int32)
    s.u_accept = torch.rand(s.T, generator=gen, device="cuda")
    s.u_sample = torch.rand(s.B, generator=gen, device="cuda")
    s.accepted = torch.empty(s.B, dtype=torch.int32, device="cuda")
    s.token = torch.empty(s.B, dtype=torch.int32, device="cuda")
    if own:
        import bwd_qwen3_layer_gb300 as K
        s.cfg = K.VerifyCfg(s.B, s.T, s.V, K.KL_F32 if dt == torch.float32 else K.KL_BF16)
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------

def run(s):
    if own:
        return OWN[s.op](s)
    return PLAIN[s.op](s)


def _own_plan(s):
    import bwd_qwen3_layer_gb300 as K
    s.state.copy_(s.start)
    K.kl_ragged_plan(s.cfg, s.new.data_ptr(), s.ctx.data_ptr(), s.table.data_ptr(), s.held.data_ptr(), s.free_list.data_ptr(), s.n_free.data_ptr(), s.cu_out.data_ptr(),
                     s.pos.data_ptr(), s.slots.data_ptr(), s.missing.data_ptr())
    return s.cu_out, s.pos, s.slots, s.table, s.held, s.free_list, s.n_free, s.missing


def _own_qkv(s):
    import bwd_qwen3_layer_gb300 as K
    c = s.case
    K.kl_ragged_qkv_rope(s.cfg, c["Hq"], c["Hkv"], D, K.KL_BF16, s.q_pre.data_ptr(), s.k_pre.data_ptr(), s.v.data_ptr(), K.ptr(s.gq), K.ptr(s.gk), 1e-6, 1e6, int(c["inter"]),
                         s.cu.data_ptr(), s.pos.data_ptr(), s.slots.data_ptr(), s.q_out.data_ptr(), s.k_pool.data_ptr(), s.v_pool.data_ptr())
    return s.q_out, s.k_pool, s.v_pool


def _own_attention(s):
    import bwd_qwen3_layer_gb300 as K
    c = s.case
    K.kl_ragged_attention(s.cfg, c["Hq"], c["Hkv"], D, K.KL_BF16, s.q.data_ptr(), s.k_pool.data_ptr(), s.v_pool.data_ptr(), s.table.data_ptr(), s.cu.data_ptr(), s.ctx.data_ptr(),
                          s.o.data_ptr(), s.lse.data_ptr(), s.ws.data_ptr(), s.ws.numel())
    return s.o, s.lse


def _own_verify(s):
    import bwd_qwen3_layer_gb300 as K
    K.kl_draft_verify(s.cfg, s.p.data_ptr(), s.V, K.ptr(s.q), s.V, s.tokens.data_ptr(), s.cu.data_ptr(), s.u_accept.data_ptr(), s.u_sample.data_ptr(), s.accepted.data_ptr(),
                      s.token.data_ptr())
    return s.accepted, s.token


def _plain_plan(s):
    s.state.copy_(s.start)
    bs, n_free = s.block, s.n_free.long()
    n = s.new.clamp(min=0).long()
    ctx, held = s.ctx.long(), s.held.long()
    want = torch.where(n > 0, (ctx + n + bs - 1) // bs, 0).clamp(max=s.max_blocks)
    take = (want - held).clamp(min=0)
    upto = take.cumsum(0)
    granted = upto <= n_free
    lb = torch.arange(s.max_blocks, device=held.device)[None, :]
    fresh = (lb >= held[:, None]) & (lb < want[:, None])
    k = (upto - take)[:, None] + lb - held[:, None]
    block = s.free_list[(n_free - 1 - k).clamp(0, s.n_blocks - 1)]
    table = torch.where(fresh, torch.where(granted[:, None], block, -1), s.table)
    left = n_free - torch.where(granted, take, 0).sum()
    # ended requests give their blocks back, in order
    ended = s.new < 0
    back = torch.where(ended, held, 0)
    at = left + (back.cumsum(0) - back)[:, None] + lb
    at = torch.where(ended[:, None] & (lb < held[:, None]), at, s.n_blocks)
    free = torch.cat([s.free_list, s.free_list[:1]]).scatter(0, at.reshape(-1), s.table.reshape(-1))[:-1]
    now_held = torch.where(ended, 0, torch.where(granted, torch.maximum(held, want), held))
    cu = torch.cat([n.new_zeros(1), n.cumsum(0)])
    r = torch.arange(s.pos.numel(), device=held.device)
    b = torch.searchsorted(cu[1:], r, right=True).clamp(max=s.B - 1)
    pos = ctx[b] + r - cu[b]
    page = pos // bs
    entry = table[b, page.clamp(max=s.max_blocks - 1)].long()
    slot = torch.where((page < now_held[b]) & (entry >= 0), entry * bs + pos % bs, -1)
    inside = r < cu[-1]
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return (i32(cu), i32(torch.where(inside, pos, s.pos)), i32(torch.where(inside, slot, s.slots)), table, i32(now_held), free, i32(left + back.sum()).view(1),
            i32(torch.where(granted, 0, take).sum()).view(1))


def _plain_qkv(s):
    c = s.case
    i = torch.arange(D // 2, device="cuda", dtype=torch.float64)
    angle = s.pos.double()[:, None] * (1e6 ** (-2.0 * i / D))[None, :]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]

    def turned(x, gain):
        x = x.float()
        if gain is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gain.float()
        if c["inter"]:
            a, b = x[..., 0::2], x[..., 1::2]
            return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).reshape(x.shape).to(torch.bfloat16)
        a, b = x[..., : D // 2], x[..., D // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1).to(torch.bfloat16)

    slots = s.slots.long()
    s.k_pool.view(-1, c["Hkv"], D)[slots] = turned(s.k_pre, s.gk)
    s.v_pool.view(-1, c["Hkv"], D)[slots] = s.v
    return turned(s.q_pre, s.gq), s.k_pool, s.v_pool


def _plain_attention(s):
    c = s.case
    Hq, Hkv = c["Hq"], c["Hkv"]
    G, B, n, L = Hq // Hkv, s.B, s.longest, s.deepest
    cu, ctx, new = s.cu.long(), s.ctx.long(), s.new.long()
    i, j = torch.arange(n, device="cuda"), torch.arange(L, device="cuda")
    blocks = s.table[:, : _up(L, s.block)].long().clamp(min=0)
    inside = (j[None, :] < (ctx + new)[:, None])[:, :, None, None]

    def cached(pool):
        x = pool[blocks].view(B, -1, Hkv, D)[:, :L].float()
        return torch.where(inside, x, 0.0).permute(0, 2, 1, 3)

    rows = (cu[:-1, None] + i[None, :]).clamp(max=s.T - 1)
    q = s.q[rows].float().view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    score = torch.matmul(q, cached(s.k_pool).transpose(2, 3)).mul_(1.0 / math.sqrt(D)).view(B, Hkv, G, n, L)
    hidden = j[None, None, :] > (ctx[:, None] + i[None, :])[:, :, None]
    score.masked_fill_(hidden[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score.view(B, Hkv, G * n, L), cached(s.v_pool)).view(B, Hkv, G, n, D) / total
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, n, Hq)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    # back to the rows of the step
    r = torch.arange(s.T, device="cuda")
    b = torch.searchsorted(cu[1:], r, right=True)
    return o[b, r - cu[b]].to(torch.bfloat16), lse[b, r - cu[b]]


def _plain_verify(s):
    cu = s.cu.long()
    first, last = cu[:-1], cu[1:] - 1
    r = torch.arange(s.T, device="cuda")
    b = torch.searchsorted(cu[1:], r, right=True)
    fed = torch.cat([s.tokens[1:], s.tokens[:1]]).long()  # the draft that row r judges
    p = s.p.gather(1, fed[:, None])[:, 0].double()
    q = s.q.gather(1, fed[:, None])[:, 0].double() if s.given_q else torch.ones_like(p)
    ok = (s.u_accept.double() * q < p) & (r < last[b])
    stop = torch.where(ok, s.T, r)  # a request's first row that is not accepted: its last one at the latest
    row = torch.full((s.B,), s.T, device="cuda").scatter_reduce(0, b, stop, "amin")
    accepted = row - first
    drafted = row < last
    weight = s.p[row].double()
    if s.given_q:
        taken = s.q[row].double()
    else:
        taken = torch.zeros_like(weight).scatter_(1, fed[row][:, None], math.inf)
    rest = (weight - taken).clamp(min=0)
    use = (drafted & (rest.sum(1) > 0))[:, None]
    c = torch.where(use, rest, weight).cumsum(1)
    x = s.u_sample.double()[:, None] * c[:, -1:]
    token = torch.searchsorted(c, x, right=True)[:, 0].clamp(max=s.V - 1)
    return accepted.to(torch.int32), token.to(torch.int32)


OWN = {"plan": _own_plan, "qkv": _own_qkv, "attention": _own_attention, "verify": _own_verify}
PLAIN = {"plan": _plain_plan, "qkv": _plain_qkv, "attention": _plain_attention, "verify": _plain_verify}


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "verify":
        # one row of target (and draft) probabilities for each request, and the drafts' own entries
        size, rows = (4 if case["dtype"] == "fp32" else 2), sum(n + 1 for n in _drafts(case))
        return {"bytes": case["B"] * case["V"] * size * (2 if case["given_q"] else 1) + rows * 16 + case["B"] * 16, "flops": 2 * case["B"] * case["V"]}
    new, ctx = _lengths(case)
    T, bs = sum(max(n, 0) for n in new), case["block"]
    if op == "plan":
        # lengths, counts and the list's head; a table entry read or written for each block of the step; position and slot of each row
        touched = sum(_up(c + n, bs) - c // bs if n > 0 else _up(c, bs) if n < 0 else 0 for n, c in zip(new, ctx))
        return {"bytes": case["B"] * 20 + touched * 8 + T * 8, "flops": 0}
    Hq, Hkv = case["Hq"], case["Hkv"]
    if op == "qkv":
        return {"bytes": 2 * T * (Hq + 2 * Hkv) * D * 2 + T * 8, "flops": 10 * T * (Hq + Hkv) * D}
    pairs = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, ctx))
    cached = sum(n + c for n, c in zip(new, ctx))
    return {"bytes": 2 * cached * Hkv * D * 2 + 2 * T * Hq * D * 2 + T * Hq * 4, "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return EXACT[s.op](s)


def _exact_plan(s):
    bs, start = s.block, s.start.cpu().tolist()
    table = [start[b * s.max_blocks:(b + 1) * s.max_blocks] for b in range(s.B)]
    at = s.B * s.max_blocks
    held, free, n_free = start[at:at + s.B], start[at + s.B:-1], start[-1]
    new, ctx = s.new.tolist(), s.ctx.tolist()
    cu, pos, slots, missing, taken, short = [0], [], [], 0, 0, False
    for b in range(s.B):
        n = max(0, new[b])
        want = min(_up(ctx[b] + n, bs), s.max_blocks) if n else 0
        more = max(0, want - held[b])
        if more and (short or taken + more > n_free):
            short, missing = True, missing + more
            table[b][held[b]:want] = [-1] * more
        else:
            for _ in range(more):
                table[b][held[b]] = free[n_free - 1 - taken]
                held[b], taken = held[b] + 1, taken + 1
        for p in range(ctx[b], ctx[b] + n):
            pos.append(p)
            slots.append(table[b][p // bs] * bs + p % bs if p // bs < held[b] and table[b][p // bs] >= 0 else -1)
        cu.append(cu[-1] + n)
    n_free -= taken
    for b in range(s.B):
        if new[b] < 0:
            free[n_free:n_free + held[b]] = table[b][:held[b]]
            n_free, held[b] = n_free + held[b], 0
    pos, slots = pos or [0], slots or [0]
    return [np.array(v, np.int32) for v in (cu, pos, slots, table, held, free, [n_free], [missing])]


def _exact_qkv(s):
    c = s.case
    rate = 1e6 ** (-2.0 * np.arange(D // 2) / D)
    angle = s.pos.cpu().numpy().astype(np.float64)[:, None] * rate
    turn = np.exp(1j * angle)[:, None, :]

    def turned(x, gain):
        x = x.double().cpu().numpy()
        if gain is not None:
            x = gain.double().cpu().numpy() * x / np.sqrt(np.mean(x * x, -1, keepdims=True) + 1e-6)
        y = np.empty_like(x)
        even, odd = (np.s_[..., 0::2], np.s_[..., 1::2]) if c["inter"] else (np.s_[..., : D // 2], np.s_[..., D // 2:])
        z = (x[even] + 1j * x[odd]) * turn
        y[even], y[odd] = z.real, z.imag
        return y

    k, v = s.k_pool.double().cpu().numpy().reshape(-1, c["Hkv"], D), s.v_pool.double().cpu().numpy().reshape(-1, c["Hkv"], D)
    slots = s.slots.cpu().numpy()
    k[slots], v[slots] = turned(s.k_pre, s.gk), s.v.double().cpu().numpy()
    shape = tuple(s.k_pool.shape)
    return turned(s.q_pre, s.gq), k.reshape(shape), v.reshape(shape)


def _exact_attention(s):
    c = s.case
    Hq, Hkv = c["Hq"], c["Hkv"]
    G = Hq // Hkv
    new, ctx, cu = s.new.tolist(), s.ctx.tolist(), s.cu.tolist()
    o, lse = torch.zeros(s.T, Hq, D, dtype=torch.float64, device="cuda"), torch.zeros(s.T, Hq, dtype=torch.float64, device="cuda")
    for b in range(s.B):
        L = ctx[b] + new[b]
        page = s.table[b, : _up(L, s.block)].long()
        keys, values = s.k_pool[page].reshape(-1, Hkv, D)[:L], s.v_pool[page].reshape(-1, Hkv, D)[:L]
        rows = slice(cu[b], cu[b + 1])
        seen = torch.arange(L, device="cuda")[None, :] <= ctx[b] + torch.arange(new[b], device="cuda")[:, None]
        for h in range(Hq):
            z = s.q[rows, h].double() @ keys[:, h // G].double().T / math.sqrt(D)
            z = torch.where(seen, z, -math.inf)
            lse[rows, h] = torch.logsumexp(z, 1)
            o[rows, h] = torch.exp(z - lse[rows, h, None]) @ values[:, h // G].double()
    return o, lse


def _exact_verify(s):
    cu, tokens = s.cu.tolist(), s.tokens.tolist()
    ua, us = s.u_accept.double().cpu().numpy(), s.u_sample.double().cpu().numpy()
    accepted, token = [], []
    for b in range(s.B):
        row, last = cu[b], cu[b + 1] - 1
        while row < last and ua[row] * (float(s.q[row, tokens[row + 1]]) if s.given_q else 1.0) < float(s.p[row, tokens[row + 1]]):
            row += 1
        w = s.p[row].double().cpu().numpy()
        if row < last:
            if s.given_q:
                rest = np.maximum(0.0, w - s.q[row].double().cpu().numpy())
            else:
                rest = w.copy()
                rest[tokens[row + 1]] = 0.0
            w = rest if rest.sum() > 0 else w
        c = np.cumsum(w)
        token.append(min(int(np.searchsorted(c, us[b] * c[-1], side="right")), s.V - 1))
        accepted.append(row - cu[b])
    return np.array(accepted, np.int32), np.array(token, np.int32)


EXACT = {"plan": _exact_plan, "qkv": _exact_qkv, "attention": _exact_attention, "verify": _exact_verify}
