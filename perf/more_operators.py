"""Operators of generating over a cache held in 8 bits and of training on what was generated: what is measured, their plain
forms and their definitions.

  append     per-head norm and rotation of a ragged step's new queries and keys; keys and values into 8-bit pages with a
             scale for each page and head
  attention  attention of each request's new tokens over its 8-bit pages
  logprobs   log probabilities of given tokens, the entropy of each row and its most likely alternatives
  grad       the gradient of those log probabilities and entropies

Head counts, widths and the vocabulary are those of the benchmark's layer (64 query heads, 8 key/value heads of 128,
151936 classes, pages of 16 tokens) or the tests' smaller ones.
"""
import math
import random

import torch

own = False

D = 128
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # the new tokens of 64 decoding requests: one slot of a page that is part full, for most
        dict(name="append_decode_64", op="append", B=64, Hq=64, Hkv=8, new_lo=1, new_hi=1, ctx_lo=900, ctx_hi=1300, block=16, norm=True, inter=False, lens=3),
        # prompts of odd lengths behind contexts of any length
        dict(name="append_prompts_9000", op="append", B=9, Hq=64, Hkv=8, new_lo=700, new_hi=1300, ctx_lo=0, ctx_hi=20000, block=16, norm=True, inter=False, lens=4),
        # one request decoding at a long context: latency
        dict(name="attn_decode_1x32768", op="attention", B=1, Hq=64, Hkv=8, new_lo=1, new_hi=1, ctx_lo=32768, ctx_hi=32768, block=16, lens=5),
        # the benchmark's decode step, contexts around 4096
        dict(name="attn_decode_64x4096", op="attention", B=64, Hq=64, Hkv=8, new_lo=1, new_hi=1, ctx_lo=3600, ctx_hi=4600, block=16, lens=6),
        # decoding requests beside chunks of prompts, few heads, pages that end inside a key tile
        dict(name="attn_mixed_20", op="attention", B=20, Hq=16, Hkv=2, new_lo=1, new_hi=600, ctx_lo=0, ctx_hi=6000, block=24, lens=8),
        # a chunk of a long prompt over what is cached already: the tensor-core end
        dict(name="attn_chunk_4096_of_16384", op="attention", B=1, Hq=64, Hkv=8, new_lo=4095, new_hi=4095, ctx_lo=12288, ctx_hi=12288, block=16, lens=9),
        # one request's token with five alternatives: latency
        dict(name="logprobs_1", op="logprobs", N=1, V=151936, dtype="bf16", top=5, masked=False),
        # a decoding step's tokens with twenty alternatives each
        dict(name="logprobs_64", op="logprobs", N=64, V=151936, dtype="fp32", top=20, masked=False),
        # rows that a grammar's mask leaves few classes of (a row none), an odd vocabulary
        dict(name="logprobs_masked_301", op="logprobs", N=301, V=32001, dtype="fp32", top=8, masked=True),
        # the tokens of whole prompts scored: no alternatives
        dict(name="logprobs_prompt_2045", op="logprobs", N=2045, V=151936, dtype="bf16", top=0, masked=False),
        # a policy gradient with an entropy bonus, masked rows, an odd vocabulary
        dict(name="grad_masked_257", op="grad", N=257, V=32001, dtype="fp32", masked=True),
        # the same over whole answers
        dict(name="grad_1021", op="grad", N=1021, V=151936, dtype="bf16", masked=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "attention", "logprobs", "logprobs", "grad"])
    lens = rng.randrange(1 << 30)
    block = rng.choice([5, 8, 16, 16, 24, 32, 64, 128])
    heads = rng.choice([(64, 8), (64, 8), (8, 1), (4, 2), (16, 2), (12, 4), (64, 8), (8, 8)])
    if op == "append":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, Hq=heads[0], Hkv=heads[1], new_lo=1, new_hi=_log(rng, 1, max(1, 9000 // B)), ctx_lo=0, ctx_hi=_log(rng, 64, 80000 // B), block=block,
                    norm=rng.choice([False, True]), inter=rng.choice([False, False, True]), lens=lens)
    if op in ("logprobs", "grad"):
        while True:
            N, V = _log(rng, 1, 2045 if op == "logprobs" else 1021), _log(rng, 1000, 151936)
            dtype = rng.choice(["fp32", "bf16"])
            if N * V * (4 if dtype == "fp32" else 2) <= 6.2e8:
                break
        case = dict(op=op, N=N, V=V, dtype=dtype, masked=rng.choice([False, False, True]))
        if op == "logprobs":
            case["top"] = rng.choice([0, 1, 2, 5, 8, 20, 32])
        return case
    while True:
        B, n, ctx = _log(rng, 1, 96), rng.choice([1, 1, _log(rng, 2, 9), _log(rng, 10, 4096)]), _log(rng, 16, 32768)
        lo = 1 if rng.random() < 0.5 else n
        # the plain form holds the scores of the whole padded batch
        if B * heads[0] * n * (ctx + n) <= 3.5e9 and B * heads[1] * (ctx + n) <= 2.2e6:
            break
    return dict(op="attention", B=B, Hq=heads[0], Hkv=heads[1], new_lo=lo, new_hi=n, ctx_lo=0, ctx_hi=ctx, block=block, lens=lens)


def _lengths(case):
    """Each request's new tokens and cached tokens: part of the case, not of the seed."""
    r = random.Random(case["lens"])
    lo, hi = case["new_lo"], case["new_hi"]
    # a wide range holds single tokens beside chunks: even over the logarithm
    new = [_log(r, lo, hi) if hi >= 16 * lo else r.randint(lo, hi) for _ in range(case["B"])]
    return new, [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]


def _up(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------

class State:
    pass


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(values):
    cu = [0]
    for v in values:
        cu.append(cu[-1] + v)
    return cu


def _pool(shape, gen):
    """Codes and scales of pages that hold values in every slot: heads of different sizes, the scale the least power of two
    that brings a page's largest value to 448 or below."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn(shape[2], 1, generator=gen, device="cuda"))
    scale = _scale(x.abs().amax((1, 3)))
    return (x / scale[:, None, :, None]).to(E4M3), scale


def _scale(largest):
    m, e = torch.frexp(largest)
    return torch.ldexp(torch.ones_like(largest), torch.where(m <= 0.875, e - 9, e - 8).where(m > 0, -64).clamp(min=-64))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = State()
    s.op, s.case = case["op"], case
    rnd = lambda *shape: torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    if s.op in ("logprobs", "grad"):
        _prepare_logits(s, case, gen)
        return s
    new, ctx = _lengths(case)
    Hq, Hkv = case["Hq"], case["Hkv"]
    s.B, s.block = case["B"], case["block"]
    held = [_up(c + n, s.block) for n, c in zip(new, ctx)]
    s.max_blocks, s.n_blocks = max(held), sum(held) + 7
    order = torch.randperm(s.n_blocks, generator=gen, device="cuda", dtype=torch.int32)
    lb = torch.arange(s.max_blocks, device="cuda")
    at = (torch.tensor(_cu(held)[:-1], device="cuda")[:, None] + lb[None, :]).clamp(max=s.n_blocks - 1)
    s.table = order[at].where(lb[None, :] < torch.tensor(held, device="cuda")[:, None], -1).contiguous()
    s.new, s.ctx, s.cu = _int(new), _int(ctx), _int(_cu(new))
    s.T, s.longest, s.deepest = _cu(new)[-1], max(new), max(n + c for n, c in zip(new, ctx))
    shape = (s.n_blocks, s.block, Hkv, D)
    s.k_pool, s.k_scale = _pool(shape, gen)
    s.v_pool, s.v_scale = _pool(shape, gen)
    if s.op == "append":
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
        if s.op == "attention":
            s.ws = torch.empty(max(256, K.kl_ragged_attention8_ws_bytes(s.cfg, Hq, Hkv, D)), dtype=torch.uint8, device="cuda")
    return s


def _prepare_logits(s, case, gen):
    s.N, s.V = case["N"], case["V"]
    dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    z = torch.randn(s.N, s.V, generator=gen, device="cuda") * 2.5
    if case["masked"]:
        # each row keeps its own share of the classes, from nearly all to a handful; the last one keeps none
        keep = 10 ** (-4 * torch.rand(s.N, 1, generator=gen, device="cuda"))
        keep[-1] = 0.0 if s.N > 1 else 0.5
        z.masked_fill_(torch.rand(s.N, s.V, generator=gen, device="cuda") >= keep, -math.inf)
    s.z = z.to(dt)
    # tokens drawn from the rows' own distributions; some rows (padding) have none
    pick = (z - torch.log(-torch.log(torch.rand(s.N, s.V, generator=gen, device="cuda").clamp(1e-7, 1 - 1e-7)))).argmax(1)
    s.tokens = torch.where(torch.arange(s.N, device="cuda") % 13 == 12, -1, pick).to(torch.int32)
    s.logprob, s.entropy, s.norm = (torch.empty(shape, device="cuda") for shape in ((s.N,), (s.N,), (s.N, 2)))
    if s.op == "logprobs":
        s.top_id = torch.empty(s.N, case["top"], dtype=torch.int32, device="cuda")
        s.top_logprob = torch.empty(s.N, case["top"], device="cuda")
        return
    # what a forward pass has left: each row's largest logit, the logarithm of the sum against it, the entropy
    _, s.entropy, s.norm, _, _ = _plain_rows(s, 0)
    s.d_logprob = torch.randn(s.N, generator=gen, device="cuda") / s.N
    s.d_entropy = 0.01 * torch.rand(s.N, generator=gen, device="cuda") / s.N
    s.dz = torch.empty_like(s.z)


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------

def run(s):
    if own:
        return OWN[s.op](s)
    return PLAIN[s.op](s)


def _own_append(s):
    import bwd_qwen3_layer_gb300 as K
    c = s.case
    K.kl_ragged_qkv_rope8(s.cfg, c["Hq"], c["Hkv"], D, K.KL_BF16, s.q_pre.data_ptr(), s.k_pre.data_ptr(), s.v.data_ptr(), K.ptr(s.gq), K.ptr(s.gk), 1e-6, 1e6, int(c["inter"]),
                          s.cu.data_ptr(), s.pos.data_ptr(), s.slots.data_ptr(), s.q_out.data_ptr(), s.k_pool.data_ptr(), s.v_pool.data_ptr(), s.k_scale.data_ptr(),
                          s.v_scale.data_ptr())
    return s.q_out, s.k_pool, s.v_pool, s.k_scale, s.v_scale


def _own_attention(s):
    import bwd_qwen3_layer_gb300 as K
    c = s.case
    K.kl_ragged_attention8(s.cfg, c["Hq"], c["Hkv"], D, K.KL_BF16, s.q.data_ptr(), s.k_pool.data_ptr(), s.v_pool.data_ptr(), s.k_scale.data_ptr(), s.v_scale.data_ptr(),
                           s.table.data_ptr(), s.cu.data_ptr(), s.ctx.data_ptr(), s.o.data_ptr(), s.lse.data_ptr(), s.ws.data_ptr(), s.ws.numel())
    return s.o, s.lse


def _own_logprobs(s):
    import bwd_qwen3_layer_gb300 as K
    K.kl_token_logprobs(s.N, s.V, K.KL_F32 if s.z.dtype == torch.float32 else K.KL_BF16, s.z.data_ptr(), s.V, s.tokens.data_ptr(), s.case["top"], s.logprob.data_ptr(),
                        s.entropy.data_ptr(), s.norm.data_ptr(), s.top_id.data_ptr(), s.top_logprob.data_ptr())
    return s.logprob, s.entropy, s.norm, s.top_id, s.top_logprob


def _own_grad(s):
    import bwd_qwen3_layer_gb300 as K
    dt = K.KL_F32 if s.z.dtype == torch.float32 else K.KL_BF16
    K.kl_token_logprobs_bwd(s.N, s.V, dt, s.z.data_ptr(), s.V, s.tokens.data_ptr(), s.norm.data_ptr(), s.entropy.data_ptr(), s.d_logprob.data_ptr(), s.d_entropy.data_ptr(), dt,
                            s.dz.data_ptr(), s.V)
    return s.dz


def _plain_append(s):
    c, bs = s.case, s.block
    i = torch.arange(D // 2, device="cuda", dtype=torch.float64)
    angle = s.pos.double()[:, None] * (1e6 ** (-2.0 * i / D))[None, :]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]

    def turned(x, gain):
        x = x.float()
        if gain is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gain.float()
        if c["inter"]:
            a, b = x[..., 0::2], x[..., 1::2]
            return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).reshape(x.shape)
        a, b = x[..., : D // 2], x[..., D // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)

    slots = s.slots.long()
    page, place = slots // bs, slots % bs
    # the first slot that this step writes of each page: what lies before it stays
    begin = torch.full((s.n_blocks,), bs, device="cuda").scatter_reduce(0, page, place, "amin")
    touched = torch.zeros(s.n_blocks, dtype=torch.bool, device="cuda").index_fill(0, page, True).nonzero()[:, 0]
    kept = torch.arange(bs, device="cuda")[None, :] < begin[touched, None]

    def append(x, pool, scale):
        largest = torch.zeros_like(scale).scatter_reduce(0, page[:, None].expand(-1, c["Hkv"]), x.abs().amax(-1), "amax")
        before = torch.where(begin[touched, None] > 0, scale[touched], 0.0)
        after = torch.maximum(before, _scale(largest[touched]))
        old = pool[touched]
        again = (old.float() * (before / after)[:, None, :, None]).to(E4M3)
        pool[touched] = torch.where((kept[:, :, None] & (after > before)[:, None, :])[..., None], again.view(torch.uint8), old.view(torch.uint8)).view(E4M3)
        scale[touched] = after
        pool.view(-1, c["Hkv"], D)[slots] = (x / scale[page][..., None]).to(E4M3)

    append(turned(s.k_pre, s.gk), s.k_pool, s.k_scale)
    append(s.v.float(), s.v_pool, s.v_scale)
    return turned(s.q_pre, s.gq).to(torch.bfloat16), s.k_pool, s.v_pool, s.k_scale, s.v_scale


def _plain_attention(s):
    c = s.case
    Hq, Hkv = c["Hq"], c["Hkv"]
    G, B, n, L = Hq // Hkv, s.B, s.longest, s.deepest
    cu, ctx, new = s.cu.long(), s.ctx.long(), s.new.long()
    i, j = torch.arange(n, device="cuda"), torch.arange(L, device="cuda")
    blocks = s.table[:, : _up(L, s.block)].long().clamp(min=0)
    inside = (j[None, :] < (ctx + new)[:, None])[:, :, None, None]

    def cached(pool, scale):
        x = (pool[blocks].float() * scale[blocks][:, :, None, :, None]).view(B, -1, Hkv, D)[:, :L]
        return torch.where(inside, x, 0.0).permute(0, 2, 1, 3)

    rows = (cu[:-1, None] + i[None, :]).clamp(max=s.T - 1)
    q = s.q[rows].float().view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    score = torch.matmul(q, cached(s.k_pool, s.k_scale).transpose(2, 3)).mul_(1.0 / math.sqrt(D)).view(B, Hkv, G, n, L)
    hidden = j[None, None, :] > (ctx[:, None] + i[None, :])[:, :, None]
    score.masked_fill_(hidden[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score.view(B, Hkv, G * n, L), cached(s.v_pool, s.v_scale)).view(B, Hkv, G, n, D) / total
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, n, Hq)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    # back to the rows of the step
    r = torch.arange(s.T, device="cuda")
    b = torch.searchsorted(cu[1:], r, right=True)
    return o[b, r - cu[b]].to(torch.bfloat16), lse[b, r - cu[b]]


def _plain_rows(s, top):
    z = s.z.float()
    largest = z.amax(1)
    some = largest > -math.inf
    x = z - torch.where(some, largest, 0.0)[:, None]
    e = x.exp()
    total = e.sum(1)
    log = total.log()
    entropy = torch.where(some, log - torch.where(e > 0, e * x, 0.0).sum(1) / total, 0.0)
    at = x.gather(1, s.tokens.clamp(min=0).long()[:, None])[:, 0] - torch.where(some, log, 0.0)
    logprob = torch.where(s.tokens < 0, 0.0, at)
    ids = values = None
    if top:
        # the values in the order of whole numbers, the index below them: ties go to the lowest one
        bits = z.view(torch.int32).long()
        order = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF))
        places = torch.arange(s.V, device="cuda")[None, :]
        ids = s.V - 1 - ((order * (1 << 31) + (s.V - 1 - places)).topk(top, 1).values % (1 << 31))
        values = x.gather(1, ids) - torch.where(some, log, 0.0)[:, None]
        ids = torch.where(values > -math.inf, ids, -1).to(torch.int32)
    return logprob, entropy, torch.stack([largest, log], 1), ids, values


def _plain_logprobs(s):
    logprob, entropy, norm, ids, values = _plain_rows(s, s.case["top"])
    return logprob, entropy, norm, s.top_id if ids is None else ids, s.top_logprob if values is None else values


def _plain_grad(s):
    some = s.norm[:, :1] > -math.inf
    x = s.z.float() - torch.where(some, s.norm.sum(1, keepdim=True), 0.0)
    p = x.exp()
    has = (s.tokens >= 0) & some[:, 0]
    g = torch.where(has, s.d_logprob, 0.0)[:, None]
    dz = -p * (g + s.d_entropy[:, None] * torch.where(p > 0, x + s.entropy[:, None], 0.0))
    return dz.scatter_add(1, s.tokens.clamp(min=0).long()[:, None], g).to(s.z.dtype)


OWN = {"append": _own_append, "attention": _own_attention, "logprobs": _own_logprobs, "grad": _own_grad}
PLAIN = {"append": _plain_append, "attention": _plain_attention, "logprobs": _plain_logprobs, "grad": _plain_grad}


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("logprobs", "grad"):
        n, size = case["N"] * case["V"], 4 if case["dtype"] == "fp32" else 2
        if op == "logprobs":
            return {"bytes": n * size + case["N"] * (20 + 8 * case["top"]), "flops": 4 * n}
        return {"bytes": 2 * n * size + case["N"] * 24, "flops": 6 * n}
    new, ctx = _lengths(case)
    T, bs, Hq, Hkv = sum(new), case["block"], case["Hq"], case["Hkv"]
    if op == "append":
        pages = sum(_up(c + n, bs) - c // bs for n, c in zip(new, ctx))
        return {"bytes": T * (4 * Hq + 2 * (2 + 1) * Hkv) * D + T * 8 + 2 * 8 * pages * Hkv, "flops": 10 * T * (Hq + Hkv) * D + 2 * T * Hkv * D}
    pairs = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, ctx))
    cached, pages = sum(n + c for n, c in zip(new, ctx)), sum(_up(c + n, bs) for n, c in zip(new, ctx))
    return {"bytes": 2 * cached * Hkv * D + 2 * 4 * pages * Hkv + 2 * T * Hq * D * 2 + T * Hq * 4, "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))


def _nearest8(x):
    """The e4m3 value next to each x of at most 448 in size (halves to the even one)."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_append(s):
    c, bs, Hkv = s.case, s.block, s.case["Hkv"]
    rate = 1e6 ** (-2.0 * torch.arange(D // 2, dtype=torch.float64, device="cuda") / D)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s.pos.double()[:, None] * rate)[:, None, :]

    def turned(x, gain):
        x = x.double()
        if gain is not None:
            x = gain.double() * x * torch.rsqrt(x.square().sum(-1, keepdim=True) / D + 1e-6)
        z = torch.complex(*(x.unflatten(-1, (-1, 2)).unbind(-1) if c["inter"] else x.unflatten(-1, (2, -1)).unbind(-2))) * turn
        return torch.stack([z.real, z.imag], -1 if c["inter"] else -2).flatten(-2)

    slots = s.slots.tolist()
    runs = []  # [first row, rows] of each page of the step
    for r, slot in enumerate(slots):
        if runs and slot == slots[r - 1] + 1 and slot % bs:
            runs[-1][1] += 1
        else:
            runs.append([r, 1])

    def append(x, pool, scale):
        pool, scale = pool.double(), scale.double()
        largest = x.abs().amax(-1).tolist()
        scales = scale.tolist()
        for r, n in runs:
            page, place = divmod(slots[r], bs)
            for h in range(Hkv):
                m, e = math.frexp(max(row[h] for row in largest[r:r + n]))
                want = 2.0 ** max(-64, -64 if m == 0 else e - 9 if m <= 0.875 else e - 8)
                if place and scales[page][h] < want:
                    pool[page, :place, h] = _nearest8(pool[page, :place, h] * scales[page][h] / want)
                scales[page][h] = max(want, scales[page][h]) if place else want
        scale = torch.tensor(scales, dtype=torch.float64, device="cuda")
        at = s.slots.long()
        pool.view(-1, Hkv, D)[at] = _nearest8(x / scale[at // bs, :, None])
        return pool, scale

    (k, ks), (v, vs) = append(turned(s.k_pre, s.gk), s.k_pool, s.k_scale), append(s.v.double(), s.v_pool, s.v_scale)
    return turned(s.q_pre, s.gq), k, v, ks, vs


def _exact_attention(s):
    c = s.case
    Hq, Hkv = c["Hq"], c["Hkv"]
    G = Hq // Hkv
    new, ctx, cu = s.new.tolist(), s.ctx.tolist(), s.cu.tolist()
    o, lse = torch.zeros(s.T, Hq, D, dtype=torch.float64, device="cuda"), torch.zeros(s.T, Hq, dtype=torch.float64, device="cuda")
    for b in range(s.B):
        L = ctx[b] + new[b]
        page = s.table[b, : _up(L, s.block)].long()
        codes = [pool[page].double() for pool in (s.k_pool, s.v_pool)]
        keys, values = ((x * scale[page].double()[:, None, :, None]).reshape(-1, Hkv, D)[:L] for x, scale in zip(codes, (s.k_scale, s.v_scale)))
        rows = slice(cu[b], cu[b + 1])
        seen = torch.arange(L, device="cuda")[None, :] <= ctx[b] + torch.arange(new[b], device="cuda")[:, None]
        for h in range(Hq):
            z = s.q[rows, h].double() @ keys[:, h // G].T / math.sqrt(D)
            z = torch.where(seen, z, -math.inf)
            lse[rows, h] = torch.logsumexp(z, 1)
            o[rows, h] = torch.exp(z - lse[rows, h, None]) @ values[:, h // G]
    return o, lse


def _exact_logprobs(s):
    N, top = s.N, s.case["top"]
    out = [torch.zeros(shape, dtype=torch.float64, device="cuda") for shape in ((N,), (N,), (N, 2), (N, top), (N, top))]
    logprob, entropy, norm, ids, values = out
    for r0 in range(0, N, 128):  # in parts: a row takes 1.2 MB in 64 bits
        part = slice(r0, min(N, r0 + 128))
        z = s.z[part].double()
        largest = z.max(1, keepdim=True).values
        none = torch.isinf(largest)
        lse = torch.logsumexp(z, 1, keepdim=True)
        lp = torch.where(none, -math.inf, z - lse)
        entropy[part] = -torch.special.xlogy(lp.exp(), lp.exp()).sum(1)
        norm[part] = torch.cat([largest, torch.where(none, -math.inf, lse - largest)], 1)
        t = s.tokens[part].long()
        logprob[part] = torch.where(t < 0, 0.0, lp[torch.arange(len(t), device="cuda"), t.clamp(min=0)])
        for k in range(top):
            best = lp.amax(1, keepdim=True)
            at = torch.where(lp == best, torch.arange(s.V, device="cuda"), s.V).amin(1, keepdim=True)
            values[part, k], ids[part, k] = best[:, 0], torch.where(best > -math.inf, at, -1)[:, 0].double()
            lp.scatter_(1, at, -math.inf)
    return logprob, entropy, norm, ids.to(torch.int32), values


def _exact_grad(s):
    dz = torch.empty(s.N, s.V, dtype=torch.float64, device="cuda")
    for r0 in range(0, s.N, 128):
        part = slice(r0, min(s.N, r0 + 128))
        z, t = s.z[part].double(), s.tokens[part].long()
        largest, log = s.norm[part].double().unbind(1)
        p = torch.exp(z - largest[:, None] - log[:, None]).nan_to_num(0.0)
        plogp = torch.special.xlogy(p, p)
        dz[part] = -s.d_entropy[part].double()[:, None] * (plogp + p * s.entropy[part].double()[:, None])
        one = (torch.arange(s.V, device="cuda")[None, :] == t[:, None]).double()
        there = ((t >= 0) & (largest > -math.inf)).double()[:, None]
        dz[part] += s.d_logprob[part].double()[:, None] * there * (one - p)
    return dz


EXACT = {"append": _exact_append, "attention": _exact_attention, "logprobs": _exact_logprobs, "grad": _exact_grad}
