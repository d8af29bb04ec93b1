"""The hand-over of P in the attention kernels (CPU only), by a search over every order of their warps' steps.

Each kernel issues S_(g+1) before it waits for P_g, reads S_g by four warps and takes their P_g through a barrier that
counts one arrival per warp. A warp that runs a step ahead must not count for another's step: the P V product of a step
may start only when every warp has written that step's P."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bwd_qwen3_layer_gb300", "csrc")
STEPS = 5


class Barrier:
    """An mbarrier's state as a tuple: (arrivals left, phases completed)."""

    @staticmethod
    def arrive(b, count):
        return (count, b[1] + 1) if b[0] == 1 else (b[0] - 1, b[1])

    @staticmethod
    def passes(b, parity):
        """A wait by parity passes when the phase before the current one has that parity."""
        return (b[1] & 1) == (parity ^ 1)


def early_products(warps, p_barriers):
    """Steps whose P V product can be issued before every warp has written its P, over all reachable states."""
    s_full0, s_free0 = tuple([(1, 0)] * 2), tuple([(warps, 0)] * 2)
    start = (0, (0,) * warps, s_full0, s_free0, tuple([(warps, 0)] * p_barriers))
    # the issuer's program: S_0, S_1, PV_0, S_2, PV_1, ..., PV_last
    program = [("S", 0)] + [x for g in range(1, STEPS) for x in (("S", g), ("PV", g - 1))] + [("PV", STEPS - 1)]
    bad, seen, todo = set(), {start}, [start]

    def put(t, i, v):
        return t[:i] + (v,) + t[i + 1:]

    while todo:
        pc, at, s_full, s_free, p_full = todo.pop()
        nxt = []
        if pc < len(program):
            kind, g = program[pc]
            if kind == "S":
                if g < 2 or Barrier.passes(s_free[g & 1], ((g >> 1) & 1) ^ 1):
                    nxt.append((pc + 1, at, put(s_full, g & 1, Barrier.arrive(s_full[g & 1], 1)), s_free, p_full))
            else:
                i, parity = (g & 1, (g >> 1) & 1) if p_barriers == 2 else (0, g & 1)
                if Barrier.passes(p_full[i], parity):
                    if any(a < 2 * g + 2 for a in at):
                        bad.add(g)
                    nxt.append((pc + 1, at, s_full, s_free, p_full))
        for w in range(warps):
            g, half = divmod(at[w], 2)
            if g >= STEPS:
                continue
            to = put(at, w, at[w] + 1)
            if half == 0:        # S_g computed: read it
                if Barrier.passes(s_full[g & 1], (g >> 1) & 1):
                    nxt.append((pc, to, s_full, put(s_free, g & 1, Barrier.arrive(s_free[g & 1], warps)), p_full))
            else:                # P_g written
                i = g & 1 if p_barriers == 2 else 0
                nxt.append((pc, to, s_full, s_free, put(p_full, i, Barrier.arrive(p_full[i], warps))))
        for s in nxt:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return bad


def test_the_search_finds_the_race_of_a_single_barrier():
    assert early_products(3, 1)
    assert not early_products(3, 2)


@pytest.mark.parametrize("source,kernel", [
    ("attention_tc.cu", "fa_fwd_tc_kernel"), ("attention_tc.cu", "fa_fwd_tc_persist_kernel"),
    ("ragged_attn.cu", "ragged_attn_kernel")])
def test_no_product_reads_a_p_that_is_not_written(source, kernel):
    text = open(os.path.join(CSRC, source)).read()
    body = text[re.search(r"__global__[^{;]*\b%s\(" % kernel, text).start():]
    body = body[:body.find("__global__", 10)]
    by_parity = re.search(r"auto p_full = \[&\]\(int s\)", body) is not None
    assert not early_products(4, 2 if by_parity else 1)
