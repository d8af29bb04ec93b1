"""The TMEM loads of the kernels' epilogues (CPU only, on the sources).

tcgen05.ld and tcgen05.wait are .aligned: every lane of the warp has to execute them together, and only a warp barrier
guarantees that after a branch that some lanes take. So a loop that loads TMEM and branches after the load must not
skip to its next round by `continue`, and ends with __syncwarp() or votes before the load (a warp's wait does)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bwd_qwen3_layer_gb300", "csrc")


def _strip(text):
    text = re.sub(r"//[^\n]*", "", text)
    return re.sub(r"/\*.*?\*/", "", text, flags=re.S)


def _loops(text):
    """(line, body) of every for loop with a braced body."""
    for m in re.finditer(r"\bfor \(", text):
        at, depth = m.end(), 1
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        rest = text[at:].lstrip()
        if not rest.startswith("{"):
            continue
        at = end = text.index("{", at)
        depth = 0
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        yield text.count("\n", 0, m.start()) + 1, text[at + 1:end - 1]


def divergent_loads(text):
    """Lines of the innermost loops around a TMEM load whose next round's load the lanes may reach apart."""
    bad = []
    for line, body in _loops(_strip(text)):
        loads = [m.end() for m in re.finditer(r"\btmem_ld_\w+(<\d+>)?\(", body)]
        inner = any(re.search(r"\btmem_ld_(32|cols)", b) for _, b in _loops(body))
        if not loads or inner or re.search(r"_warp\(|_sync\(|__syncwarp\(", body[:loads[0]]):
            continue
        after = body[loads[-1]:]
        if re.search(r"\bif (constexpr )?\(", after) or "store" in after:
            last = [s.strip() for s in re.split(r"[;{}]", body) if s.strip()][-1]
            if "continue" in after or last != "__syncwarp()":
                bad.append(line)
    return bad


def test_the_check_sees_lanes_that_leave():
    load = "tmem_ld_32x32b_x32(a, v); tmem_ld_wait();"
    assert divergent_loads("for (int c = 0; c < 4; ++c) { %s if (!mine) continue; put(v); }" % load)
    assert divergent_loads("for (int c = 0; c < 4; ++c) { %s if (mine) { put(v); } }" % load)
    assert not divergent_loads("for (int c = 0; c < 4; ++c) { %s if (mine) { put(v); } __syncwarp(); }" % load)
    assert not divergent_loads("for (int c = 0; c < 4; ++c) { %s for (int e = 0; e < 8; ++e) v[e] *= 2; }" % load)


@pytest.mark.parametrize("source", sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))))
def test_lanes_meet_before_the_next_tmem_load(source):
    with open(os.path.join(CSRC, source)) as f:
        assert divergent_loads(f.read()) == []
