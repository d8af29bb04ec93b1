"""The waits of the 8-bit attention's pipeline (CPU only), by a search over every order of its warps' steps.

A wait by parity passes when the phase before the one it means has not completed yet either, so each wait needs an earlier one
that says it has. The model is one item of several key tiles: the copies of values (four stages, landing as late as they like; a
key tile is waited for by the warp alone whose products free it), the warp that looks up the scales, the warps that issue the
score products and the P V products (three buffers of scores and weights), and the two groups of softmax warps that take the
steps in turn. At each wait that passes and at each arrival the phase must be the one that was meant."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bwd_qwen3_layer_gb300", "csrc", "ragged_attn8.cu")
STAGES, BUFFERS, TOLD, SCALES, QUARTERS = 4, 3, 4, 4, 2       # (two of the four quarters of the rows: all pairs of quarters look
                                                              # alike; of the rings of scales the shorter one)


def _of(done, slot, ring):
    """Phases of a ring's barrier `slot` that are complete once steps 0 .. done - 1 have arrived."""
    return max(0, -(-(done - slot) // ring))


class Search:
    """few: both quarters hear each other's maxima (few rows). pairs: their weights have two buffers. idle: the last quarter has no rows. tail_first: the last tile's value
    rows are cleared before the step's scores are waited for. scales_last: a warp says that its weights are written before it says that
    it has read the scales."""

    def __init__(self, steps, few=False, pairs=False, idle=False, tail_first=False, scales_last=False):
        self.steps, self.few, self.pairs, self.idle, self.tail_first, self.scales_last = steps, few, pairs, idle, tail_first, scales_last
        self.wrong = set()

    def wait(self, name, phases, phase):
        """Whether a wait for the end of phase `phase` (from 0) passes when `phases` have ended."""
        if (phases & 1) != ((phase & 1) ^ 1):
            return False
        if phases != phase + 1:
            self.wrong.add(name)
        return True

    def run(self):
        n_told = 1 if self.few else QUARTERS
        # values landed, score products, P V products issued and done, each warp's place by quarter and
        # group, arrivals at p_full and at told (arrivals of the open phase, phases ended); scales written, arrivals at sc_empty
        start = (0, 0, 0, 0, ((0, 0),) * QUARTERS, ((0, 0),) * BUFFERS, ((0, 0),) * (TOLD * n_told), 0, ((0, 0),) * SCALES)
        seen, todo = {start}, [start]
        while todo:
            s = todo.pop()
            after = list(self.next(s))
            if not after:
                assert s[3] == self.steps, "the search ends in a state where everything waits"
            for t in after:
                if t not in seen:
                    seen.add(t)
                    todo.append(t)
        return self.wrong

    def arrive(self, name, bars, i, count, phase):
        """One of `count` arrivals that end phase `phase`."""
        n, phases = bars[i]
        if phases != phase:
            self.wrong.add("an arrival at " + name)
        b = (0, phases + 1) if n + 1 == count else (n + 1, phases)
        return bars[:i] + (b,) + bars[i + 1:]

    def next(self, s):
        values, scores, issued, done, at, p_full, told, scales, read = s
        if values < self.steps and values < done + STAGES:
            yield values + 1, scores, issued, done, at, p_full, told, scales, read
        n = scores
        if n < self.steps and (n < BUFFERS or self.wait("p_done for S", _of(done, n % BUFFERS, BUFFERS), n // BUFFERS - 1)):
            yield values, scores + 1, issued, done, at, p_full, told, scales, read
        n = issued
        if n < self.steps and self.wait("v_full", _of(values, n % STAGES, STAGES), n // STAGES) \
                and self.wait("p_full", p_full[n % BUFFERS][1], n // BUFFERS):
            if any(at[q][n & 1] < 6 * (n // 2) + 3 for q in range(QUARTERS)):
                self.wrong.add("a product before its weights")
            yield values, scores, issued + 1, done, at, p_full, told, scales, read
        if done < issued:
            yield values, scores, issued, done + 1, at, p_full, told, scales, read
        n = scales
        if n < self.steps and (n < SCALES or self.wait("sc_empty", read[n % SCALES][1], n // SCALES - 1)):
            yield values, scores, issued, done, at, p_full, told, scales + 1, read
        for q in range(QUARTERS):
            for g in range(2):
                for t in self.softmax(s, q, g):
                    yield t

    def busy(self, q):
        return not (self.idle and q == QUARTERS - 1)

    def softmax(self, s, q, g):
        """The next step of quarter q's warp of group g, whose steps are g, g + 2, ...: six places each."""
        values, scores, issued, done, at, p_full, told, scales, read = s
        own, part = divmod(at[q][g], 6)
        n = 2 * own + g
        if n >= self.steps:
            return
        busy = self.busy(q)
        ring = 0 if self.few else q * TOLD
        count = QUARTERS if self.few else 1

        def to(place, p=p_full, m=told, r=read):
            return values, scores, issued, done, at[:q] + (at[q][:g] + (place,) + at[q][g + 1:],) + at[q + 1:], p, m, scales, r

        def tail():
            return n + 1 < self.steps or self.wait("v_full of the tail", _of(values, n % STAGES, STAGES), n // STAGES)

        def s_full():
            return self.wait("s_full", _of(scores, n % BUFFERS, BUFFERS), n // BUFFERS) and \
                (not busy or self.wait("sc_full", _of(scales, n % SCALES, SCALES), n // SCALES))

        base = 6 * own
        if part == 0:                               # scores, and the values' tail
            if not (tail() and s_full() if self.tail_first else s_full() and tail()):
                return
            yield to(base + 1) if busy else to(base + 2)
        elif part == 1:                             # hears the step before, tells its own maxima
            if n > 0 and not self.wait("told", told[ring + (n - 1) % TOLD][1], (n - 1) // TOLD):
                return
            yield to(base + 2, m=self.arrive("told", told, ring + n % TOLD, count, n // TOLD))
        elif part == 2:                             # (few rows: hears them all;) O at a new scale, weights
            if busy and self.few and not self.wait("told", told[ring + n % TOLD][1], n // TOLD):
                return
            if self.pairs and n > 1 and not self.wait("p_done for P", _of(done, (n - 2) % BUFFERS, BUFFERS), (n - 2) // BUFFERS):
                return
            if busy and n > 0:                      # (only if the maximum is raised: the step goes on either way)
                self.wait("p_done for O", _of(done, (n - 1) % BUFFERS, BUFFERS), (n - 1) // BUFFERS)
            yield to(base + 3)
        else:                                       # weights written, scales read: one after the other
            if (part == 3) != self.scales_last:
                yield to(base + part + (1 if part == 3 else 2), r=self.arrive("sc_empty", read, n % SCALES, QUARTERS, n // SCALES))
            else:
                yield to(base + part + (1 if part == 3 else 2), p=self.arrive("p_full", p_full, n % BUFFERS, QUARTERS, n // BUFFERS))


KINDS = [dict(), dict(few=True), dict(idle=True), dict(few=True, pairs=True)]


def test_the_search_finds_a_tail_cleared_too_early():
    assert "v_full of the tail" in Search(5, tail_first=True).run()
    assert "v_full of the tail" in Search(5, few=True, tail_first=True).run()
    assert not Search(4, tail_first=True).run()     # four tiles: no stage is used twice


def test_the_search_finds_scales_that_are_given_back_too_early():
    assert "an arrival at sc_empty" in Search(5, idle=True, scales_last=True).run()


def _scales_last(text):
    """Whether a step's warps arrive at p_full before they arrive at sc_empty."""
    body = text[text.index("// Step j of the piece by a warp with rows"):]
    p, sc = ([m.start() for m in re.finditer(r"mbar_arrive\(%s\(n\)\)" % x, body)] for x in ("p_full", "sc_empty"))
    assert len(p) == len(sc) == 3
    return any(a < b for a, b in zip(p, sc))


def _tail_first(text):
    """Whether the kernel's steps (whole tiles', few rows', those of warps without rows) clear the tail before they wait for S."""
    body = text[text.index("// Step j of the piece by a warp with rows"):]
    tails = [m.start() for m in re.finditer(r"clear_tail\(end", body)]
    waits = [m.start() for m in re.finditer(r"a8_wait\(s_full\(n\)", body)]
    assert len(tails) == len(waits) == 3
    return [t < w for t, w in zip(tails, waits)]


@pytest.mark.parametrize("steps", [5, 6])
@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_every_wait_is_for_the_phase_that_is_meant(kind, steps):
    text = open(SOURCE).read()
    first = _tail_first(text)
    # the step of warps without rows beside one with rows: either may be the early one
    early = [first[0], first[1], first[0] or first[2], first[1]][kind]
    assert not Search(steps, tail_first=early, scales_last=_scales_last(text), **KINDS[kind]).run()
