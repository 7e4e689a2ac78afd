"""The barriers of the chunked linear attention kernels, on the CPU: the order of
waits and arrivals is read from the kernel's source, and played by a scheduler
that always holds one warp back.  An mbarrier is looked at by the parity of a
phase, so a warp that looks two phases late waits for one that cannot come."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "gated_delta_rule_ckda_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0
        if self.left == 0:
            self.left = self.count
            self.phase += 1

    def done(self, parity):
        return (self.phase & 1) != parity


def role(text, start, end):
    """(operation, barrier) in the order of the source between two marks."""
    body = text[text.index(start):text.index(end, text.index(start))]
    body = re.sub(r"//[^\n]*", "", body)
    body = body[body.index("for (int c = 0; c < chunks; ++c)"):]
    ops = re.findall(r"(warp_wait|warp_publish|warp_arrive|mbar_arrive|group_sync)\(bars \+ (B_\w+)",
                     body)
    assert len(ops) > 4
    return ops


P_MARK, STATE_MARK, END_MARK = "- P and o", "-- state", "-- teardown"


@pytest.mark.parametrize("slots", [5, 6])
@pytest.mark.parametrize("victim", range(15))
def test_forward_waits_see_their_phase(slots, victim):
    """Of the loading, issuing, decay, four P and eight state warps, the victim moves only
    when no other can: every warp still gets through all chunks."""
    text = source("ckda_linear_fwd.cu")
    p_ops = [o for o in role(text, P_MARK, STATE_MARK) if o != ("warp_wait", "B_FULL")]  # (tails)
    s_ops = role(text, STATE_MARK, END_MARK)
    chunks = 7
    count = dict(B_P=4, B_HREADY=8, B_KT=8, B_GFREE=12, B_STAGED=4)
    bars = {}

    def bar(name, i=0):
        return bars.setdefault((name, i), Barrier(count.get(name, 1)))

    def loads():
        for i in range(3 * chunks):
            if i >= slots:
                j = i - slots
                c = j // 3
                yield bar("B_O" if j % 3 == 0 else "B_DF", c & 1), (c >> 1) & 1
            bar("B_FULL", i % slots).arrive()

    def full(i):
        return bar("B_FULL", i % slots), (i // slots) & 1

    def issues():
        for c in range(-1, chunks):
            par = c & 1
            if c >= 0:
                yield full(3 * c + 2)
                yield bar("B_P"), par
                bar("B_PV").arrive()
                yield bar("B_HREADY"), par
                bar("B_O", par).arrive()
            if c + 1 < chunks:
                yield full(3 * (c + 1))
                yield full(3 * (c + 1) + 1)
                if c >= 0:
                    yield bar("B_PV"), par
                bar("B_S").arrive()
            if c >= 0:
                yield bar("B_KT"), par
                bar("B_DF", par).arrive()

    def decays():
        for c in range(chunks):
            if c > 0:
                yield bar("B_GFREE"), (c - 1) & 1
            bar("B_G").arrive()

    def warp(ops, lead):
        for c in range(chunks):
            par = c & 1
            for op, name in ops:
                if op == "group_sync":
                    bar(name).arrive()
                    yield bar(name), par
                elif op != "warp_wait":
                    if name != "B_HFREE" or lead:
                        bar(name).arrive()
                elif name in ("B_O", "B_DF"):
                    yield bar(name, par), (c >> 1) & 1
                elif name == "B_HFREE":
                    if c > 0:
                        yield bar(name), (c - 1) & 1
                elif name == "B_FULL":
                    yield full(3 * c + 1)
                else:
                    yield bar(name), par
                yield None  # another may go first

    warps = [loads(), issues(), decays()] + [warp(p_ops, i == 0) for i in range(4)] + \
            [warp(s_ops, False) for _ in range(8)]
    waits = {}

    def move(i):
        """Whether warp i, held back or not, got further."""
        if i in waits and waits[i] is not None and not waits[i][0].done(waits[i][1]):
            return False
        try:
            waits[i] = next(warps[i])
        except StopIteration:
            left.discard(i)
        return True

    left = set(range(len(warps)))
    while left:
        if not any([move(i) for i in sorted(left) if i != victim]):
            assert victim in left and move(victim), f"warps {sorted(left)} wait for ever"
