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


def play(warps, victim):
    """Runs generators that yield (barrier, parity) to wait for, or None: the victim moves only
    when no other can, and all get to their end."""
    waits, left = {}, set(range(len(warps)))

    def move(i):
        """Whether warp i got further."""
        if waits.get(i) is not None and not waits[i][0].done(waits[i][1]):
            return False
        try:
            waits[i] = next(warps[i])
        except StopIteration:
            left.discard(i)
        return True

    while left:
        if not any([move(i) for i in sorted(left) if i != victim]):
            assert victim in left and move(victim), f"warps {sorted(left)} wait for ever"


def role(text, start, end):
    """(operation, barrier) in the order of the source between two marks."""
    body = text[text.index(start):text.index(end, text.index(start))]
    body = re.sub(r"//[^\n]*", "", body)
    body = body[re.search(r"for \((int c = 0)?; c < chunks; \+\+c\)", body).start():]
    ops = re.findall(r"(warp_wait|warp_publish|warp_arrive|mbar_arrive)\(bars \+ (B_\w+)", body)
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

    play([loads(), issues(), decays()] + [warp(p_ops, i == 0) for i in range(4)] +
         [warp(s_ops, False) for _ in range(8)], victim)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("victim", range(15))
def test_state_waits_see_their_phase(back, victim):
    """The same for the kernel of the states: loads, products, decays, four scaling warps and
    eight with the state."""
    code = code_of("ckda_linear_state.cu")
    at = code.index("else if (warp >= 4 && warp < 8)")
    split = code.index("else if (warp >= 8)", at)
    pattern = r"(warp_wait|warp_publish|warp_arrive|mbar_arrive)\(bars \+ (B_\w+)(?: \+ (ix \+ 1))?"
    scale = [o[:2] for o in re.findall(pattern, code[at:split]) if not o[2]]  # (but tails)
    body, _ = loop_at(code, code.index("for (; i < chunks;", split))
    state = [o[:2] for o in re.findall(pattern, body)]
    assert scale == [("warp_wait", "B_G"), ("mbar_arrive", "B_GFREE"), ("warp_wait", "B_FULL"),
                     ("warp_wait", "B_DF"), ("warp_publish", "B_KT")]
    assert state == [("warp_wait", "B_G"), ("mbar_arrive", "B_GFREE"), ("warp_wait", "B_DF"),
                     ("warp_arrive", "B_DFREE")]
    chunks, slots = 7, 4
    steps = chunks if back else chunks - 1
    count = dict(B_KT=4, B_DFREE=8, B_GFREE=12)
    bars = {}

    def bar(name, i=0):
        return bars.setdefault((name, i), Barrier(count.get(name, 1)))

    def loads():
        for i in range(2 * steps):
            if i >= slots:
                yield bar("B_EMPTY", i % slots), (i // slots - 1) & 1
            bar("B_FULL", i % slots).arrive()
        for j in range(max(0, 2 * steps - slots), 2 * steps):
            yield bar("B_FULL", j % slots), (j // slots) & 1

    def issues():
        for i in range(steps):
            ix, p = 2 * i % slots, i & 1
            yield bar("B_FULL", ix + 1), (i // 2) & 1
            if i >= 2:
                yield bar("B_DFREE", p), (i // 2 - 1) & 1
            yield bar("B_KT"), p
            for b in (bar("B_DF", p), bar("B_EMPTY", ix), bar("B_EMPTY", ix + 1)):
                b.arrive()

    def decays():
        for i in range(steps):
            if i >= 1:
                yield bar("B_GFREE"), (i - 1) & 1
            bar("B_G").arrive()

    def warp(ops, lag):
        for i in range(steps):
            for op, name in ops:
                if op != "warp_wait":
                    bar(name, i & 1 if name == "B_DFREE" else 0).arrive()
                elif name == "B_G":
                    yield bar(name), i & 1
                elif name == "B_FULL":
                    yield bar(name, 2 * i % slots), (i // 2) & 1
                elif i >= lag:  # the product of this step, or of the one before
                    yield bar(name, (i - lag) & 1), ((i - lag) // 2) & 1
                yield None

    play([loads(), issues(), decays()] + [warp(scale, 1) for _ in range(4)] +
         [warp(state, 0) for _ in range(8)], victim)


def code_of(name):
    return re.sub(r"//[^\n]*", "", source(name))


def loop_at(code, start):
    """The braces' content of the loop that begins at or behind `start`, and what follows it."""
    at = code.index("{", start)
    depth, end = 0, at
    for end in range(at, len(code)):
        depth += {"{": 1, "}": -1}.get(code[end], 0)
        if depth == 0:
            break
    return code[at + 1:end], code[end + 1:]


@pytest.mark.parametrize("name,mark,counter,per", [
    ("ckda_linear_fwd.cu", "int w = warp - 4", "c", lambda i: 1),
    ("ckda_linear_state.cu", "const int s = (warp - 8) >> 2", "i", lambda i: 1 + (i > 0))])
def test_a_warp_that_gives_up_meets_the_others(name, mark, counter, per):
    """Named hardware barriers wait without a limit: wherever a warp leaves its loop, it meets
    the others in as many more as they may come to."""
    code = code_of(name)
    body, behind = loop_at(code, code.index(f"for (; {counter} < chunks;", code.index(mark)))
    assert body.count("named_sync(") == per(1)
    left = re.search(r"leave_group\(\d, \d+, ([^;]*)\);", behind[:200]).group(1)
    syncs = [m.start() for m in re.finditer(r"named_sync\(", body)]
    gives_up = [m.start() for m in re.finditer(r"warp_wait\(", body)]
    assert syncs and gives_up
    for chunks in (1, 2, 5):
        for i in range(chunks + 1):
            done = sum(per(j) for j in range(i))
            more = [sum(s < g for s in syncs) - (per(1) - per(i)) for g in gives_up]
            for m in [0] if i == chunks else more:
                rest = eval(left, {"chunks": chunks, counter: i})
                assert done + m + max(rest, 0) == sum(per(j) for j in range(chunks)), (i, m)


def test_gradient_groups_count_their_barriers():
    """The same for the gradient kernel, whose groups of warps count the barriers they met."""
    code = code_of("ckda_linear_bwd.cu")
    body, behind = loop_at(code, code.index("for (unsigned block", code.index("auto together")))
    assert "named_sync" not in body
    put = body[body.index("auto put"):body.index("};", body.index("auto put"))]
    tail, rest = loop_at(put, put.index("if (tail)"))
    assert tail.count("together()") == 1 and put.count("together()") == 2
    # A: dQ, half of dV where values are wider than 64, and two more; B: dK; C: half of dV
    assert body.count("together()") - 2 == 2
    assert [m for m in re.findall(r"put\(&(\w+)", body)] == ["mdq", "mdk", "mdv"]
    assert "if (wg == 2 || (wg == 0 && VP == 2))" in body
    each = re.search(r"all \+= ([^;]*);", behind).group(1)
    py = re.sub(r"\(([^()]*) \? (\w+) : (\w+)\)", r"(\2 if \1 else \3)", each)
    for wg, VP, t in ((wg, VP, t) for wg in range(3) for VP in (1, 2) for t in (False, True)):
        puts = 1 + (wg == 0 and VP == 2)
        assert eval(py, dict(wg=wg, VP=VP, tail=t)) == puts * (1 + t) + 2 * (wg == 0)
    assert "leave_group(1 + wg, 128, all - met)" in behind


@pytest.mark.parametrize("name", ["ckda_linear_fwd.cu", "ckda_linear_state.cu"])
def test_loads_in_flight_are_waited_for(name):
    """However many loads a CTA has begun when it gives up, it waits for the last phase of each
    slot before its shared memory is given back."""
    code = code_of(name)
    m = re.search(r"for \(int j = (max\(0, i - kSlots\)); j < i; \+\+j\)\s*"
                  r"mbar_wait\(bars \+ B_FULL \+ ([^,]*), ([^;]*)\);", code)
    assert m
    slot, parity = m.group(2), m.group(3).replace("/", "//")
    for slots in (4, 5, 6):
        for begun in range(20):
            last = {}
            for i in range(begun):
                last[i % slots] = (i // slots) & 1  # parity of the phase that this load completes
            env = lambda **kw: dict(kSlots=slots, i=begun, max=max, **kw)
            waited = {eval(slot, env(j=j)): eval(parity, env(j=j))
                      for j in range(eval(m.group(1), env()), begun)}
            assert waited == last, (slots, begun)


def test_gradient_loads_in_flight_are_waited_for():
    """The same for the gradient kernel: five barriers, a phase a chunk each."""
    code = code_of("ckda_linear_bwd.cu")
    at = code.index("int begun = 0;")
    body, behind = loop_at(code, code.index("for (; block < blocks;", at))
    stages = {b: int(s) for b, s in re.findall(r"\{(B_\w+), (\d)\}", behind[:300])}
    assert len(stages) == 5
    for b, s in stages.items():  # begun reaches s right behind the loads on b
        loads = [m.start() for m in re.finditer(rf"bars \+ {b}[,)]", body)]
        mark = body.index(f"begun = {s};")
        assert loads and all(x < mark for x in loads)
        assert s == 1 or min(loads) > body.index(f"begun = {s - 1};")
    head = code[code.index("for (; block < blocks;", at):][:90]
    assert "par ^= 1, begun = 0" in head
    rule = re.sub(r"\s+", " ", behind[:500])
    assert ("if (begun >= l[1] || block != blockIdx.x) "
            "mbar_wait(bars + l[0], begun >= l[1] ? par : par ^ 1);") in rule
