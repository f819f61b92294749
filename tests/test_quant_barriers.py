"""The hardware barriers of the products of block-quantised operands, which have no limit,
after a bounded wait that gave up: each role's steps are read from the kernel's source and
run as a model, with give-ups at every sum and in every order of the warps. No warp may
count twice in one meeting, and all have to come to their end."""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_route_layout_gb300", "csrc",
                      "ep_qlinear_mma.cu")
EPILOGUE_WARPS = 8
MEETING = 1 + EPILOGUE_WARPS            # warps of a hardware barrier


def code(text):
    return [line.split("//")[0].strip() for line in text.splitlines()]


def body(lines, opening):
    """The lines of the block that the first line with `opening` opens, and the number behind it."""
    at = next(i for i, line in enumerate(lines) if opening in line)
    depth = 0
    for i in range(at, len(lines)):
        depth += lines[i].count("{") - lines[i].count("}")
        if depth == 0:
            return lines[at + 1:i], i + 1
    raise AssertionError(opening)


STEPS = [(r"if \(n_acc >= 2\) named_sync\((\d) \+ \(n_acc & 1\)", "sync_later"), (r"named_sync\((\d) \+ \(n_acc & 1\)", "sync"),
         (r"named_arrive\((\d) \+ \(n_acc & 1\)", "arrive"), (r"warp_wait\(&bar->acc_full\[", "sum"), (r"mma8_commit\(sum0", "commit"),
         (r"&bar->met\) = n_acc \+ 1", "publish"), (r"wait_met\(bar, n_acc\)", "paced")]


def steps(lines):
    """What a role does for one sum: (what, number of the barrier)."""
    found = []
    for line in lines:
        for pattern, what in STEPS:
            m = re.search(pattern, line)
            if m:
                found.append((what, int(m.group(1)) if m.groups() else None))
                break
    return found


def roles(text):
    lines = code(text)
    marks = ["} else if (warp == 1) {", "} else if (warp == 2) {", "} else if (warp == 3 &&", "registers_more<"]
    at = [next(i for i, line in enumerate(lines) if mark in line) for mark in marks]
    end = next(i for i, line in enumerate(lines) if "tmem_free_own(" in line)
    parts = lines[at[0]:at[1]], lines[at[1]:at[2]], lines[at[3]:end]
    for part in parts:
        assert sum("for (int kb = w.kb0; kb < w.kb1; ++kb, ++n_acc" in line for line in part) == 1
    mma, sums, epilogue = [steps(body(part, "for (int kb = w.kb0;")[0]) for part in parts]
    assert any("for (int last = n_acc < 2 ? 0 : n_acc - 2; last < n_acc; ++last) named_sync(1 + (last & 1)" in line for line in parts[0])
    return mma, sums, epilogue


class Model:
    """n sums. `mma_gives_up`, `sums_gives_up`: the sum at which that warp's wait gives up, n for
    none. A warp is a generator that yields a condition to wait for."""

    def __init__(self, text, n, mma_gives_up, sums_gives_up):
        mma, sums, epilogue = roles(text)
        self.n = n
        self.arrived = {b: [] for b in (1, 2, 3, 4)}
        self.phase = dict.fromkeys(self.arrived, 0)
        self.made = set()
        self.met = 0
        self.warps = {"mma": self.mma(mma, mma_gives_up), "sums": self.sums(sums, sums_gives_up)}
        for i in range(EPILOGUE_WARPS):
            self.warps[f"epilogue {i}"] = self.epilogue(f"epilogue {i}", epilogue)

    def arrive(self, who, barrier):
        assert who not in self.arrived[barrier], f"{who} counts twice at barrier {barrier}"
        self.arrived[barrier].append(who)
        phase = self.phase[barrier]
        if len(self.arrived[barrier]) == MEETING:
            self.arrived[barrier] = []
            self.phase[barrier] += 1
        return lambda: self.phase[barrier] > phase

    def mma(self, plan, gives_up):
        ok = True
        for i in range(self.n):
            ok = ok and i != gives_up
            for what, barrier in plan:
                if what == "sync" or (what == "sync_later" and i >= 2):
                    yield self.arrive("mma", barrier + (i & 1))
                elif what == "commit" and ok:
                    self.made.add(i)
                elif what == "publish":
                    yield lambda: True
                    self.met = i + 1
            yield lambda: True
        for i in range(max(self.n - 2, 0), self.n):
            yield self.arrive("mma", 1 + (i & 1))

    def sums(self, plan, gives_up):
        ok = True
        for i in range(self.n):
            for what, barrier in plan:
                if what == "sum" and ok:
                    ok = i != gives_up
                    if ok:          # it comes, or the wait runs out
                        yield lambda: i in self.made or self.stuck
                        ok = i in self.made
                elif what == "paced" and not ok:
                    yield lambda: self.met > i
                elif what == "arrive":
                    yield lambda: True
                    self.arrive("sums", barrier + (i & 1))

    def epilogue(self, who, plan):
        for i in range(self.n):
            for what, barrier in plan:
                if what == "sync":
                    yield self.arrive(who, barrier + (i & 1))
                elif what == "arrive":
                    yield lambda: True
                    self.arrive(who, barrier + (i & 1))

    def run(self, order):
        waiting = dict.fromkeys(self.warps, lambda: True)
        while waiting:
            self.stuck = False
            ready = [w for w in waiting if waiting[w]()]
            if not ready:           # a second later: bounded waits give up
                self.stuck = True
                ready = [w for w in waiting if waiting[w]()]
            assert ready, f"{sorted(waiting)} wait for ever"
            who = order.choice(ready)
            try:
                waiting[who] = next(self.warps[who])
            except StopIteration:
                del waiting[who]


def source():
    with open(SOURCE) as f:
        return f.read()


def test_the_roles_are_as_the_model_takes_them():
    mma, sums, epilogue = roles(source())
    assert [w for w, _ in mma] == ["sync_later", "commit", "publish"]
    assert [w for w, _ in sums] == ["sum", "paced", "arrive"]
    assert [w for w, _ in epilogue] == ["sync", "arrive"]


@pytest.mark.parametrize("n", [1, 2, 3, 4, 7, 16])
def test_every_role_comes_to_its_end_wherever_a_wait_gives_up(n):
    text = source()
    for mma_gives_up in range(n + 1):
        for sums_gives_up in range(n + 1):
            for seed in range(6):
                Model(text, n, mma_gives_up, sums_gives_up).run(random.Random(seed * 1000 + mma_gives_up * 50 + sums_gives_up))


def test_the_model_finds_a_warp_that_runs_ahead():
    """Without its wait for the MMA warp, the sums' warp tells of sums that are two ahead."""
    text = source().replace("wait_met(bar, n_acc);", "")
    found = 0
    for seed in range(20):
        try:
            Model(text, 8, 8, 2).run(random.Random(seed))
        except AssertionError:
            found += 1
    assert found >= 19


def test_a_sum_that_nobody_saw_marks_the_call_as_failed():
    """The sums' warp says so whatever wait of its own gave up, ahead of telling the epilogue."""
    lines = code(source())
    sums = lines[next(i for i, line in enumerate(lines) if "} else if (warp == 2) {" in line):]
    loop, _ = body(sums, "for (int kb = w.kb0;")
    gave_up, after = body(loop, "if (!ok) {")
    assert any("bar->failed = 1;" in line for line in gave_up)
    assert next(i for i, line in enumerate(loop) if "named_arrive(" in line) >= after
