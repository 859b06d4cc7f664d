"""The hand-overs between the roles of the tensor-core passes of linear attention, on the CPU.

csrc/linattn_tc.cu hands tiles, products and states from role to role through mbarriers, which are
waited for by the parity of their phase, and through named barriers.  A wait by parity is sound only
while the barrier is at most one phase ahead of the waiter: two phases on it looks not done, and a wait for
a phase whose predecessor is still open looks done.  Each role is written here as the sequence of its
waits and signals, and run with the others under schedules that hold one of them back as long as anything else
can move, which gives the rest the largest lead that the hand-overs allow.  How often each barrier exists
is read from the source.
"""
import os
import re
from collections import deque

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = open(os.path.join(ROOT, "chunked_scan_mixer_gb300", "csrc", "linattn_tc.cu")).read()


def copies(first, NS):
    """How many barriers each name of an enum of the source stands for."""
    body = re.search(r"enum \{ (" + first + r" = 0.*?)kBars", SOURCE, re.S).group(1)
    at, value, last = {}, {"NS": NS}, -1
    for item in filter(None, (x.strip() for x in body.split(","))):
        name, _, expr = (x.strip() for x in item.partition("="))
        last = sum(value[x.strip()] if x.strip() in value else int(x) for x in expr.split("+")) if expr else last + 1
        at[name] = value[name] = last
    names = list(at)
    return {n: at[names[i + 1]] - at[n] if i + 1 < len(names) else None for i, n in enumerate(names)}


class Machine:
    """Roles as generators that yield ("wait", bar, phase), ("sync", name, members) or ("arrive", name, members);
    commits and copies complete later, in order, by the role "engine"."""

    def __init__(self, counts):
        self.counts, self.phase, self.arrived = counts, {}, {}
        self.named, self.queue, self.late = {}, deque(), []

    def signal(self, bar):
        n = self.arrived.get(bar, 0) + 1
        if n == self.counts.get(bar[0], 1):
            self.phase[bar] = self.phase.get(bar, 0) + 1
            n = 0
        self.arrived[bar] = n

    def commit(self, *bar):
        self.queue.append(bar)

    def may_go(self, who, op):
        if op[0] == "wait":
            _, bar, phase = op
            have = self.phase.get(bar, 0)
            assert have <= phase + 1, f"{who} waits for phase {phase} of {bar}, which is {have - phase - 1} phases on"
            if have & 1 != phase & 1:
                assert have == phase + 1, f"{who} passes phase {phase} of {bar}, of which {have} are done"
                return True
            return False
        _, name, members = op
        here = self.named.setdefault(name, {})
        if who not in here:
            here[who] = op[0]
            if len(here) == len(members):
                assert set(here) == set(members), (name, here)
                self.done[name] = {w for w, kind in here.items() if kind == "sync" and w != who}
                self.named[name] = {}
                return True
        elif op[0] == "arrive":
            raise AssertionError(f"{who} arrives twice at {name}")
        return op[0] == "arrive"

    def run(self, roles, held):
        self.done = {}
        roles = {n: g for n, g in roles.items()}
        todo = {}
        for n, g in roles.items():
            todo[n] = next(g, None)
        waiting = {}  # named barrier that a role sits in

        def step(who):
            if who == "engine":
                if not self.queue:
                    return False
                self.signal(self.queue.popleft())
                return True
            op = todo[who]
            if op is None:
                return False
            if who in waiting:
                if who not in self.done.get(waiting[who], ()):
                    return False
                self.done[waiting.pop(who)].discard(who)
            elif not self.may_go(who, op):
                if op[0] == "sync":
                    waiting[who] = op[1]
                return False
            todo[who] = next(roles[who], None)
            return True

        order = [n for n in (*roles, "engine") if n != held] + [held]
        while any(todo.values()) or self.queue:
            for who in order:
                if step(who):
                    break
            else:
                raise AssertionError(f"nothing can move: {todo}")


def output_pass(D, kind, items, nit, lengths, steep, held):
    """lin_out_tc_kernel.  kind: "q" several queries on a key head, "k" several keys on a state, "" one of each."""
    NS, early = (4, True) if D == 64 else (2, False)
    n = copies("XF", NS)
    mode_a, mode_b = kind == "q", kind == "k"
    total = nit * items
    m = Machine({"E": 2})
    A, B, G, S = "A", "B", "mma", "mma_s"

    def item(it):
        return it // items, it % items

    def mma():
        for it in range(-1, total):
            ci, r = item(it) if it >= 0 else (0, -1)
            first, last = r == 0, r == items - 1
            new_y, end_y = not mode_b or first, not mode_b or last
            ki = it if mode_b else ci

            def products():
                if first and ci > 0:
                    yield "sync", "SP", (G, B)
                yield "sync", f"GT{it & 1}", (G, A)
                if new_y and steep:
                    m.commit("BC", 0)
                if not mode_a or first:
                    yield "wait", ("VF", ki % NS), ki // NS
                    if lengths:
                        yield "sync", f"VZ{ki & 1}", (G, B, S)
                if steep and new_y:
                    yield "sync", "SC", (G, A)
                if end_y:
                    m.commit("YD", 0)
                if mode_a and last:
                    m.commit("YL", 0)
                if mode_b:
                    m.commit("E", ki % NS)
                    m.commit("YI", 0)

            if it > 0 and (mode_b or it + 1 < total):
                yield "wait", ("YI" if mode_b else "YD", 0), it - 1
            if not early and it >= 0:
                yield from products()
            if it + 1 < total:
                cn, rn = item(it + 1)
                xn, kn = (cn, it + 1) if mode_b else (it + 1, cn if mode_a else it + 1)
                if not mode_b or rn == 0:
                    yield "wait", ("XF", xn % NS), xn // NS
                if not mode_a or rn == 0:
                    yield "wait", ("KF", kn % NS), kn // NS
                m.commit("BG", (it + 1) % n["BG"])
                if mode_a and rn == items - 1:
                    m.commit("BGK", cn % n["BGK"])
            if early and it >= 0:
                yield from products()
        yield "wait", ("YI" if mode_b else "YL" if mode_a else "YD", 0), (nit if mode_a else total) - 1
        assert not any(c[0] in ("YD", "YL", "YI", "E", "BG", "BGK") for c in m.queue), "the CTA would end before a commit"

    def mma_s():
        tiles, per = (nit, 1) if mode_a else (total, items)
        done = 0
        for ki in range(tiles):
            if lengths:
                yield "sync", f"VZ{ki & 1}", (G, B, S)
            if ki // per + 1 >= nit:
                continue
            for piece in range(1 if D == 64 else 2):
                yield "sync", "KT", (S, B)
                yield "wait", ("VF", ki % NS), ki // NS
                m.commit("SD" if D == 64 or piece else "SH", 0)
            done += 1
        if done:
            yield "wait", ("SD", 0), done - 1

    def loads():
        nx = nkv = 0
        for it in range(total):
            ci, r = item(it)
            if not mode_b or r == 0:
                if nx >= NS:
                    yield "wait", ("XE", nx % NS), nx // NS - 1
                m.commit("XF", nx % NS)
                nx += 1
            if not mode_a or r == 0:
                if nkv >= NS:
                    yield "wait", ("E", nkv % NS), nkv // NS - 1
                m.commit("KF", nkv % NS)
                m.commit("VF", nkv % NS)
                nkv += 1

    def stores():
        for g in range(nit if mode_b else total):
            yield "wait", ("OS", g % NS), g // NS
            m.signal(("XE", g % NS))

    def epilogue():
        groups = 0
        for it in range(-1, total):
            ci, r = item(it) if it >= 0 else (0, -1)
            last = r == items - 1
            new_y, end_y = it >= 0 and (not mode_b or r == 0), it >= 0 and (not mode_b or last)
            if it >= 0:
                yield "arrive", f"GT{it & 1}", (G, A)
            if steep and new_y:
                yield "wait", ("BC", 0), groups
                yield "arrive", "SC", (G, A)
            for step in range(2):
                if (step == 0) == early:
                    if it + 1 < total:
                        yield "wait", ("BG", (it + 1) % n["BG"]), (it + 1) // n["BG"]
                elif end_y:
                    yield "wait", ("YD", 0), groups
                    if not mode_b and last:
                        m.signal(("E", (ci if mode_a else it) % NS))
                    m.signal(("OS", groups % NS))
                    groups += 1

    def state():
        tiles, per = (nit, 1) if mode_a else (total, items)
        for ki in range(tiles):
            ci, last = ki // per, ki % per == per - 1
            if mode_a and lengths:
                yield "wait", ("VF", ki % NS), ki // NS
            if not mode_a:
                yield "wait", ("KF", ki % NS), ki // NS
                yield "wait", ("BG", ki % n["BG"]), ki // n["BG"]
                if lengths:
                    yield "wait", ("VF", ki % NS), ki // NS
            if lengths:
                yield "arrive", f"VZ{ki & 1}", (G, B, S)
            if ci + 1 >= nit:
                m.signal(("E", ki % NS))
                continue
            if mode_a:
                yield "wait", ("KF", ki % NS), ki // NS
                yield "wait", ("BGK", ci % n["BGK"]), ci // n["BGK"]
            yield "arrive", "KT", (S, B)
            if D != 64:
                yield "wait", ("SH", 0), ki
                yield "arrive", "KT", (S, B)
            yield "wait", ("SD", 0), ki
            m.signal(("E", ki % NS))
            if last:
                yield "wait", ("YL" if mode_a else "YD", 0), ci
                yield "arrive", "SP", (G, B)

    m.run({G: mma(), S: mma_s(), "loads": loads(), "stores": stores(), A: epilogue(), B: state()}, held)


def summary_pass(D, P, total, held):
    """lin_sum_tc_kernel over ``total`` tiles."""
    NS, NP = (4 if D == 64 else 2), (1 if D == 128 and P == 3 else 2)
    m = Machine({})
    G, B = "mma", "B"

    def mma():
        for it in range(total):
            yield "wait", ("VF", it % NS), it // NS
            if it >= 2:
                yield "sync", f"DR{it & 1}", (G, B)
            yield "sync", f"KT{it & 1}", (G, B)
            m.commit("E", it % NS)
            m.commit("AD", it & 1)

    def loads():
        for it in range(total):
            if it >= NS:
                yield "wait", ("E", it % NS), it // NS - 1
            m.commit("KF", it % NS)
            m.commit("VF", it % NS)

    def pieces():
        def drain(it):
            yield "wait", ("AD", it & 1), it >> 1
            if it + 2 < total:
                yield "arrive", f"DR{it & 1}", (G, B)

        for it in range(total + 1):
            if NP == 1 and it > 0:
                yield from drain(it - 1)
            if it < total:
                yield "wait", ("KF", it % NS), it // NS
                yield "wait", ("VF", it % NS), it // NS
                yield "arrive", f"KT{it & 1}", (G, B)
            if NP == 2 and it > 0:
                yield from drain(it - 1)

    m.run({G: mma(), "loads": loads(), B: pieces()}, held)


@pytest.mark.parametrize("held", ["mma", "mma_s", "loads", "stores", "A", "B", "engine"])
@pytest.mark.parametrize("kind, items", [("", 1), ("q", 2), ("q", 3), ("q", 4), ("k", 2), ("k", 3), ("k", 4)])
@pytest.mark.parametrize("D", [64, 128])
def test_no_role_of_the_output_pass_outruns_a_wait(D, kind, items, held):
    for nit in range(1, 12):
        for lengths in (False, True):
            for steep in (False, True):
                output_pass(D, kind, items, nit, lengths, steep, held)


@pytest.mark.parametrize("held", ["mma", "loads", "B", "engine"])
@pytest.mark.parametrize("D, P", [(64, 2), (64, 3), (128, 2), (128, 3)])
def test_no_role_of_the_summary_pass_outruns_a_wait(D, P, held):
    for total in range(1, 14):
        summary_pass(D, P, total, held)
