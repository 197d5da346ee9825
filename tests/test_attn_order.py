"""Order of the paged attention's two softmax slots, explored on the CPU.

A CTA's issuer and its two slots are three programs that meet at mbarriers.
Every interleaving of them is walked for short lists of units (rows in both
slots or in one, so many key tiles), with K, V, Q and the units always there.
A slot that marks values of unit u (in place u & 1) must not do so while the
other slot has yet to read the marks of an earlier unit in that place, and
every walk must end."""
import itertools

import pytest


def issuer(units):
    for two, n in units:
        if two:
            yield from [("signal", "s0"), ("signal", "s1")]
            for j in range(n):
                more = j + 1 < n
                for i in (0, 1):
                    yield ("wait", f"p{i}")
                    yield ("signal", f"s{i}" if more else f"o{i}")
        else:
            for j in range(min(n, 2)):
                yield ("signal", f"s{j}")
            for j in range(n):
                yield ("wait", f"p{j & 1}")
                yield ("signal", f"s{j & 1}" if j + 2 < n else f"o{j & 1}")


def slot(i, units, ordered):
    pending = False
    for u, (two, n) in enumerate(units):
        tiles = range(n) if two else range(i, n, 2)
        for _ in tiles:
            if i == 0 or not two:  # any tile may hold values that some rows do not see
                if ordered and i == 0:
                    yield ("seen", u)
                yield ("mark", u)
            yield ("wait", f"s{i}")
            if pending:
                yield ("wait", "merged")
                pending = False
            yield ("signal", f"p{i}")
        if pending:
            yield ("wait", "merged")
            pending = False
        if len(tiles):
            yield ("wait", f"o{i}")
        if not two:
            yield ("signal", "merge")
            yield ("wait", "merge")
        yield ("read", u)
        if i == 1:
            yield ("signal", f"seen{u & 1}")
        if not two:
            yield ("signal", "merged")
            pending = True


COUNT = {"merge": 2, "merged": 2}


def explore(units, ordered):
    """True if no walk marks a place that the other slot has yet to read; raises on a walk that cannot end."""
    progs = [list(issuer(units)), list(slot(0, units, ordered)), list(slot(1, units, ordered))]
    names = sorted({a[1] for p in progs for a in p if a[0] in ("wait", "signal")} | {"seen0", "seen1"})
    at = {b: k for k, b in enumerate(names)}
    clean, todo, known = True, [((0, 0, 0), (0,) * len(names))], set()  # where each program is, arrivals of each barrier
    waits = [[] for _ in progs]
    for p, prog in enumerate(progs):  # phase parity that each wait asks for: its number among the program's waits there
        n = {}
        for a in prog:
            if a[0] == "wait":
                waits[p].append(n.get(a[1], 0) & 1)
                n[a[1]] = n.get(a[1], 0) + 1
            else:
                waits[p].append(None)
    read_at = [{a[1]: k for k, a in enumerate(prog) if a[0] == "read"} for prog in progs]
    while todo:
        pcs, arr = todo.pop()
        if (pcs, arr) in known:
            continue
        known.add((pcs, arr))
        moved = False

        def passes(bar, parity):
            return ((arr[at[bar]] // COUNT.get(bar, 1)) & 1) != parity
        for p, prog in enumerate(progs):
            if pcs[p] == len(prog):
                continue
            what, x = prog[pcs[p]]
            new = arr
            if what == "wait" and not passes(x, waits[p][pcs[p]]):
                continue
            if what == "seen" and not passes(f"seen{x & 1}", ((x >> 1) & 1) ^ 1):
                continue
            if what == "signal":
                new = tuple(v + (k == at[x]) for k, v in enumerate(arr))
            if what == "mark":
                other = 3 - p
                for v in range(x & 1, x, 2):
                    if pcs[other] <= read_at[other][v]:
                        clean = False
            moved = True
            todo.append((tuple(c + (k == p) for k, c in enumerate(pcs)), new))
        assert moved or all(c == len(g) for c, g in zip(pcs, progs)), f"stuck at {pcs} of {units}"
    return clean


KINDS = [(True, 1), (True, 2), (False, 1), (False, 2), (False, 3)]


@pytest.mark.parametrize("n", [3, 4])
def test_marks_are_read_before_their_place_is_taken_again(n):
    for units in itertools.product(KINDS, repeat=n):
        assert explore(units, True), units


def test_marks_need_the_order():
    """Without slot 0's wait, a unit of one key tile lets it get two units ahead."""
    assert not explore([(True, 1)] * 3, False)
    assert not explore([(True, 2), (True, 1), (False, 1)], False)
