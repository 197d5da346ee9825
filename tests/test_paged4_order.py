"""Walks over the units of the 4-bit attention of few rows, on the CPU.

A CTA's warps meet at barriers whose number hangs on its units, and units hang
on row_start and kv_len in device memory. A caller may break the rules and
change them under the kernel: then the output means nothing, but every warp has to
meet the others, every walk has to end, and no unit may lie outside the batch
or the block table. The walk (take and next) is restated here with lengths that
change between two looks at a sequence."""
import itertools

TILE, CELLS, H = 128, 2, 2


class Walk:
    """`look` gives (rows, tokens) of a sequence as they are when it is looked at."""

    def __init__(self, look, batch, group, unit, cap, cta, ctas):
        self.look, self.batch, self.group, self.unit, self.cap = look, batch, group, unit, cap
        seqs = [look(b) for b in range(batch)]
        total = H * sum(self.tiles(s, q) + CELLS for s in seqs for q in range(self.count(s)))
        self.per = max(CELLS + 1, -(-total // ctas))
        want = cta * self.per
        self.any = want < total
        self.left = min(self.per, total - want)
        for self.b, self.s in enumerate(seqs):
            for self.hk, self.qt in itertools.product(range(H), range(self.count(self.s))):
                n = self.tiles(self.s, self.qt) + CELLS
                if want < n:
                    self.cell = want
                    return
                want -= n

    def count(self, s):
        return -(-s[0] * self.group // self.unit)

    def tiles(self, s, q):
        token = (min(s[0] * self.group, (q + 1) * self.unit) - 1) // self.group
        seen = min(self.cap, s[1] - s[0] + token + 1)
        return 1 if seen <= 0 else -(-seen // TILE)

    def take(self):
        full = self.tiles(self.s, self.qt)
        end = min(full + CELLS, self.cell + self.left)
        t0 = max(0, self.cell - CELLS)
        n = max(0, end - CELLS) - t0
        self.left -= end - self.cell
        self.cell = 0
        rows = min(self.unit, self.s[0] * self.group - self.qt * self.unit)
        pieces = 1 + -(-(full - n) // self.per) if t0 == 0 and 0 < n < full else 0
        return dict(b=self.b, hk=self.hk, rows=rows, t0=t0, n=n, last=self.left <= CELLS, pieces=pieces)

    def next(self):
        self.qt += 1
        if self.qt < self.count(self.s):
            return
        self.qt, self.hk = 0, self.hk + 1
        if self.hk < H:
            return
        self.hk, self.b, self.s = 0, self.b + 1, (0, 0)
        while self.b < self.batch:
            self.s = self.look(self.b)
            if self.s[0]:
                break
            self.b += 1
        self.any = self.b < self.batch

    def units(self):
        while self.any:
            w = self.take()
            yield w
            if w["last"]:
                return
            self.next()


SEQS = [(1, 700), (1, 40), (0, 9), (2, 300), (1, 1), (1, 900), (1, 128)]
NEW = [(1, 30), (1, 900), (1, 60), (2, 10), (1, 2000), (1, 3), (0, 0)]


def changing(old, new, at):
    """Lengths that become the new ones behind the at-th look."""
    looks = itertools.count()
    return lambda b: (new if next(looks) >= at else old)[b]


def walks(cta, ctas, old=SEQS, new=NEW):
    for at in range(3 * len(old)):
        yield list(Walk(changing(old, new, at), len(old), 4, 8, 1024, cta, ctas).units())


def meets(units):
    return sum(1 + (w["rows"] > 0) for w in units)


def test_lengths_as_they_were_cover_every_tile_once():
    for ctas in (1, 3, 8, 40):
        got = [(w["b"], w["hk"], t) for c in range(ctas) for w in Walk(lambda b: SEQS[b], len(SEQS), 4, 8, 1024, c, ctas).units()
               for t in range(w["t0"], w["t0"] + w["n"])]
        want = [(b, h, t) for b, (r, n) in enumerate(SEQS) if r for h in range(H) for t in range(-(-n // TILE))]
        assert sorted(got) == want


def test_warps_that_look_by_themselves_might_not_meet():
    """Why one thread looks for all of them."""
    assert any(len({meets(u) for u in walks(c, ctas)}) > 1 for ctas in (1, 3) for c in range(ctas))


def test_every_walk_ends_inside_the_batch():
    for old, new in itertools.permutations([SEQS, NEW, [(0, 0)] * 7, [(2, 5000)] * 7], 2):
        for ctas in (1, 3, 8):
            for c in range(ctas):
                for units in walks(c, ctas, old, new):
                    assert len(units) <= 4 * H * len(old)
                    for w in units:
                        assert w["b"] < len(old) and 1 <= w["rows"] <= 8 and w["n"] >= 0
                        assert 0 <= w["t0"] and w["t0"] + w["n"] <= 1024 // TILE


def test_a_cut_may_count_pieces_that_nobody_has():
    """Why the join looks at no more pieces than CTAs that follow."""
    worst = max(w["pieces"] - (ctas - c) for old, new in ((SEQS, [(2, 5000)] * 7), ([(1, 5)] * 7, [(1, 1000)] * 7)) for ctas in (3, 8)
                for c in range(ctas) for units in walks(c, ctas, old, new) for w in units)
    assert worst > 0
