"""A model of the barriers of cached attention over 8-bit caches, run over random interleavings.

Beside the roles of the 16-bit form (two softmax groups, one MMA thread per slot) the warps that turn K's and V's bytes into
operands fetch the scales of later tiles into a ring of stages that no barrier guards: the order of the products has to
prove that a stage's last readers are done. The model checks that, with the kernel's fetch distances; that the rows'
factors and operands are the ones that are meant; and that nothing waits for ever. Rings that are too short have to be
found."""
import random

import pytest

RAW = 3                      # stages of bytes that are fetched ahead
PARTS = {1: 2, 2: 4}         # of a tile, by the query tiles of a group
STAGES = {1: 8, 2: 4}        # of scales
OPERANDS = 2                 # K's tiles, and V's


class Bar:
    def __init__(self, n):
        self.n, self.c, self.phase = n, 0, 0

    def arrive(self):
        self.c += 1
        if self.c == self.n:
            self.c, self.phase = 0, self.phase + 1

    def passed(self, phase):  # a wait on the phase's parity
        return (self.phase & 1) != (phase & 1)


def model(nt, pieces, rnd, ss):
    """One CTA that works through `pieces` (their numbers of key tiles). Raises AssertionError where it goes wrong."""
    total = sum(pieces)
    bars = {"QF": Bar(1), "QE": Bar(2), "OF": Bar(2)}
    for i in range(OPERANDS):
        for n in "KV":
            bars[n + "F", i], bars[n + "E", i] = Bar(1), Bar(nt)
    for i in range(ss):
        bars["SC", i] = Bar(2)
    for s in (0, 1):
        for b in ("SF", "PF", "ML", "OR"):
            bars[b, s] = Bar(1)
    ring = {"K": [None] * OPERANDS, "V": [None] * OPERANDS}
    scales = {"K": [None] * ss, "V": [None] * ss}
    q, factors, scores = [None], [None, None], [None, None]
    pipe, lock, ended = {0: [], 1: []}, [0], []

    def softmax(slot):
        g = 0
        for p, n in enumerate(pieces):
            first = True
            for j in range((slot ^ g) & 1, n * nt, 2):
                tile = (g + j) // nt
                yield ("SC", tile % ss), tile // ss
                yield ("SF", slot), (g + j) >> 1
                assert scores[slot] == ("S", g + j)
                if first:
                    assert factors[p & 1] == p
                first = False
                for _ in range(3):  # it reads them until its weights are there
                    assert scales["K"][tile % ss] == scales["V"][tile % ss] == tile
                    yield
                scores[slot] = ("P", g + j)
                bars["PF", slot].arrive()
                yield
            yield "OF", p
            if nt == 1:
                for b in ("ML", "OR"):
                    bars[b, slot].arrive()
                    yield (b, slot ^ 1), p
            g += n * nt
        ended.append(slot)

    def convert(name):
        parts, fetched, n = PARTS[nt], 0, 0

        def fetch(i):
            tile, part = divmod(i, parts)
            if tile < total and part == 0:
                scales[name][tile % ss] = tile

        for fetched in range(RAW):
            fetch(fetched)
        fetched = RAW
        for p, tiles in enumerate(pieces):
            if name == "V":  # its warps bring the rows
                if p:
                    yield "QE", p - 1
                q[0] = None
                yield
                q[0], factors[p & 1] = p, p
                bars["QF"].arrive()
                yield
            for _ in range(tiles):
                bars["SC", n % ss].arrive()
                yield
                if n >= OPERANDS:
                    yield (name + "E", n % OPERANDS), n // OPERANDS - 1
                ring[name][n % OPERANDS] = None
                for _ in range(parts):
                    yield
                    fetch(fetched)
                    fetched += 1
                ring[name][n % OPERANDS] = n
                bars[name + "F", n % OPERANDS].arrive()
                n += 1
                yield

    def mma(slot):
        st = dict(left=0, kn=0, next=0, piece=-1, more=True)

        def share(first, tiles):  # the slot's first tile of a piece and its number of tiles
            skip = 0 if nt == 2 else (slot ^ first) & 1
            return first + skip, tiles if nt == 2 else (tiles - skip + 1) // 2

        def find():
            while st["left"] == 0:
                if st["piece"] + 1 == len(pieces):
                    st["more"] = False
                    return
                st["piece"] += 1
                st["kn"], st["left"] = share(st["next"], pieces[st["piece"]])
                st["next"] += pieces[st["piece"]]
                yield "QF", st["piece"]
                if st["left"] == 0:
                    pipe[slot].append(("commit", "QE"))
            yield ("KF", st["kn"] % OPERANDS), st["kn"] // OPERANDS

        def issue():
            kn = st["kn"]
            pipe[slot].append(("S", kn, kn * 2 + slot if nt == 2 else kn, st["piece"]))
            pipe[slot].extend([("commit", ("SF", slot)), ("commit", ("KE", kn % OPERANDS))])
            st["kn"] += 3 - nt
            st["left"] -= 1
            if st["left"] == 0:
                pipe[slot].append(("commit", "QE"))

        def batch(products):
            while nt == 2 and lock[0]:
                yield "lock", 0
            lock[0] = 1
            products()
            yield
            lock[0] = 0

        yield from find()
        if st["more"]:
            yield from batch(issue)
        first = done = 0
        for p, tiles in enumerate(pieces):
            kn, left = share(first, tiles)
            first += tiles
            for i in range(left):
                same = st["left"] > 0
                if same:
                    yield from find()
                yield ("VF", kn % OPERANDS), kn // OPERANDS
                yield ("PF", slot), done

                def products():
                    pipe[slot].extend([("PV", kn, kn * 2 + slot if nt == 2 else kn), ("commit", ("VE", kn % OPERANDS))])
                    if i + 1 == left:
                        pipe[slot].append(("commit", "OF"))
                    if same:
                        issue()

                yield from batch(products)
                kn += 3 - nt
                done += 1
                if not same and st["more"]:
                    yield from find()
                    if st["more"]:
                        yield from batch(issue)
            if left == 0:
                if p:
                    yield "OF", p - 1
                pipe[slot].append(("commit", "OF"))

    def execute(slot):
        op = pipe[slot].pop(0)
        if op[0] == "commit":
            bars[op[1]].arrive()
        elif op[0] == "S":
            assert ring["K"][op[1] % OPERANDS] == op[1] and q[0] == op[3]
            scores[slot] = ("S", op[2])
        else:
            assert ring["V"][op[1] % OPERANDS] == op[1] and scores[slot] == ("P", op[2])

    roles = [softmax(0), softmax(1), convert("K"), convert("V"), mma(0), mma(1)]
    waits, alive = [None] * len(roles), set(range(len(roles)))
    weight = [rnd.random() ** 2 + 0.02 for _ in range(8)]  # some roles are slow, some fast
    while alive or pipe[0] or pipe[1]:
        free = lambda w: w is None or (not lock[0] if w[0] == "lock" else bars[w[0]].passed(w[1]))  # noqa: E731
        acts = [("role", r, weight[r]) for r in alive if free(waits[r])]
        acts += [("pipe", s, weight[6 + s]) for s in (0, 1) if pipe[s]]
        assert acts, "everything waits"
        what, i, _ = rnd.choices(acts, [a[2] for a in acts])[0]
        if what == "pipe":
            execute(i)
            continue
        try:
            waits[i] = next(roles[i])
        except StopIteration:
            alive.discard(i)
    assert sorted(ended) == [0, 1]


def runs(count, nt, ss):
    bad = 0
    for seed in range(count):
        rnd = random.Random(seed)
        pieces = [rnd.choice([1, 1, 2, 3, 5, rnd.randint(1, 12)]) for _ in range(rnd.randint(1, 8))]
        try:
            model(nt, pieces, rnd, ss)
        except AssertionError:
            bad += 1
    return bad


@pytest.mark.parametrize("nt", [1, 2])
def test_stages_of_scales_need_no_barrier(nt):
    assert runs(500, nt, STAGES[nt]) == 0


def test_six_stages_would_do_for_one_query_tile():
    assert runs(500, 1, 6) == 0


@pytest.mark.parametrize("nt,ss", [(1, 4), (1, 2), (2, 3), (2, 2)])
def test_shorter_rings_are_found(nt, ss):
    assert runs(300, nt, ss) > 0
