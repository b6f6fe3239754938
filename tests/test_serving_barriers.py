"""A model of the cached-attention kernel's barriers, run over random interleavings.

The tensor-core kernel's roles (two softmax groups, the Q loader, the TMA warps of K and V, one MMA thread per slot) meet
on mbarriers that are waited on by parity. The model has the same roles, arrival counts, stage counts and order of waits
and commits, an in-order tensor pipe per thread and loads that land in any order; it checks that every MMA finds the
operands it means, that every result is read whole, and that nothing waits for ever. Two mistakes, planted in the model,
have to be found: an arrival for a piece without tiles that does not wait for the piece before, and an odd number of
stages that the two slots share."""
import random

import pytest


class Bar:
    def __init__(self, n):
        self.n, self.c, self.phase = n, 0, 0

    def arrive(self):
        self.c += 1
        if self.c == self.n:
            self.c, self.phase = 0, self.phase + 1

    def passed(self, phase):  # a wait on the phase's parity
        return (self.phase & 1) != (phase & 1)


def model(nt, pieces, rnd, stages, waits_before_empty=True):
    """One CTA that works through `pieces` (their numbers of key tiles). Raises AssertionError where it goes wrong."""
    ks, vs = stages
    bars = {"QF": Bar(1), "QE": Bar(2), "OF": Bar(2)}
    for i in range(ks):
        bars["KF", i], bars["KE", i] = Bar(1), Bar(nt)
    for i in range(vs):
        bars["VF", i], bars["VE", i] = Bar(1), Bar(nt)
    for s in (0, 1):
        for b in ("SF", "PF", "ML", "OR"):
            bars[b, s] = Bar(1)
    k, v, q, scores, out = [None] * ks, [None] * vs, [None], [None, None], [None, None]
    pipe, landing, lock, ended = {0: [], 1: []}, [], [0], []

    def softmax(slot):
        g = 0
        for p, n in enumerate(pieces):
            for j in range((slot ^ g) & 1, n * nt, 2):
                yield ("SF", slot), (g + j) >> 1
                assert scores[slot] == ("S", g + j)
                yield
                scores[slot] = ("P", g + j)
                bars["PF", slot].arrive()
                yield
            yield "OF", p
            if nt == 2:
                assert out[slot] == (p, n)
            else:  # the slots' accumulators come together
                bars["ML", slot].arrive()
                yield ("ML", slot ^ 1), p
                share = [sum((g + t) & 1 == s for t in range(n)) for s in (0, 1)]
                yield
                assert all(out[s] == (p, share[s]) for s in (0, 1) if share[s])
                bars["OR", slot].arrive()
                yield ("OR", slot ^ 1), p
            g += n * nt
        ended.append(slot)

    def load_q():
        for p in range(len(pieces)):
            if p:
                yield "QE", p - 1
            q[0] = None
            yield
            q[0] = p
            bars["QF"].arrive()

    def tma(name, n_stages, ring):
        n = 0
        for tiles in pieces:
            for _ in range(tiles):
                if n >= n_stages:
                    yield (name + "E", n % n_stages), n // n_stages - 1
                ring[n % n_stages] = None
                landing.append((name, n % n_stages, n, ring))
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
                tiles = pieces[st["piece"]]
                st["kn"], st["left"] = share(st["next"], tiles)
                st["next"] += tiles
                yield "QF", st["piece"]
                if st["left"] == 0:
                    pipe[slot].append(("commit", "QE"))
            yield ("KF", st["kn"] % ks), st["kn"] // ks

        def issue():
            kn = st["kn"]
            pipe[slot].append(("S", kn, kn * 2 + slot if nt == 2 else kn, st["piece"]))
            pipe[slot].extend([("commit", ("SF", slot)), ("commit", ("KE", kn % ks))])
            st["kn"] += 3 - nt
            st["left"] -= 1
            if st["left"] == 0:
                pipe[slot].append(("commit", "QE"))

        def take():
            while nt == 2 and lock[0]:
                yield "lock", 0
            lock[0] = 1

        def batch():
            yield from take()
            issue()
            yield
            lock[0] = 0

        yield from find()
        if st["more"]:
            yield from batch()
        first = done = 0
        for p, tiles in enumerate(pieces):
            kn, left = share(first, tiles)
            first += tiles
            for i in range(left):
                same = st["left"] > 0
                if same:
                    yield from find()
                yield ("VF", kn % vs), kn // vs
                yield ("PF", slot), done
                yield from take()
                pipe[slot].extend([("PV", kn, kn * 2 + slot if nt == 2 else kn, p, i), ("commit", ("VE", kn % vs))])
                yield
                if i + 1 == left:
                    pipe[slot].append(("commit", "OF"))
                if same:
                    issue()
                lock[0] = 0
                kn += 3 - nt
                done += 1
                if not same and st["more"]:
                    yield from find()
                    if st["more"]:
                        yield from batch()
            if left == 0:
                if waits_before_empty and p:
                    yield "OF", p - 1
                pipe[slot].append(("commit", "OF"))

    def execute(slot):
        op = pipe[slot].pop(0)
        if op[0] == "commit":
            bars[op[1]].arrive()
        elif op[0] == "S":
            assert k[op[1] % ks] == op[1] and q[0] == op[3]
            scores[slot] = ("S", op[2])
        else:
            assert v[op[1] % vs] == op[1] and scores[slot] == ("P", op[2])
            out[slot] = (op[3], 1 if op[4] == 0 else out[slot][1] + 1)

    roles = [softmax(0), softmax(1), load_q(), tma("K", ks, k), tma("V", vs, v), mma(0), mma(1)]
    waits, alive = [None] * len(roles), set(range(len(roles)))
    weight = [rnd.random() ** 2 + 0.02 for _ in range(10)]  # some roles are slow, some fast
    while alive or pipe[0] or pipe[1] or landing:
        free = lambda w: w is None or (not lock[0] if w[0] == "lock" else bars[w[0]].passed(w[1]))  # noqa: E731
        acts = [("role", r, weight[r]) for r in alive if free(waits[r])]
        acts += [("pipe", s, weight[7 + s]) for s in (0, 1) if pipe[s]]
        if landing:
            acts.append(("land", rnd.randrange(len(landing)), weight[9]))
        assert acts, "everything waits"
        what, i, _ = rnd.choices(acts, [a[2] for a in acts])[0]
        if what == "pipe":
            execute(i)
        elif what == "land":
            name, stage, n, ring = landing.pop(i)
            ring[stage] = n
            bars[name + "F", stage].arrive()
        else:
            try:
                waits[i] = next(roles[i])
            except StopIteration:
                alive.discard(i)
    assert sorted(ended) == [0, 1]


STAGES = {1: (2, 4), 2: (3, 2)}  # K and V stages of the kernel


def runs(count, **kw):
    bad = 0
    for seed in range(count):
        rnd = random.Random(seed)
        nt = kw.get("nt") or rnd.choice([1, 2])
        pieces = [rnd.choice([1, 1, 2, 3, 4, 7, 12]) for _ in range(rnd.randint(1, 6))]
        try:
            model(nt, pieces, rnd, kw.get("stages") or STAGES[nt], kw.get("waits_before_empty", True))
        except AssertionError:
            bad += 1
    return bad


def test_every_interleaving_is_right():
    assert runs(1500) == 0


@pytest.mark.parametrize("mistake", [dict(nt=1, waits_before_empty=False), dict(nt=1, stages=(3, 3))])
def test_planted_mistakes_are_found(mistake):
    assert runs(1500, **mistake) > 0
