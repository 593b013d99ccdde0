"""The barrier protocols of the latent attention's kernels on the host, as
``attn_barriers`` runs that of the attention: lat_tree_kernel, and attn_wide_kernel with
its ring of pieces.

``split_done`` False gives pv_done one barrier for all tiles, as a softmax warp that
waits for the last two of an item would meet it: the model shows why there are two."""
import random

from attn_barriers import Aliased, Bar


class Overwritten(Exception):
    pass


class Tree:
    """items: dicts n (tiles) and m0 (masked from there on); moves(half, tile) says whether the maximum moves there."""

    def __init__(self, count, items, halves, parts, moves, split_done=True):
        b = lambda name: Bar(name, count[name.split("[")[0]])  # noqa: E731
        self.items, self.nh, self.nr, self.moves, self.split = items, halves, parts, moves, split_done
        self.kv_full, self.kv_empty = ([b(f"{n}[{i}]") for i in range(halves)] for n in ("kv_full", "kv_empty"))
        self.part_of = [None] * parts                 # the tile whose key part, or P, a place holds
        self.s_full, self.p_full, self.pv_done, self.sched_full, self.sched_empty = (
            [b(f"{n}[{i}]") for i in range(2)] for n in ("s_full", "p_full", "pv_done", "sched_full", "sched_empty"))
        self.q_full, self.q_empty = b("q_full"), b("q_empty")
        self.votes = [Bar(f"vote{h}", 4) for h in range(2)]
        self.scores, self.values, self.copies, self.q_copies, self.posted = [], [], [], [], {}
        self.roles = {"copy": self.tma(), "s": self.s(), "o": self.o(), "q": self.q()}
        for h in range(2):
            for w in range(4):
                self.roles[f"soft{h}{w}"] = self.soft(h)
        # what runs beside the warps: the products of each issuer, in its order, the copies of tiles and of Q
        self.beside = {"scores": self.scores, "values": self.values, "tiles": self.copies, "qcopies": self.q_copies}

    def tma(self):
        pos = tiles = 0
        for i, it in enumerate(self.items + [None]):
            if i >= 2:
                yield self.sched_empty[i & 1], (i >> 1) - 1
            self.posted[i] = it
            self.sched_full[i & 1].arrive()
            if it is None:
                return
            for _ in range(it["n"]):
                for z in range(2):
                    if pos >= self.nh:
                        yield self.kv_empty[pos % self.nh], pos // self.nh - 1
                    if z:                             # the key part comes with the second half: no barrier of its own
                        if self.part_of[tiles % self.nr] is not None:
                            raise Overwritten(f"tile {tiles} over tile {self.part_of[tiles % self.nr]}")
                        self.part_of[tiles % self.nr] = tiles
                    self.copies.append(self.kv_full[pos % self.nh].arrive)
                    pos += 1
                    yield None
                tiles += 1

    def free(self, tile):
        self.part_of[tile % self.nr] = None

    def s(self):
        pos = t = i = 0
        while True:
            yield self.sched_full[i & 1], i >> 1
            it = self.posted[i]
            if it is None:
                return
            yield self.q_full, i
            for j in range(it["n"]):
                if t >= 2:
                    yield self.p_full[t & 1], (t >> 1) - 1
                for _ in range(2):
                    yield self.kv_full[pos % self.nh], pos // self.nh
                    pos += 1
                self.scores.append(self.s_full[t & 1].arrive)
                if j + 1 == it["n"]:
                    self.scores.append(self.q_empty.arrive)
                t += 1
                yield None
            self.sched_empty[i & 1].arrive()
            i += 1

    def o(self):
        t = i = 0
        while True:
            yield self.sched_full[i & 1], i >> 1
            it = self.posted[i]
            if it is None:
                return
            for _ in range(it["n"]):
                yield self.p_full[t & 1], t >> 1
                self.values.append(self.kv_empty[2 * t % self.nh].arrive)
                self.values.append(lambda t=t: self.free(t))
                self.values.append(self.kv_empty[(2 * t + 1) % self.nh].arrive)
                self.values.append(self.pv_done[t & 1 if self.split else 0].arrive)
                t += 1
                yield None
            self.sched_empty[i & 1].arrive()
            i += 1

    def q(self):
        i = 0
        while True:
            yield self.sched_full[i & 1], i >> 1
            if self.posted[i] is None:
                return
            if i > 0:
                yield self.q_empty, i - 1
            self.q_copies.append(self.q_full.arrive)
            yield None
            self.sched_empty[i & 1].arrive()
            i += 1

    def done(self, t):
        return (self.pv_done[t & 1], t >> 1) if self.split else (self.pv_done[0], t)

    def soft(self, h):
        ns = nv = i = 0

        def vote():
            nonlocal nv
            self.votes[h].arrive()
            nv += 1
            return self.votes[h], nv - 1
        while True:
            yield self.sched_full[i & 1], i >> 1
            yield vote()
            it = self.posted[i]
            if it is None:
                return
            for j in range(it["n"]):
                yield self.s_full[ns & 1], ns >> 1
                if j >= it["m0"]:                     # the scan
                    for pos in (2 * ns, 2 * ns + 1):
                        yield self.kv_full[pos % self.nh], pos // self.nh
                yield vote()
                if self.moves(h, ns):
                    yield vote()
                    if j > 0:
                        yield self.done(ns - 1)
                self.p_full[ns & 1].arrive()
                ns += 1
                yield None
            if ns > 1:
                yield self.done(ns - 2)
            yield self.done(ns - 1)
            yield vote()
            self.sched_empty[i & 1].arrive()
            i += 1


class Prompt:
    """attn_wide_kernel's expanded form: items as in ``attn_barriers``, a ring of pieces (2 of a value tile, 3 of a key tile)."""

    def __init__(self, count, items, stages=7):
        b = lambda name: Bar(name, count[name.split("[")[0]])  # noqa: E731
        self.items, self.stages = items, stages
        self.kv_full, self.kv_empty = [b(f"kv_full[{i}]") for i in range(4)], [b(f"kv_empty[{i}]") for i in range(stages)]
        self.s_full, self.p_full, self.o_done, self.sched_full, self.sched_empty = (
            [b(f"{n}[{i}]") for i in range(2)] for n in ("s_full", "p_full", "o_done", "sched_full", "sched_empty"))
        self.q_full, self.q_empty = b("q_full"), b("q_empty")
        self.v_posted = [[b(f"v_posted[{p}][{z}]") for z in range(3)] for p in range(2)]
        self.v_clean = [[b(f"v_clean[{p}][{z}]") for z in range(3)] for p in range(2)]
        self.v_tile, self.seen, self.pipe, self.copies, self.q_copies, self.posted = {}, {}, [], [], [], {}
        self.roles = {"copy": self.tma(), "mma": self.mma(), "help2": self.helper(2), "help3": self.helper(3)}
        for h in range(2):
            for w in range(4):
                self.roles[f"soft{h}{w}"] = self.soft(h)
        self.beside = {"pipe": self.pipe, "tiles": self.copies, "q": self.q_copies}

    def tma(self):
        pos = tiles = 0
        for i, it in enumerate(self.items + [None]):
            if i >= 2:
                yield self.sched_empty[i & 1], (i >> 1) - 1
            self.posted[i] = it
            self.sched_full[i & 1].arrive()
            if it is None:
                return
            n, ahead = it["n"], 2 if it["twin"] else 1
            for q in range(n + ahead):
                for pieces in ([2] if q >= ahead else []) + ([3] if q < n else []):
                    for z in range(pieces):
                        if pos + z >= self.stages:
                            yield self.kv_empty[(pos + z) % self.stages], (pos + z) // self.stages - 1
                        if z == (1 if pieces == 2 else 0):       # armed: the copies' bytes are what completes it
                            self.armed(tiles)
                    z = q - ahead - it["m0"]
                    if pieces == 2 and z >= 0:
                        self.v_tile[i & 1, z] = tiles
                        self.v_posted[i & 1][z].arrive()
                    self.copies.append(self.kv_full[tiles & 3].arrive)
                    pos += pieces
                    tiles += 1
                    yield None

    def armed(self, t):
        """A barrier is armed for a tile when nobody waits for its last phase any more."""
        if self.kv_full[t & 3].done != t >> 2 or self.seen.get(t - 4, 0) != (t - 4 >= 0):
            raise Aliased(f"kv_full[{t & 3}] armed for tile {t}")

    def full(self, t):
        return self.kv_full[t & 3], t >> 2

    def mma(self):
        issue = self.pipe.append
        pos, tiles, i, nps, clean = 0, 0, 0, [0, 0], {}

        def scores(h, at, last, q_last):
            if last:
                for z in range(3):
                    issue(self.kv_empty[(at + z) % self.stages].arrive)
            issue(self.s_full[h].arrive)
            if q_last:
                issue(self.q_empty.arrive)
        while True:
            yield self.sched_full[i & 1], i >> 1
            it = self.posted[i]
            if it is None:
                return
            n, m0, n0, n1, twin = (it[k] for k in ("n", "m0", "n0", "n1", "twin"))
            ahead = 2 if twin else 1
            yield self.q_full, i
            for j in range(min(ahead, n)):
                yield self.full(tiles)
                self.seen[tiles] = 1
                tiles += 1
                if twin:
                    scores(j, pos, True, j + 1 == n)
                else:
                    scores(0, pos, n1 == 0, j + 1 == n and n1 == 0)
                    if n1 > 0:
                        scores(1, pos, True, j + 1 == n)
                pos += 3
                yield None
            for j in range(n):
                at = pos
                yield self.full(tiles)
                self.seen[tiles] = 1
                tiles += 1
                if j >= m0:
                    key = (i & 1, j - m0)
                    yield self.v_clean[key[0]][key[1]], clean.get(key, 0)
                    clean[key] = clean.get(key, 0) + 1
                pos += 2
                keys = False
                for h, nh in enumerate((n0, n1)):
                    if (j & 1) == h if twin else j < nh:
                        more, tail = (j + 2 < n if twin else j + 1 < nh), twin or h or n1 == 0
                        yield self.p_full[h], nps[h]
                        nps[h] += 1
                        if tail:
                            issue(self.kv_empty[at % self.stages].arrive)
                            issue(self.kv_empty[(at + 1) % self.stages].arrive)
                        if not more:
                            issue(self.o_done[h].arrive)
                        if more and not keys:
                            yield self.full(tiles)
                            self.seen[tiles] = 1
                            keys = True
                        if more:
                            scores(h, pos, tail, tail and j + ahead + 1 == n)
                        yield None
                if j + ahead < n:
                    pos += 3
                    tiles += 1
            self.sched_empty[i & 1].arrive()
            i += 1

    def soft(self, h):
        ns = ni = i = 0
        while True:
            yield self.sched_full[i & 1], i >> 1
            it = self.posted[i]
            if it is None:
                return
            nt = it["n1"] if h else it["n0"]
            for _ in range(nt):
                yield self.s_full[h], ns
                ns += 1
                self.p_full[h].arrive()
                yield None
            if nt:
                yield self.o_done[h], ni
                ni += 1
            self.sched_empty[i & 1].arrive()
            i += 1

    def helper(self, warp):
        uses, i = {}, 0
        while True:
            yield self.sched_full[i & 1], i >> 1
            it = self.posted[i]
            if it is None:
                return
            if warp == 2:
                if i > 0:
                    yield self.q_empty, i - 1
                self.q_copies.append(self.q_full.arrive)
                yield None
            for j in range(it["m0"], it["n"]):
                z = j - it["m0"]
                key = (i & 1, z)
                yield self.v_posted[i & 1][z], uses.get(key, 0)
                uses[key] = uses.get(key, 0) + 1
                yield self.full(self.v_tile[key])
                self.v_clean[i & 1][z].arrive()
                yield None
            self.sched_empty[i & 1].arrive()
            i += 1


def random_tree_items(rng, n, longest):
    out = []
    for _ in range(n):
        t = rng.randint(1, longest)
        out.append(dict(n=t, m0=t - rng.randint(0, min(2, t))))
    return out


def moves_by(seed, often):
    """The same answer for the four warps of a half."""
    return lambda h, t: random.Random(f"{seed} {h} {t}").random() < often
