"""The barrier protocol of attn_wide_kernel on the host: its roles as
coroutines over counted phases, run under schedules that hold one role back as
long as another can move.

A wait names the number of the phase that it is for; the hardware has the phase's
parity only.  That is enough as long as the barrier is in that phase or has just
left it.  Two phases on, the wait blocks for a phase that may never end; one phase
short, it passes early.  ``run`` raises Aliased where a wait meets such a barrier, and
Stuck where nothing can move before all roles have ended.

``CLEAN_BY_ITEM`` and ``Q_BY_COPIER`` are the two points that keep the helper warps
(Q rows, scan of masked values) from being overtaken: v_clean has a barrier per
item parity, and only the warp that copies Q waits for its place to be free.
Without them (one v_clean for all items behind a v_next barrier, both helper warps
waiting for q_empty) the model shows what may go wrong."""
import random
import re

STAGES = {128: 2, 64: 4}


class Aliased(Exception):
    pass


class Stuck(Exception):
    pass


def counts(source):
    """Arrivals a phase by barrier, from the kernel's mbar_init calls."""
    return {m.group(1): int(m.group(2)) for m in re.finditer(r"mbar_init\(&s\.(\w+)[^,]*, (\d+)\)", source)}


class Bar:
    def __init__(self, name, count):
        self.name, self.count, self.left, self.done = name, count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1

    def over(self, phase):
        """Whether `phase` has ended, as the parity tells it; the barrier has to be in it or in the next one."""
        if self.done not in (phase, phase + 1):
            raise Aliased(f"{self.name}: wait for phase {phase} meets phase {self.done}")
        return self.done == phase + 1


class Model:
    """items: dicts n, m0, n0, n1, twin (as ApItem).  Coroutines yield (barrier, phase) to wait for, or None."""

    def __init__(self, count, items, stages, clean_by_item=True, q_by_copier=True):
        b = lambda name, key=None: Bar(name, count[key or name.split("[")[0]])
        self.items, self.stages, self.by_item, self.by_copier = items, stages, clean_by_item, q_by_copier
        self.kv_full, self.kv_empty = ([b(f"{n}[{i}]") for i in range(stages)] for n in ("kv_full", "kv_empty"))
        self.s_full, self.p_full, self.o_done, self.sched_full, self.sched_empty = (
            [b(f"{n}[{i}]") for i in range(2)] for n in ("s_full", "p_full", "o_done", "sched_full", "sched_empty"))
        self.q_full, self.q_empty = b("q_full"), b("q_empty")
        self.v_posted = [[b(f"v_posted[{p}][{z}]") for z in range(3)] for p in range(2)]
        self.v_clean = [[b(f"v_clean[{p}][{z}]") for z in range(3)] for p in range(2)]
        self.v_next = Bar("v_next", 1)
        self.v_pos, self.pipe, self.copies, self.q_copies, self.posted = {}, [], [], [], {}
        self.roles = {"copy": self.tma(), "mma": self.mma(), "help2": self.helper(2), "help3": self.helper(3)}
        for h in range(2):
            for w in range(4):
                self.roles[f"soft{h}{w}"] = self.soft(h)
        # what runs beside the warps: the tensor pipe, the tile copies, the copies of Q
        self.beside = {"pipe": self.pipe, "tiles": self.copies, "q": self.q_copies}

    def item(self, i):
        return self.posted[i]

    def tma(self):
        pos = 0
        for i, it in enumerate(self.items + [None]):
            if i >= 2:
                yield self.sched_empty[i & 1], (i >> 1) - 1
            self.posted[i] = it
            self.sched_full[i & 1].arrive()
            if it is None:
                return
            n, ahead = it["n"], 2 if it["twin"] else 1
            for q in range(n + ahead):
                if q >= n and q < ahead:
                    continue
                slot = pos % self.stages
                if pos >= self.stages:
                    yield self.kv_empty[slot], pos // self.stages - 1
                z = q - ahead - it["m0"]
                if z >= 0:
                    self.v_pos[i & 1, z] = pos
                    self.v_posted[i & 1][z].arrive()
                self.copies.append(self.kv_full[slot].arrive)
                pos += 1
                yield None

    def mma(self):
        pos, i = 0, 0
        nps, clean = [0, 0], {}
        issue = self.pipe.append
        while True:
            yield self.sched_full[i & 1], i >> 1
            it = self.item(i)
            if it is None:
                return
            n, m0, n0, n1, twin = (it[k] for k in ("n", "m0", "n0", "n1", "twin"))
            ahead = 2 if twin else 1
            yield self.q_full, i
            for j in range(min(ahead, n)):
                yield self.kv_full[pos % self.stages], pos // self.stages
                for h in ([j] if twin else [0, 1] if n1 > 0 else [0]):
                    issue(self.s_full[h].arrive)
                issue(self.kv_empty[pos % self.stages].arrive)
                if j + 1 == n:
                    issue(self.q_empty.arrive)
                pos += 1
                yield None
            for j in range(n):
                slot = pos % self.stages
                yield self.kv_full[slot], pos // self.stages
                if j >= m0:
                    key = (i & 1 if self.by_item else 0, j - m0)
                    yield self.v_clean[key[0]][key[1]], clean.get(key, 0)
                    clean[key] = clean.get(key, 0) + 1
                if j + 1 == n:
                    self.v_next.arrive()
                for h, nh in enumerate((n0, n1)):
                    if (j & 1) == h if twin else j < nh:
                        yield self.p_full[h], nps[h]
                        nps[h] += 1
                        issue((self.s_full[h] if (j + 2 < n if twin else j + 1 < nh) else self.o_done[h]).arrive)
                        if twin or h or n1 == 0:
                            issue(self.kv_empty[slot].arrive)
                            if j + ahead + 1 == n:
                                issue(self.q_empty.arrive)
                        yield None
                pos += 1
            self.sched_empty[i & 1].arrive()
            i += 1

    def soft(self, h):
        ns = ni = i = 0
        while True:
            yield self.sched_full[i & 1], i >> 1
            it = self.item(i)
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
            it = self.item(i)
            if it is None:
                return
            if i > 0 and (warp == 2 or not self.by_copier):
                yield self.q_empty, i - 1
            if warp == 2:
                self.q_copies.append(self.q_full.arrive)
                yield None
            if i > 0 and not self.by_item:
                yield self.v_next, i - 1
            for j in range(it["m0"], it["n"]):
                z = j - it["m0"]
                key = (i & 1, z)
                yield self.v_posted[i & 1][z], uses.get(key, 0)
                uses[key] = uses.get(key, 0) + 1
                pos = self.v_pos[key]
                yield self.kv_full[pos % self.stages], pos // self.stages
                self.v_clean[i & 1 if self.by_item else 0][z].arrive()
                yield None
            self.sched_empty[i & 1].arrive()
            i += 1


def run(model, pick):
    """Moves the roles one step at a time in the order of `pick`(names that can move) until all warps have ended."""
    live, wants = dict(model.roles), dict.fromkeys(model.roles)
    while live:
        ready = [n for n in live if wants[n] is None or wants[n][0].over(wants[n][1])] + [n for n, q in model.beside.items() if q]
        if not ready:
            raise Stuck({n: (w[0].name, w[1]) for n, w in wants.items() if n in live and w})
        n = pick(ready)
        if n in model.beside:
            model.beside[n].pop(0)()
            continue
        try:
            wants[n] = next(live[n])
        except StopIteration:
            del live[n]


def schedules(seed, roles):
    """Each role in turn as the slowest, each as the fastest, and random ones."""
    for slow in roles:
        yield lambda ready, s=slow: next((n for n in ready if n != s), s)
        yield lambda ready, s=slow: s if s in ready else ready[0]
        rng = random.Random(f"{seed} {slow}")
        yield lambda ready, s=slow, r=rng: r.choice([n for n in ready if n != s] or [s])
    rng = random.Random(seed)
    for _ in range(8):
        yield lambda ready, r=rng: r.choice(ready)


def random_items(rng, n, longest):
    """Items as the kernel makes them: row tiles together (n0 <= n1 = n, or n1 = 0) or twins; up to three masked tiles."""
    out = []
    for _ in range(n):
        t = rng.randint(1, longest)
        masked = rng.randint(0, min(3, t))
        kind = rng.choice(["pair", "single", "twin"])
        n0, n1 = {"pair": (max(1, t - rng.randint(0, 1)), t), "single": (t, 0), "twin": ((t + 1) // 2, t // 2)}[kind]
        out.append(dict(n=t, m0=t - masked + (rng.randint(0, 2) if not masked else 0), n0=n0, n1=n1, twin=kind == "twin"))
    return out
