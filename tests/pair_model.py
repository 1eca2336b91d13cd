"""A model of the per-channel product's mbarrier protocol, for randomized
checking: the roles of both blocks of one pair of `pair_kernel`, on the
scheduler of pipeline_model.

One MMA reads both blocks' operands, so `ready` and `dempty` are the first
block's and count both, while `consumed` and `dfull` are committed to both.
The model adds to its base: an expect of two copies, and the accumulators,
which are being written from a chunk's first MMA until its last one is done.

Only tests use this module; it shares nothing with the kernel source beyond
restating its waits and arrivals."""
import random

import pipeline_model as pm

KA = 4          # operand A buffers
ND = 2          # accumulators
CHUNK = 8       # K steps of an accumulator

# token slots, units of a K step, word slots
CONFIGS = {64: dict(kx=4, per=1, nw=8), 96: dict(kx=4, per=1, nw=8), 128: dict(kx=4, per=1, nw=8),
           192: dict(kx=8, per=2, nw=8)}


class _Uneven(random.Random):
    """Chooses as random.Random, but seldom a role of this run's slow ones."""

    def __init__(self, seed, names):
        super().__init__(seed)
        self.slow = {n for n in names if self.random() < 0.25}

    def choice(self, options):
        quick = [o for o in options if o[0] != "a" or o[1]["name"] not in self.slow]
        return super().choice(quick if quick and self.random() < 0.995 else options)


class _Pair(pm._Sim):
    def _step(self, a):
        a["wait"] = None
        try:
            act = next(a["gen"])
        except StopIteration:
            a["done"] = True
            return
        if act[0] == "wait":
            a["wait"] = (act[1], act[2])
        elif act[0] == "arrive":
            self.bars[act[1]].arrive(self)
        elif act[0] == "expect":         # (name, copies)
            bar = self.bars[act[1]]
            bar.tx += act[2]
            bar.arrive(self)
        elif act[0] == "copy":           # (name, resource)
            self._begin(act[2], "w", a["name"])

            def land(name=act[1], res=act[2]):
                self._end(res, "w")
                self.bars[name].tx -= 1
                self.bars[name]._check()
            self.inflight.append(land)
        elif act[0] == "mma":            # (reads, accumulators, first of its chunk)
            for r in act[1]:
                self._begin(r, "r", a["name"])
            if act[3]:
                for d in act[2]:
                    self._begin(d, "w", a["name"])
            rec = {"done": False}
            order = self.mmas["pair"]
            order.append(rec)

            def finish(rec=rec, reads=act[1]):
                for r in reads:
                    self._end(r, "r")
                rec["done"] = True
            rec["finish"] = finish
            if len(order) == 1 or order[-2]["done"]:
                self.inflight.append(self._next_mma)
        elif act[0] == "written":        # the chunk's accumulators, when its MMAs are done
            self.commits.append(([m for m in self.mmas["pair"] if not m["done"]], tuple(act[1])))
            self._flush_commits()
        elif act[0] == "commit":
            self.commits.append(([m for m in self.mmas["pair"] if not m["done"]], act[1]))
            self._flush_commits()
        else:
            self._begin(act[1], act[0][0], a["name"])
            self._end(act[1], act[0][0])

    def _next_mma(self):                 # MMAs of one thread complete in order
        order = self.mmas["pair"]
        rec = next(m for m in order if not m["done"])
        rec["finish"]()
        if any(not m["done"] for m in order):
            self.inflight.append(self._next_mma)

    def _flush_commits(self):
        keep = []
        for prior, what in self.commits:
            if not all(m["done"] for m in prior):
                keep.append((prior, what))
            elif isinstance(what, tuple):
                for d in what:
                    self._end(d, "w")
            else:
                self.bars[what].arrive(self)
        self.commits = keep


def _roles(c, segments):
    """segments: the K steps of each of the pair's segments."""
    kx, per, nw = c["kx"], c["per"], c["nw"]
    steps = sum(segments)

    def words(b):
        for j in range(steps):
            yield ("wait", f"wempty{b}.{j % nw}", ((j // nw) & 1) ^ 1)
            yield ("expect", f"wfull{b}.{j % nw}", 1)
            yield ("copy", f"wfull{b}.{j % nw}", f"W{b}.{j % nw}")
        for j in range(max(0, steps - nw), steps):
            yield ("wait", f"wfull{b}.{j % nw}", (j // nw) & 1)

    def tokens(b):
        units = steps * per
        for u in range(units):
            yield ("wait", f"consumed{b}.{u % kx}", ((u // kx) & 1) ^ 1)
            if b == 0:
                yield ("expect", f"ready{u % kx}", 2)
            yield ("copy", f"ready{u % kx}", f"X{b}.{u % kx}")
        for u in range(max(0, units - kx), units):
            yield ("wait", f"consumed{b}.{u % kx}", (u // kx) & 1)

    def mmas():
        u = chunk = 0
        for n in segments:
            for i in range(n * per):
                ci = i % (CHUNK * per)
                if ci == 0 and not c.get("no_dempty"):
                    yield ("wait", f"dempty{chunk % ND}", ((chunk // ND) & 1) ^ 1)
                yield ("wait", f"ready{u % kx}", (u // kx) & 1)
                ds = [f"D{b}.{chunk % ND}" for b in (0, 1)]
                yield ("mma", [f"{r}{b}.{u % m}" for b in (0, 1) for r, m in (("A", KA), ("X", kx))], ds, ci == 0)
                ends = ci == CHUNK * per - 1 or i == n * per - 1
                if ends:
                    yield ("written", ds)
                for b in (0, 1) if not c.get("commit_to_one") else (0,):
                    yield ("commit", f"consumed{b}.{u % kx}")
                if ends:
                    for b in (0, 1):
                        yield ("commit", f"dfull{b}.{chunk % ND}")
                    chunk += 1
                u += 1
        yield ("commit", "mma_done")
        yield ("wait", "mma_done", 0)

    def widening(b, group):
        for j in range(steps):
            if (j & 1) != group:
                continue
            yield ("wait", f"wfull{b}.{j % nw}", (j // nw) & 1)
            if c.get("early_release"):
                yield ("arrive", f"wempty{b}.{j % nw}")
            for u in range(j * per, (j + 1) * per):
                if u >= KA and not c.get("no_consumed"):
                    yield ("wait", f"consumed{b}.{(u - KA) % kx}", ((u - KA) // kx) & 1)
                # the words may be loaded as late as here
                yield ("read", f"W{b}.{j % nw}")
                yield ("write", f"A{b}.{u % KA}")
                yield ("arrive", f"ready{u % kx}")
            if not c.get("early_release"):
                yield ("arrive", f"wempty{b}.{j % nw}")

    def epilogue(b, w):
        chunk = 0
        for n in segments:
            for _ in range(0, n, CHUNK):
                yield ("wait", f"dfull{b}.{chunk % ND}", (chunk // ND) & 1)
                yield ("read", f"D{b}.{chunk % ND}")
                yield ("arrive", f"dempty{chunk % ND}")
                chunk += 1
        if w == 0:        # sums, or others' partials, come into the rings
            for i in range(nw):
                yield ("write", f"W{b}.{i}")
            for i in range(kx):
                yield ("write", f"X{b}.{i}")

    roles = [("mmas", mmas())]
    for b in (0, 1):
        roles += [(f"words {b}", words(b)), (f"tokens {b}", tokens(b))]
        # a warp's lanes act as one; the four warps of a widening group, and the
        # eight of an epilogue, on warps' own counts
        roles += [(f"widening {b}.{g}.{w}", widening(b, g)) for g in (0, 1) for w in range(c["warps"])]
        roles += [(f"epilogue {b}.{w}", epilogue(b, w)) for w in range(2 * c["warps"])]
    return roles


def run(T, segments, seed, **change):
    """One randomized run of a pair's blocks; None if it finished cleanly."""
    c = dict(CONFIGS[T], warps=4)
    c.update(change)
    sim = _Pair(seed)
    for i in range(c["kx"]):
        sim.bar(f"ready{i}", 2 * c["warps"] + 1)
    for i in range(ND):
        sim.bar(f"dempty{i}", 4 * c["warps"])
    sim.bar("mma_done")
    for b in (0, 1):
        for i in range(c["nw"]):
            sim.bar(f"wfull{b}.{i}")
            sim.bar(f"wempty{b}.{i}", c["warps"])
        for i in range(c["kx"]):
            sim.bar(f"consumed{b}.{i}")
        for i in range(ND):
            sim.bar(f"dfull{b}.{i}")
    for name, gen in _roles(c, segments):
        sim.agents.append({"name": name, "gen": gen, "wait": None, "done": False})
    sim.rng = _Uneven(seed, [a["name"] for a in sim.agents])
    return sim.run()
