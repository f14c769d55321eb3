"""The warps of the bf16 shared-prefix attention (csrc/shared_attn_tc.cu) as a
discrete-event model: what a wait that runs out does to the others.

Every mbarrier wait has a limit; the named barriers at which the softmax warps
meet have none.  So after a timeout all softmax warps still have to pass the
same barriers: they follow the producer's list of segments to its end, which
a producer that gives up publishes too, and a warp that has given up arrives
at no mbarrier any more, so that the others run out as well and nobody gets
ahead.  The model runs the roles with their waits, arrivals and barriers over
random segments, lets one agent stall for longer than the limit at a random
place, and every agent has to come to its end."""
import heapq
import pathlib
import random
import re

import pytest

LIMIT = 1000.0
SOURCE = (pathlib.Path(__file__).parents[1] / "long_prefix_attention_b200/csrc/shared_attn_tc.cu").read_text()
SEG_WAITS, SEGS = (int(re.search(rf"constexpr int {k} = (\d+);", SOURCE)[1]) for k in ("kSegWaits", "kSegs"))


class Bar:
    """An mbarrier: `count` arrivals complete a phase."""

    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self, n=1):
        self.left -= n
        assert self.left >= 0, "more arrivals than a phase has"
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def done(self, parity):
        return (self.phase & 1) != parity


class Sim:
    def __init__(self, segs, ring, rng, stall, end_on_abort=True, seg_waits=SEG_WAITS, failed_arrive=False):
        self.segs, self.ring, self.rng = segs, ring, rng
        self.end_on_abort, self.seg_waits, self.failed_arrive = end_on_abort, seg_waits, failed_arrive
        self.now, self.heap, self.tick, self.blocked, self.named = 0.0, [], 0, {}, {}
        self.published = [None] * SEGS
        self.seg_full = [Bar(1) for _ in range(SEGS)]
        self.kv_full, self.kv_empty = [Bar(1) for _ in range(ring)], [Bar(2) for _ in range(ring)]
        self.s_full, self.p_full = [Bar(1), Bar(1)], [Bar(4), Bar(4)]     # one arrival per warp
        self.o_full = [Bar(1), Bar(1)]
        self.turn = [[Bar(1) for _ in range(ring // 2)] for _ in range(2)]
        self.errors, self.finished = set(), set()
        self.stall = stall or (None, 0, 0.0)                              # (agent, its how many-th event, time)
        self.count = {}
        self.agents = {"prod": self.producer(), "iss0": self.issuer(0), "iss1": self.issuer(1)}
        for w in range(8):
            self.agents[f"soft{w}"] = self.softmax(w)

    # ---- scheduler: agents yield ("wait", bar, parity), ("meet", name, n), ("after", fn, delay) or ("work", t)
    def push(self, t, what):
        self.tick += 1
        heapq.heappush(self.heap, (t, self.tick, what))

    def run(self):
        for a in self.agents:
            self.push(0.0, ("go", a, None))
        while self.heap:
            self.now, _, what = heapq.heappop(self.heap)
            assert self.now < 200 * LIMIT, "no end in sight"
            if what[0] == "call":
                what[1]()
                self.wake()
            elif what[0] == "limit":
                if self.blocked.get(what[1], (None,))[0] == what[2]:
                    del self.blocked[what[1]]
                    self.step(what[1], False)
            else:
                self.step(what[1], what[2])
        return self.finished == set(self.agents)

    def wake(self):
        for a, (_, bar, parity) in list(self.blocked.items()):
            if bar.done(parity):
                del self.blocked[a]
                self.push(self.now, ("go", a, True))

    def step(self, a, value):
        try:
            r = self.agents[a].send(value)
        except StopIteration:
            self.finished.add(a)
            return
        self.wake()
        self.count[a] = self.count.get(a, 0) + 1
        late = self.stall[2] if self.stall[:2] == (a, self.count[a]) else 0.0
        if r[0] == "work":
            self.push(self.now + r[1] + late, ("go", a, None))
        elif r[0] == "after":
            self.push(self.now + r[2], ("call", r[1]))
            self.push(self.now + late, ("go", a, None))
        elif r[0] == "wait":
            if r[1].done(r[2]):
                self.push(self.now + late, ("go", a, True))
            else:
                self.tick += 1
                self.blocked[a] = (self.tick, r[1], r[2])
                self.push(self.now + LIMIT + late, ("limit", a, self.tick))
        else:
            self.named.setdefault(r[1], []).append(a)
            if len(self.named[r[1]]) == r[2]:
                for b in self.named.pop(r[1]):
                    self.push(self.now + late, ("go", b, None))

    # ---- roles
    def producer(self):
        ok, segs, n = True, 0, 0

        def publish(s):
            nonlocal segs
            self.published[segs % SEGS] = (segs, s)
            self.seg_full[segs % SEGS].arrive()
            segs += 1

        todo = list(self.segs)
        nxt = todo.pop(0) if todo else None
        publish(nxt)
        while ok and nxt is not None:
            cur, nxt = nxt, (todo.pop(0) if todo else None)
            publish(nxt)
            for _ in range(2 * cur["n"]):
                slot = n % self.ring
                if n >= self.ring:
                    ok = ok and (yield ("wait", self.kv_empty[slot], ((n // self.ring) - 1) & 1))
                if not ok:
                    break
                n += 1
                yield ("after", self.kv_full[slot].arrive, self.rng.uniform(1, 4))
        if self.end_on_abort and nxt is not None:
            publish(None)
        if not ok:
            self.errors.add("prod")

    def issuer(self, x):
        ok, segs, step, unit0 = True, 0, 0, 0
        p_bit, turns = 0, [0] * (self.ring // 2)
        steps = []                        # (item of K, first of the segment, last, dual, j, n)

        def more():
            nonlocal ok, segs, step, unit0
            while not steps:
                ok = ok and (yield ("wait", self.seg_full[segs % SEGS], (segs // SEGS) & 1))
                s = self.published[segs % SEGS][1] if ok else None
                segs += 1
                if s is None:
                    return False
                dual, n = s["rows"] > 128, s["n"]
                js = range(n) if dual else range(x ^ (step & 1), n, 2)
                steps.extend((2 * (unit0 + j), j, n, dual, j == js[0], j == js[-1]) for j in js)
                step += 2 * n if dual else n
                unit0 += n
            return True

        def scores(it):
            nonlocal ok
            item, j, n, dual, _, _ = it
            if dual and (x == 1 or j > 0):
                i = (item // 2) % (self.ring // 2)
                ok = ok and (yield ("wait", self.turn[x][i], turns[i]))
                turns[i] ^= 1
            ok = ok and (yield ("wait", self.kv_full[item % self.ring], (item // self.ring) & 1))
            if ok:
                def fin():
                    self.s_full[x].arrive()
                    self.kv_empty[item % self.ring].arrive(1 if dual else 2)
                yield ("after", fin, self.rng.uniform(1, 3))

        have = yield from more()
        if have:
            yield from scores(steps[0])
        while ok and have:
            item, j, n, dual, _, last = steps.pop(0)
            item += 1
            ok = ok and (yield ("wait", self.kv_full[item % self.ring], (item // self.ring) & 1))
            ok = ok and (yield ("wait", self.p_full[x], p_bit))
            p_bit ^= 1
            if not ok:
                break

            def fin(item=item, last=last, dual=dual):
                if last:
                    self.o_full[x].arrive()
                self.kv_empty[item % self.ring].arrive(1 if dual else 2)
            yield ("after", fin, self.rng.uniform(1, 3))
            have = yield from more()
            if have:
                yield from scores(steps[0])
        if not ok:
            self.errors.add(f"iss{x}")

    def softmax(self, w):
        x, ok, sn, on, step, seg, unit0 = w >> 2, True, 0, [0, 0], 0, 0, 0
        while True:
            got = False
            for _ in range(self.seg_waits):
                got = yield ("wait", self.seg_full[seg % SEGS], (seg // SEGS) & 1)
                if got:
                    break
            at, s = self.published[seg % SEGS] if got else (seg, None)
            assert at == seg, "a segment was replaced before it was read"
            ok = ok and got
            seg += 1
            if s is None:
                break
            rows, n = s["rows"], s["n"]
            dual = rows > 128
            j0, dj = (0, 1) if dual else (x ^ (step & 1), 2)
            item0 = unit0
            step += 2 * n if dual else n
            unit0 += n
            if j0 >= n:
                on[x ^ 1] += 1
                continue
            joint = dual or n > 1
            for j in range(j0, n, dj):
                ok = ok and (yield ("wait", self.s_full[x], sn & 1))
                sn += 1
                if dual and w % 4 == 0 and (x == 0 or j + 1 < n) and (ok or self.failed_arrive):
                    self.turn[x ^ 1][(item0 + j + x) % (self.ring // 2)].arrive()
                yield ("work", self.rng.uniform(1, 3))
                if ok or self.failed_arrive:
                    self.p_full[x].arrive()
            for y in ((x, x ^ 1) if joint else (x,)):
                ok = ok and (yield ("wait", self.o_full[y], on[y] & 1))
                on[y] += 1
            meets = 2 if rows > 32 else 4
            if joint or rows <= 32 or s["fixable"]:
                for _ in range(meets):
                    yield ("meet", "both", 8) if joint else ("meet", x, 4)
                    yield ("work", self.rng.uniform(0, 1))
        if not ok:
            self.errors.add(f"soft{w}")


def segments(rng):
    """Short, middle and tall tiles; many of a single unit."""
    return [dict(rows=rng.choice([8, 20, 60, 128, 200, 256]), n=rng.choice([1, 1, 1, 2, 3, 7]), fixable=rng.random() < 0.3)
            for _ in range(rng.randint(1, 40))]


def stall_time(rng):
    return rng.choice([rng.uniform(LIMIT - 10, LIMIT + 40), 3.5 * LIMIT])


@pytest.mark.parametrize("ring", [4, 8])
def test_the_roles_run_through_without_a_stall(ring):
    for seed in range(40):
        rng = random.Random(seed)
        sim = Sim(segments(rng), ring, rng, None)
        assert sim.run() and not sim.errors


@pytest.mark.parametrize("ring", [4, 8])
def test_every_warp_ends_after_a_timeout(ring):
    """One agent stalls at any of its events: for about the limit, so that some of the
    others give up and some do not, or for several."""
    timeouts = 0
    for seed in range(400):
        rng = random.Random(seed)
        who = rng.choice(["prod", "prod", "prod", "iss0", "iss1", *(f"soft{w}" for w in range(8))])
        sim = Sim(segments(rng), ring, rng, (who, rng.randint(1, 60), stall_time(rng)))
        assert sim.run(), (seed, who, sorted(set(sim.agents) - sim.finished))
        timeouts += bool(sim.errors)
    assert timeouts > 100          # the stalls reach the others
