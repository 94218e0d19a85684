"""The barriers of attn_qat_cross's kernel, simulated on the host.

The roles of one CTA (csrc/attn_cross.cu) as coroutines that wait and arrive as the kernel's warps
do, in a random order; the MMAs and copies that a warp issues end later, in the order of that warp
alone.  Barriers have parities only, as mbarriers have.  Everything that is shared carries a tag of
what it should hold (tile, segment, unit), and each access checks it: a buffer taken too early, a
phase passed that was another one's, a description overwritten, or roles that wait for one another
for ever show up on some order.

Runs are lists of segments (rows over 128 or not, tiles, which tiles' pages are absent); one and
two halves of the rows follow each other in any order.
"""
import random

import pytest

SEGS = 8  # descriptions of segments that are kept


class Wrong(Exception):
    pass


def need(ok, *what):
    if not ok:
        raise Wrong(*what)


class Bar:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passed(self, parity):
        return self.phase & 1 != parity


class Cta:
    def __init__(self, segments, stages, rng, fault=None):
        self.rng, self.stages, self.fault = rng, stages, fault
        self.segments = segments
        # tile: (segment, first, last, absent)
        self.tiles = [(s, i == 0, i == len(absent) - 1, absent[i])
                      for s, (both, absent) in enumerate(segments) for i in range(len(absent))]
        n = stages
        self.full, self.empty = [Bar(1) for _ in range(n)], [Bar(2 + 1 + 4) for _ in range(n)]
        self.k_ready = [Bar(1) for _ in range(n)]
        self.v_full, self.v_empty = [Bar(4) for _ in range(2)], [Bar(1) for _ in range(2)]
        self.q_full, self.q_empty = [Bar(4) for _ in range(2)], [Bar(2) for _ in range(2)]
        self.s_full = [[Bar(2) for _ in range(3)] for _ in range(2)]
        self.p_full, self.pv_done = [Bar(4) for _ in range(3)], [Bar(1) for _ in range(3)]
        self.o_full, self.o_read = [Bar(1) for _ in range(2)], [Bar(8) for _ in range(2)]
        self.merge = [[Bar(1) for _ in range(4)] for _ in range(2)]
        self.described, self.q_first = [Bar(1) for _ in range(SEGS)], Bar(12)
        # what the shared places hold
        self.desc, self.k, self.v = [None] * n, [None] * n, [[None] * 4, [None] * 4]
        self.k_arranged = [None] * n
        self.segs = [None] * SEGS
        self.q = [[None] * 4, [None] * 4]
        self.sf_q = [[None, None], [None, None]]  # [stream][buffer]
        self.sf_k = [[None, None], [None, None]]
        self.units = [[None] * 3, [None] * 3]
        self.s = [None] * 3                       # (unit, MMA done)
        self.p = [[None] * 4 for _ in range(3)]
        self.o = [(None, 0), (None, 0)]           # segment, PVs of it
        self.ml = [[None] * 4, [None] * 4]
        self.queues = {}
        self.segs[0] = 0                          # described by the thread that finds the run
        self.described[0].arrive()

    def both(self, seg):
        return self.segments[seg][0]

    def issue(self, warp, f):
        self.queues.setdefault(warp, []).append(f)

    # ---- the roles
    def first_q(self, w):  # all warps but the issuing ones, before their own part
        if w >= 12:
            self.q[0][w - 12] = 0
        (self.q_first if w < 12 else self.q_full[0]).arrive()

    def producer(self):
        n = 0
        for seg, (_, absent) in enumerate(self.segments):
            yield self.described[seg % SEGS], (seg // SEGS) & 1
            need(self.segs[seg % SEGS] == seg, "producer's segment")
            for _ in absent:
                st = n % self.stages
                yield self.empty[st], ((n // self.stages) & 1) ^ 1
                self.desc[st] = n
                self.k[st], self.k_arranged[st] = n, None
                self.full[st].arrive()
                n += 1

    def decoder(self, w):
        self.first_q(8 + w)
        yield None
        for n in range(len(self.tiles)):
            st, b = n % self.stages, n & 1
            yield self.full[st], (n // self.stages) & 1
            need(self.desc[st] == n, "decoder's tile")
            if w == 0:
                self.k_arranged[st] = n
                self.k_ready[st].arrive()
            yield self.v_empty[b], ((n >> 1) & 1) ^ 1
            need(self.k[st] == n, "V's codes")
            yield None
            self.v[b][w] = n
            self.v_full[b].arrive()
            self.empty[st].arrive()

    def query(self, w):
        self.first_q(12 + w)
        yield None
        for seg in range(1, len(self.segments)):
            if w == 0:
                self.segs[seg % SEGS] = seg
                self.described[seg % SEGS].arrive()
            yield self.described[seg % SEGS], (seg // SEGS) & 1
            need(self.segs[seg % SEGS] == seg, "query's segment")
            if self.fault != "q_empty":
                yield self.q_empty[seg & 1], ((seg >> 1) & 1) ^ 1
            self.q[seg & 1][w] = seg
            self.q_full[seg & 1].arrive()

    def scores(self, stream):
        u, word, me = stream, 0, f"s{stream}"
        for n, (seg, first, last, absent) in enumerate(self.tiles):
            st, qb, both = n % self.stages, seg & 1, self.both(seg)
            yield self.k_ready[st], (n // self.stages) & 1
            need(self.desc[st] == n, "S's tile")
            if first:
                yield self.q_full[qb], (seg >> 1) & 1
            if n == 0:
                yield self.q_first, 0
            for j in range(2 if both else 1):
                end = j == both
                bar = self.s_full[0 if self.fault == "s_full" else stream][
                    u % 3 if self.fault == "s_full" else word]
                self.units[stream][word] = (u, first and j == 0, last and end,
                                            n == len(self.tiles) - 1 and end, both, seg)
                word = (word + 1) % 3
                if self.fault != "pv_done":
                    yield self.pv_done[u % 3], ((u // 3) & 1) ^ 1

                def mma(u=u, n=n, st=st, seg=seg, qb=qb, first=first, j=j, absent=absent):
                    if j == 0 and first:
                        need(self.q[qb] == [seg] * 4, "scales of q~", seg, self.q[qb])
                        self.sf_q[stream][qb] = seg
                    if j == 0 and not absent:
                        need(self.k_arranged[st] == n, "scales of K")
                        self.sf_k[stream][n & 1] = n
                    if not absent:
                        need(self.k[st] == n and self.q[qb] == [seg] * 4, "operands of S")
                        need(self.sf_q[stream][qb] == seg and self.sf_k[stream][n & 1] == n, "scales")
                    # S over the P that the PV three units before has read
                    need(self.s[u % 3] is None or self.s[u % 3] == (u - 3, "read"), "buffer of S")
                    self.s[u % 3] = (u, "S")

                self.issue(me, mma)
                self.issue(me, bar.arrive)
                if end:
                    self.issue(me, self.empty[st].arrive)
                yield None
                bar.arrive()
                u += 2
            if last:
                self.issue(me, self.q_empty[qb].arrive)

    def products(self):
        u = 0
        for n, (seg, first, last, _) in enumerate(self.tiles):
            st, b, halves = n % self.stages, n & 1, 2 if self.both(seg) else 1
            yield self.full[st], (n // self.stages) & 1
            need(self.desc[st] == n, "PV's tile")
            self.empty[st].arrive()
            yield self.v_full[b], (n >> 1) & 1
            for x in range(2 * halves):
                stream = x & 1
                start = first and x < 2
                if start and seg > 0 and self.fault != "o_read":
                    yield self.o_read[stream], (seg - 1) & 1
                yield self.p_full[u % 3], (u // 3) & 1

                def mma(u=u, n=n, b=b, seg=seg, stream=stream, start=start):
                    need(self.p[u % 3] == [u] * 4 and self.s[u % 3] == (u, "S"), "P", u)
                    need(self.v[b] == [n] * 4, "V", n, self.v[b])
                    need(start or self.o[stream][0] == seg, "O")
                    self.o[stream] = (seg, 1 if start else self.o[stream][1] + 1)
                    self.s[u % 3] = (u, "read")

                self.issue("pv", mma)
                self.issue("pv", self.pv_done[u % 3].arrive)
                if x == 2 * halves - 1:
                    self.issue("pv", self.v_empty[b].arrive)
                if last and x >= 2 * halves - 2:
                    self.issue("pv", self.o_full[stream].arrive)
                yield None
                u += 1

    def softmax(self, stream, quarter):
        self.first_q(4 * stream + quarter)
        yield None
        u, k, ends, joins, done = stream, 0, 0, 0, 0
        while True:
            bar = self.s_full[0][u % 3] if self.fault == "s_full" else self.s_full[stream][k % 3]
            parity = (u // 3 if self.fault == "s_full" else k // 3) & 1
            yield bar, parity
            what = self.units[stream][k % 3]
            need(what is not None and what[0] == u, "the unit's word", u, what)
            _, start, end, last, both, seg = what
            need(seg == ends and self.segs[ends % SEGS] == seg, "the softmax's segment")
            need(self.s[u % 3] == (u, "S"), "S", u, self.s[u % 3])
            if start:
                done = 0
            elif self.rng.random() < 0.5:  # the maximum is raised: O so far
                yield self.pv_done[(u - 2) % 3], ((u - 2) // 3) & 1
                need(self.o[stream] == (seg, done), "O to rescale", self.o[stream], seg, done)
            yield None
            self.p[u % 3][quarter] = u
            self.p_full[u % 3].arrive()
            done += 1
            u, k = u + 2, k + 1
            if end:
                yield self.o_full[stream], ends & 1
                ends += 1
                if not both:
                    self.ml[stream][quarter] = seg
                    self.merge[stream][quarter].arrive()
                    yield self.merge[stream ^ 1][quarter], joins & 1
                    joins += 1
                    need(self.ml[stream ^ 1][quarter] == seg, "the other stream's sums")
                    need(self.o[stream ^ 1][0] == seg, "the other stream's O")
                yield None
                need(self.o[stream] == (seg, done), "O", self.o[stream], seg, done)
                if not both:
                    need(self.o[stream ^ 1][0] == seg, "the other stream's O, read")
                self.o_read[stream].arrive()
                self.o_read[stream if both else stream ^ 1].arrive()
                yield None  # rows out: the segment's place is still read
                need(self.segs[(ends - 1) % SEGS] == seg, "the segment's place")
            if last:
                return

    def run(self):
        roles = {"producer": self.producer(), "pv": self.products()}
        for i in range(2):
            roles[f"s{i}"] = self.scores(i)
            for w in range(4):
                roles[f"softmax{i}{w}"] = self.softmax(i, w)
        for w in range(4):
            roles[f"v{w}"], roles[f"q{w}"] = self.decoder(w), self.query(w)
        waits = dict.fromkeys(roles)
        # some roles slower than others, which of them differs from run to run
        weight = {r: self.rng.choice((0.05, 0.3, 1, 1, 1)) for r in list(roles) + ["async"]}
        while roles:
            ready = [r for r in roles if waits[r] is None or waits[r][0].passed(waits[r][1])]
            ready += [("async", w) for w, q in self.queues.items() if q]
            need(ready, "for ever waiting", sorted(roles))
            r = self.rng.choices(ready, [weight[r if isinstance(r, str) else "async"]
                                         for r in ready])[0]
            if isinstance(r, tuple):
                self.queues[r[1]].pop(0)()
                continue
            try:
                waits[r] = next(roles[r])
            except StopIteration:
                del roles[r], waits[r]
        for q in self.queues.values():
            for f in q:
                f()


def segments(rng, most):
    kinds = rng.choice(((False,), (True,), (False, True), (False, True), (False, True)))
    lengths = rng.choice(((1,), (1, 2), (1, 1, 2, 3, 5), (4, 5)))
    return [(rng.choice(kinds), [rng.random() < 0.1 for _ in range(rng.choice(lengths))])
            for _ in range(rng.randint(1, most))]


@pytest.mark.parametrize("stages", [3, 8])
@pytest.mark.parametrize("seed", range(8))
def test_every_order_ends_and_reads_what_it_should(seed, stages):
    rng = random.Random(100 * stages + seed)
    for _ in range(25):
        Cta(segments(rng, 6), stages, rng).run()
    for _ in range(3):
        Cta(segments(rng, 30), stages, rng).run()


@pytest.mark.parametrize("fault", ["q_empty", "pv_done", "o_read", "s_full"])
def test_a_missing_wait_and_a_barrier_of_both_streams_show(fault):
    """s_full: one barrier for both streams, by the unit's number.  A stream that has none of three
    units in turn is then phases behind, and its parity is another phase's."""
    rng = random.Random(5)
    for _ in range(300):
        try:
            Cta(segments(rng, 6), 3, rng, fault).run()
        except Wrong:
            return
    pytest.fail("not seen")
