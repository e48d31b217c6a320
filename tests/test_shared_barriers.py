"""The barriers of the shared-prefix decode kernel, on the host (no GPU).

An mbarrier wait sees the parity of its phase only.  A wait for phase k is sound
if phase k - 1 has surely completed before it starts (else the phase of the same
parity before that one lets it pass) and phase k + 1 surely does not complete
before it has passed (else it blocks).  "Surely" is a matter of order, not of
time: this file lays down what every role of shared_attend_kernel does for a list
of segments - the order in each role, every arrival, every copy and product
that completes by itself - as a directed graph, and asks for each wait whether
those two orders follow from it.  So latencies play no part, and what holds here
holds for any.  The ring depths are read from the kernel's source.

Waits that the kernel makes only if a value asks for them (a row's maximum moved,
a tile has keys to mask) must be sound where they are made, but order nothing
for the rest of the program.
"""
from __future__ import annotations

import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tiled_attention_17_b200", "csrc",
                      "decode_shared.cu")


def depths(d):
    """(K slots, V slots, K barriers, V barriers, segments, query loads) of the kernel at head size d."""
    with open(SOURCE) as f:
        text = f.read()

    def by_size(name):
        a, b = re.search(rf"\b{name} = D == 128 \? (\d+) : (\d+)", text).groups()
        return int(a if d == 128 else b)

    def one(name):
        return int(re.search(rf"\b{name} = (\d+);", text).group(1))

    return (by_size("kKStages"), by_size("kVStages"), by_size("kKBars"), by_size("kVBars"), one("kSegments"),
            one("kQLoads"))


class Graph:
    def __init__(self):
        self.preds = []        # of each node
        self.done = {}         # (barrier, phase) -> node of its completion
        self.arrivals = {}     # (barrier, phase) -> how many
        self.count = {}        # barrier -> arrivals a phase takes
        self.waits = []        # (node before, node that goes on after, barrier, phase)

    def node(self, *preds):
        self.preds.append([p for p in preds if p is not None])
        return len(self.preds) - 1

    def phase(self, barrier, k):
        if (barrier, k) not in self.done:
            self.done[barrier, k] = self.node()
            self.arrivals[barrier, k] = 0
        return self.done[barrier, k]

    def arrive(self, node, barrier, k, n=1):
        self.preds[self.phase(barrier, k)].append(node)
        self.arrivals[barrier, k] += n

    def faults(self):
        """Waits that do not follow from the order (and phases that do not take their arrivals)."""
        found = []
        for (barrier, k), n in self.arrivals.items():
            if n != self.count[barrier]:
                found.append(f"{barrier}: phase {k} gets {n} arrivals")
        succs = [[] for _ in self.preds]
        missing = [len(p) for p in self.preds]
        for i, ps in enumerate(self.preds):
            for p in ps:
                succs[p].append(i)
        before = [0] * len(self.preds)   # bit sets of what comes before a node, itself among them
        ready, seen = [i for i, m in enumerate(missing) if m == 0], 0
        while ready:
            i = ready.pop()
            seen += 1
            before[i] |= 1 << i
            for s in succs[i]:
                before[s] |= before[i]
                missing[s] -= 1
                if missing[s] == 0:
                    ready.append(s)
        if seen != len(self.preds):
            return found + ["the roles wait for one another"]
        complete = {key: sum(1 << p for p in set(self.preds[i])) for key, i in self.done.items()}   # its arrivals
        for (barrier, k), i in self.done.items():
            earlier = complete.get((barrier, k - 1), 0)
            if any(before[p] & earlier != earlier for p in self.preds[i]):
                found.append(f"{barrier}: an arrival of phase {k} may come before phase {k - 1} is complete")
        for start, after, barrier, k in self.waits:
            earlier = complete.get((barrier, k - 1), 0)
            if before[start] & earlier != earlier:
                found.append(f"{barrier}: a wait for phase {k} may start before phase {k - 1} is complete")
            if (barrier, k + 1) in self.done and not before[self.done[barrier, k + 1]] >> after & 1:
                found.append(f"{barrier}: phase {k + 1} may complete before a wait for phase {k} has passed")
        return found


class Role:
    """One warp's (or warpgroup's) program."""

    def __init__(self, g):
        self.g, self.at, self.pending = g, g.node(), []

    def step(self):
        self.at = self.g.node(self.at)
        for w in self.pending:   # waits end before what comes next in their role
            self.g.waits.append((w[0], self.at, *w[1:]))
        self.pending = []

    def wait(self, barrier, k, sure=True):
        self.step()
        start = self.at
        if sure:
            self.at = self.g.node(start, self.g.phase(barrier, k))
        self.pending.append((start, barrier, k))
        if sure:
            self.step()

    def arrive(self, barrier, k, n=1):
        self.step()
        self.g.arrive(self.at, barrier, k, n)

    def copy(self, barrier, k):
        """A copy whose landing is the barrier's phase."""
        self.step()
        self.g.arrive(self.g.node(self.at), barrier, k)


class Issuer(Role):
    """A warp that issues products: a commit completes after all products before it."""
    last = None

    def commit(self, barrier, k):
        self.step()
        self.last = self.g.node(self.at, self.last)
        self.g.arrive(self.last, barrier, k)


def kernel(segments, ks, vs, kb, vb, kseg, qloads, weights=2):
    """The graph of one CTA.  segments: (kind "wide" | "narrow" | "own", steps), prefixes first.  kb, vb: arrival
    barriers of K and V tiles; weights: barriers that own keys' weights go round."""
    g = Graph()
    segs, g0, turn = [], 0, 0
    for kind, tiles in segments + [("own", 0)]:
        segs.append((kind == "wide", kind == "own", tiles, g0, turn))
        g0 += tiles
        if kind != "wide":
            turn ^= tiles & 1
    for name, n, count in (("KF", kb, 1), ("VF", vb, 1), ("KE", ks, 2), ("VE", vs, 2)):
        for i in range(n):
            g.count[name, i] = count
    for e in range(kseg):
        g.count["GF", e], g.count["GE", e] = 1, 4 + 4   # the softmax warpgroups as two workers each
    for t in (0, 1):
        for h in (0, 1):
            g.count["SF", t, h], g.count["PR", t, h], g.count["OD", t, h], g.count["SO", t, h] = 1, 2, 1, 1
        g.count["OF", t], g.count["X", t] = 2, 2
        for u in range(qloads):
            g.count["QF", t, u] = 1

    def take(role, n):
        role.wait(("GF", n % kseg), n // kseg)
        role.arrive(("GE", n % kseg), n // kseg)
        return segs[n]

    def first_of(seg, t):   # a row tile's first step and its stride
        wide, _, _, _, tile_first = seg
        return (0, 1) if wide else ((t ^ tile_first) & 1, 2)

    planner = Role(g)
    for n in range(len(segs)):
        if n >= kseg:
            planner.wait(("GE", n % kseg), n // kseg - 1)
        planner.arrive(("GF", n % kseg), n // kseg)

    for full, empty, bars, slots in (("KF", "KE", kb, ks), ("VF", "VE", vb, vs)):
        role, tile = Role(g), 0
        loads, last_step, last_own = [0, 0], [0, 0], [False, False]
        for n in range(len(segs)):
            wide, own, tiles, at, tile_first = take(role, n)
            for t in (0, 1):
                if full == "VF" or tiles == 0 or not wide and tiles == 1 and t != tile_first:
                    continue
                q = last_step[t]
                if loads[t] and not (own and last_own[t]) and q + ks >= at:
                    role.wait(("KE", q % ks), q // ks)
                role.copy(("QF", t, loads[t] % qloads), loads[t] // qloads)
                loads[t] += 1
                last_step[t] = at + (tiles - 1 if wide else tiles - 1 - ((tile_first + tiles - 1 + t) & 1))
                last_own[t] = own
            for _ in range(tiles):
                if tile >= slots:
                    role.wait((empty, tile % slots), tile // slots - 1)
                role.copy((full, tile % bars), tile // bars)
                tile += 1

    def issue(t):
        role = Issuer(g)
        steps = used = n = 0   # steps and segments of this row tile
        while True:
            seg = wide, own, tiles, at, _ = take(role, n)
            if tiles == 0:
                return
            first, stride = first_of(seg, t)
            if first >= tiles:
                n += 1
                continue
            role.wait(("QF", t, used % qloads), used // qloads)
            if own:
                k, j, due, start = 0, first, None, True
                while True:
                    have = j < tiles
                    tile = at + j
                    if have:
                        role.wait(("KF", tile % kb), tile // kb)
                        role.commit(("SO", t, k & 1), k >> 1)
                        role.commit(("KE", tile % ks), tile // ks)
                        role.arrive(("KE", tile % ks), tile // ks)
                    if k > 0:
                        v, starts, of = due
                        role.wait(("VF", v % vb), v // vb)
                        if starts and of > 0:
                            role.wait(("OF", t), of - 1)
                        role.wait(("PR", t, (k - 1) % weights), steps + (k - 1) // weights)
                        role.commit(("OD", t, (k - 1) & 1), steps + ((k - 1) >> 1))
                        role.commit(("VE", v % vs), v // vs)
                        role.arrive(("VE", v % vs), v // vs)
                    if not have:
                        return
                    due, start = (tile, start, used), False
                    k += 1
                    j += 2
                    while j >= tiles:
                        n += 1
                        seg = _, _, tiles, at, _ = take(role, n)
                        j = first_of(seg, t)[0]
                        if tiles == 0:
                            break
                        if j < tiles:
                            used, start = used + 1, True
                            role.wait(("QF", t, used % qloads), used // qloads)
            j, tile = first - stride, at + first   # step of the products, tile of the next scores
            while True:
                more, v, formed = j + stride < tiles, tile - stride, 0
                if j >= 0:
                    role.wait(("VF", v % vb), v // vb)
                if j == first and used > 0:
                    role.wait(("OF", t), used - 1)
                for h in (0, 1):
                    if j >= 0:
                        role.wait(("PR", t, h), steps)
                        role.commit(("OD", t, h), steps)
                        role.wait(("OD", t, h), steps)
                    if more:
                        role.wait(("KF", tile % kb), tile // kb, sure=h == 1)   # only tried at the first half
                        while h == 1 and formed <= h:   # (earlier if the try succeeds: no later order depends on it)
                            role.commit(("SF", t, formed), steps + (j >= 0))
                            formed += 1
                        if h == 1:
                            role.commit(("KE", tile % ks), tile // ks)
                            if not wide:
                                role.arrive(("KE", tile % ks), tile // ks)
                if j >= 0:
                    role.commit(("VE", v % vs), v // vs)
                    if not wide:
                        role.arrive(("VE", v % vs), v // vs)
                    steps += 1
                if not more:
                    break
                j += stride
                tile += stride
            used += 1
            n += 1

    def softmax(t):
        role = Role(g)
        steps = k = exchanges = segments_done = 0
        held, base = [0, 0], None
        for n in range(len(segs)):
            seg = wide, own, tiles, at, _ = take(role, n)
            if tiles == 0:
                return
            j, stride = first_of(seg, t)
            if j >= tiles:
                continue
            if own and base is None:
                base = steps

            def exchange():
                nonlocal exchanges
                role.arrive(("X", t), exchanges)
                role.wait(("X", t), exchanges)
                exchanges += 1

            first = True
            while j < tiles:
                v = at + j
                if own:
                    role.wait(("SO", t, k & 1), k >> 1)
                    role.wait(("VF", v % vb), v // vb, sure=False)   # keys to mask
                    exchange()
                    if not first:
                        role.wait(("OD", t, (k + 1) & 1), held[(k + 1) & 1] - 1, sure=False)   # a maximum moved
                    held[k & 1] += 1
                    role.arrive(("PR", t, k % weights), base + k // weights)
                    k += 1
                else:
                    for h in (0, 1):
                        role.wait(("SF", t, h), steps)
                        held[h] += 1
                        if h == 0:
                            role.wait(("VF", v % vb), v // vb, sure=False)
                        if not first:
                            role.wait(("OD", t, h ^ 1), held[h ^ 1] - 1, sure=False)
                        role.arrive(("PR", t, h), steps)
                        first = False
                    steps += 1
                j += stride
                first = False
            if own:
                exchange()
            h = (k + 1) & 1 if own else 1
            role.wait(("OD", t, h), held[h] - 1)
            role.arrive(("OF", t), segments_done)
            segments_done += 1

    for t in (0, 1):
        issue(t)
        softmax(t)
        softmax(t)
    return g


def lists(seed, n):
    """Lists of segments as the planner makes them: prefixes, then own keys."""
    rng = random.Random(seed)
    for _ in range(n):
        yield ([(rng.choice(("wide", "narrow")), rng.choice((1, 1, 2, 3, 5, 9))) for _ in range(rng.randrange(5))]
               + [("own", rng.choice((1, 1, 2, 2, 3, 6))) for _ in range(rng.randrange(12))])


@pytest.mark.parametrize("d", [64, 128])
def test_every_wait_follows_from_the_order(d):
    for segments in [[], [("wide", 9)], [("narrow", 9)], [("own", 9)], [("own", 1)] * 20, [("narrow", 1)] * 9,
                     [("wide", 1), ("narrow", 7), ("wide", 2)] + [("own", 3)] * 5] + list(lists(d, 120)):
        assert kernel(segments, *depths(d)).faults() == [], segments


@pytest.mark.parametrize("what", ["K", "V", "weights"])
def test_fewer_barriers_alias(what):
    # one barrier for each slot of a ring, or one for all weights of own keys: a wait may fall two phases behind
    ks, vs, kb, vb, *rest = depths(128)
    if what == "K":
        graphs = (kernel(s, ks, vs, ks, vb, *rest) for s in lists(1, 200))
        barrier = "KF"
    elif what == "V":
        graphs = (kernel(s, ks, vs, kb, vs, *rest) for s in lists(2, 200))
        barrier = "VF"
    else:
        graphs = (kernel(s, ks, vs, kb, vb, *rest, weights=1) for s in lists(3, 200))
        barrier = "PR"
    assert any(f"'{barrier}'" in f for graph in graphs for f in graph.faults())
