"""Executable models of the synchronisation in the gated tensor-core kernels, checked under random
schedules: ``BackwardModel`` (gated_backward_tc.cuh), ``StateModel`` (gated_state_tc.cuh) and
``PrefillModel`` (gated_prefill_tc.cuh) in long_context_04_b200/csrc.

As in ``tc_protocol.py`` there is no arithmetic: each agent is a generator that mirrors one role of
a kernel, a group of warps being two or four agents, and asynchronous work (TMA landings and
stores, MMA completions, commit arrivals) happens in random order between the agents' steps.
Checked in every schedule:
  * the parity rules of every wait, and that every arrival lands in the phase its sender means;
  * whoever reads a place (a product, a warp, a TMA store) finds the data it means, landed,
    complete and with the rows behind the sequence zeroed;
  * nothing is overwritten before all who were to read it have, or while a product or a store
    still reads it, and no accumulator while a product is in flight on it;
  * ordinary stores are fenced (proxy fence) before a product or a TMA store reads them, and
    ordinary reads before TMA writes their place;
  * no deadlock, nothing in flight at the end.
Not modelled: the abort paths, register shares, TMEM allocation.
"""
from __future__ import annotations

from pair_protocol import STEP, Barrier, ProtocolError, _Ev
from tc_protocol import TcModel


class Place:
    """A piece of shared memory or an accumulator."""

    def __init__(self, name):
        self.name, self.tag, self.zeroed = name, None, True
        self.need = set()        # who still has to read what it holds
        self.reading, self.writing = {}, {}
        self.stored = set()      # agents whose ordinary stores are not fenced yet
        self.loaded = set()      # agents whose ordinary reads are not fenced yet

    def busy(self, exclude=None):
        return any(n for w, n in self.reading.items() if w != exclude) or \
            any(n for w, n in self.writing.items() if w != exclude)


class _Stored:
    """A TMA store's reads of its places are done."""

    def __init__(self, places, bar):
        self.places, self.bar = places, bar

    def arrive(self, phase, who):
        for p in self.places:
            p.reading["store"] -= 1
        self.bar.arrive(phase, who)


class Engine(TcModel):
    ISSUERS = ()

    def __init__(self, mutations=()):
        self.mut = frozenset(mutations)
        self.inflight, self.commits = [], []
        self.fifo = {i: [] for i in self.ISSUERS}
        self.issued = {i: 0 for i in self.ISSUERS}
        self.completed = {i: 0 for i in self.ISSUERS}
        self.bulk = {}

    def agents(self):
        return self.roles

    # ------------------------------------------------------------------ primitives
    def _fill(self, who, p, tag, need, what):
        if p.need:
            raise ProtocolError(f"{who}: {what} of {tag} over {p.name} ({p.tag}) that "
                                f"{sorted(p.need)} still have to read")
        p.tag, p.need = tag, set(need)

    def load(self, who, p, tag, bar, phase, need, zeroed=True):
        """TMA load; the caller has announced its bytes."""
        if p.busy():
            raise ProtocolError(f"{who}: TMA load of {tag} into {p.name} while it is in use")
        if p.loaded or p.stored:
            raise ProtocolError(f"{who}: TMA load of {tag} into {p.name} behind ordinary accesses of "
                                f"{sorted(p.loaded | p.stored)} without a proxy fence")
        self._fill(who, p, tag, need, "TMA load")
        p.zeroed = zeroed
        p.writing["tma"] = p.writing.get("tma", 0) + 1
        self.inflight.append(_Ev("tma", p, bar, phase, who))

    def _holds(self, who, p, tag, what, zeroed=True):
        if p.tag != tag or any(p.writing.values()):
            raise ProtocolError(f"{who}: {what} finds {p.name} holding {p.tag}"
                                f"{' (in flight)' if any(p.writing.values()) else ''}, wants {tag}")
        if zeroed and not p.zeroed:
            raise ProtocolError(f"{who}: {what} reads {p.name} before its last rows were zeroed")

    def read(self, who, p, tag, zeroed=False, smem=True):
        self._holds(who, p, tag, "a read", zeroed)
        if who not in p.need:
            raise ProtocolError(f"{who}: reads {p.name} ({tag}) unannounced")
        p.need.discard(who)
        if smem:
            p.loaded.add(who)

    def write(self, who, p, tag, need, smem=True):
        if p.busy():
            raise ProtocolError(f"{who}: stores {tag} into {p.name} while it is in use")
        self._fill(who, p, tag, need, "a store")
        p.zeroed = True
        if smem:
            p.stored.add(who)

    def update(self, who, p, tag, new):
        """An accumulator read, changed and written back."""
        if p.tag != tag or p.busy():
            raise ProtocolError(f"{who}: rescales {p.name} holding {p.tag}, wants {tag}, at rest")
        p.tag = new

    def zero(self, who, p, tag):
        self._holds(who, p, tag, "zeroing", zeroed=False)
        p.zeroed = True
        p.stored.add(who)

    def fence(self, who):
        for p in self.places:
            p.loaded.discard(who)
            p.stored.discard(who)

    def place(self, name):
        p = Place(name)
        self.places.append(p)
        return p

    def product(self, issuer, what, reads, acc, tag, new, need, keep, zeroed=True):
        for p, t in reads:
            if any(n for w, n in p.writing.items() if w not in (issuer,)):
                raise ProtocolError(f"{issuer}: {what} reads {p.name} while it is written")
            if p.tag != t:
                raise ProtocolError(f"{issuer}: {what} reads {p.name} holding {p.tag}, wants {t}")
            if p.stored:
                raise ProtocolError(f"{issuer}: {what} reads {p.name} behind stores of {sorted(p.stored)} "
                                    f"without a proxy fence")
            if zeroed and not p.zeroed:
                raise ProtocolError(f"{issuer}: {what} reads {p.name} before its last rows were zeroed")
            p.need.discard(what)
            p.reading[issuer] = p.reading.get(issuer, 0) + 1
        if acc.busy(exclude=issuer):
            raise ProtocolError(f"{issuer}: {what} writes {acc.name} while it is in use")
        if keep:
            if acc.tag != tag:
                raise ProtocolError(f"{issuer}: {what} adds to {acc.name} holding {acc.tag}, wants {tag}")
            acc.tag = new
            acc.need = set(need)
        else:
            self._fill(issuer, acc, new, need, what)
        acc.writing[issuer] = acc.writing.get(issuer, 0) + 1
        self.fifo[issuer].append(([p for p, _ in reads], [acc]))
        self.issued[issuer] += 1

    def tma_store(self, who, places, tag):
        for p in places:
            self._holds(who, p, tag, "a TMA store")
            if p.stored:
                raise ProtocolError(f"{who}: TMA store of {p.name} behind stores of {sorted(p.stored)} "
                                    f"without a proxy fence")
            p.need.discard(who)
            p.reading["store"] = p.reading.get("store", 0) + 1
        bar, n = self.bulk.setdefault(who, [Barrier(f"stores of {who}", 1), 0])
        self.inflight.append(_Ev("arrive", _Stored(places, bar), n, who))
        self.bulk[who][1] = n + 1

    def stores_read(self, who):
        """Wait for this agent's stores to have read shared memory."""
        if who in self.bulk and self.bulk[who][1]:
            yield ("wait", self.bulk[who][0], self.bulk[who][1] - 1)

    def _check_wait(self, who, bar, n, start):
        if bar.name.startswith("stores of"):   # a count, not a parity
            return
        super()._check_wait(who, bar, n, start)


class BackwardModel(Engine):
    """One CTA over tiles, ``tails`` saying of each whether its block is partial.  ``stream``: D = 128
    (second parts through one slot, P over v), else D = 64."""

    ISSUERS = ("mma",)
    A, B = ("A0", "A1"), ("B0", "B1")

    def __init__(self, tails, stream=True, have_s=True, have_ds=True, mutations=()):
        super().__init__(mutations)
        self.tails, self.stream, self.hs, self.hd = tails, stream, have_s, have_ds
        self.places = []
        for n in ("q", "k", "do", "ds", "low", "gates", "ts", "tt", "tdq", "tdk", "sums"):
            setattr(self, n, self.place(n))
        self.v, self.s = ([self.place(f"{n}{i}") for i in range(2)] for n in ("v", "s"))
        self.p = self.v if stream else [self.place(f"p{i}") for i in range(2)]
        self.rc = [self.place(f"rowcol{i}") for i in range(2)]
        self.re = [self.place(f"rs{i}") for i in range(2)]
        one = ("full_vo full_k full_qs full_ds low_full low_free low_done gates first_full dv1_full dv_full dq_full "
               "out_full tail done dg_done")
        self.bar = {n: Barrier(n, 1) for n in one.split()}
        self.bar.update({n: Barrier(n, 2) for n in "s_free p_ready scaled dv_read dk_read dq_read".split()})
        self.dlows = 2 if stream and have_ds else 0
        self.lows = self.dlows + (2 if stream and have_s else 0)
        self.roles = {"load": self.loader(), "mma": self.issuer(), "dg": self.dg()}
        self.roles.update({a: self.scores(a, i) for i, a in enumerate(self.A)})
        self.roles.update({b: self.first_terms(b, i) for i, b in enumerate(self.B)})

    def w(self, name, phase):
        return ("wait", self.bar[name], phase)

    def low_tag(self, t, i):
        return ("dsl" if i < self.dlows else "sl", t, i & 1)

    # ---------------------------------------------------------------- warp 0
    def loader(self):
        who, n = "load", len(self.tails)
        count = [0]

        def ds(t):
            self.bar["full_ds"].arrive(t, who, 1 if self.hd else 0)
            if self.hd:
                self.load(who, self.ds, ("ds", t), self.bar["full_ds"], t, {"v dS", "k dS"})

        def low(t, i):
            self.bar["low_full"].arrive(count[0], who, 1)
            what = f"{'v dS' if i < self.dlows else 'do S'} low{i & 1}"
            self.load(who, self.low, self.low_tag(t, i), self.bar["low_full"], count[0], {what})
            count[0] += 1

        def vo(t):
            z = not self.tails[t]
            self.bar["full_vo"].arrive(t, who, 3)
            low_do = {"do S low0", "do S low1"} if self.stream and self.hs else set()
            self.load(who, self.do, ("do", t), self.bar["full_vo"], t,
                      {"t", "P do"} | ({"do S"} if self.hs else set()) | low_do, z)
            for p in self.v:
                need = {"t"} | ({"v dS"} if self.hd else set()) | ({"v dS low0", "v dS low1"} if self.dlows else set())
                self.load(who, p, ("v", t), self.bar["full_vo"], t, need, z)

        def k(t):
            self.bar["full_k"].arrive(t, who, 1)
            need = {"s", "dP k"} | ({"k dS"} | set(self.B) if self.hd else set())
            self.load(who, self.k, ("k", t), self.bar["full_k"], t, need, not self.tails[t])

        def qs(t):
            self.bar["full_qs"].arrive(t, who, 3 if self.hs else 1)
            need = {"s", "dP q"} | (set(self.B) if self.hs else set())
            self.load(who, self.q, ("q", t), self.bar["full_qs"], t, need, not self.tails[t])
            if self.hs:
                for p in self.s:
                    self.load(who, p, ("s", t), self.bar["full_qs"], t, {"do S"})

        vo(0)
        k(0)
        qs(0)
        ds(0)
        if self.lows:
            low(0, 0)
        yield STEP
        free = tails = 0
        for t in range(n):
            self.write(who, self.gates, ("G", t), set(self.A) | set(self.B))
            self.bar["gates"].arrive(t, who)
            yield STEP
            if self.tails[t]:
                for b in ("full_qs", "full_k", "full_vo"):
                    yield self.w(b, t)
                for p, tag in [(self.q, "q"), (self.k, "k"), (self.do, "do")] + [(p, "v") for p in self.v]:
                    self.zero(who, p, (tag, t))
                if "no_fence_tail" not in self.mut:
                    self.fence(who)
                self.bar["tail"].arrive(tails, who)
                tails += 1
                yield STEP
            for i in range(1, self.lows + 1):
                if i == self.lows and t + 1 == n:
                    break
                if "low_no_wait" not in self.mut:
                    yield self.w("low_free", free)
                free += 1
                low(t if i < self.lows else t + 1, i % self.lows)
                yield STEP
            if t + 1 < n:
                yield self.w("dv1_full", t)
                ds(t + 1)
                yield STEP
                yield self.w("dv1_full" if "vo_early" in self.mut else "dv_full", t)
                vo(t + 1)
                yield STEP
                yield self.w("dq_full", t)
                k(t + 1)
                yield STEP
                yield self.w("dq_full" if "qs_early" in self.mut else "out_full", t)
                qs(t + 1)
                yield STEP

    # ---------------------------------------------------------------- warp 1
    def issuer(self):
        who, low_n, tails = "mma", 0, 0
        for t, tail in enumerate(self.tails):
            yield self.w("full_vo", t)
            if tail:
                if "no_tail_wait" not in self.mut:
                    yield self.w("tail", tails)
                tails += 1
            if t:
                yield self.w("dv_read", t - 1)
            vv = [(p, ("v", t)) for p in self.v]
            self.product(who, "t", [(self.do, ("do", t))] + vv, self.tt, None, ("t", t), self.A, False)
            yield self.w("full_ds", t)
            if t:
                yield self.w("dk_read", t - 1)
            # (the sum of the products that reach an accumulator before it is rescaled)
            parts = 0

            def low(place, tag, what, i):
                nonlocal low_n, parts
                yield self.w("low_full", low_n)
                acc, name = (self.tdk, "dk") if i < self.dlows else (self.tdq, "dq")
                self.product(who, what, [(self.low, self.low_tag(t, i))] + [(p, (tag, t)) for p in place],
                             acc, (name, t, parts), (name, t, parts + 1), self.B, True)
                parts += 1
                self.commit(who, self.bar["low_free"], low_n)
                low_n += 1

            if self.hd:
                self.product(who, "v dS", vv + [(self.ds, ("ds", t))], self.tdk, None, ("dk", t, 0), self.B, False)
                if self.dlows:
                    yield from low(self.v, "v", "v dS low0", 0)
            yield self.w("full_k", t)
            yield self.w("full_qs", t)
            self.product(who, "s", [(self.q, ("q", t)), (self.k, ("k", t))], self.ts, None, ("s", t), self.A, False)
            if t:
                yield self.w("dq_read", t - 1)
            if self.hs:
                self.product(who, "do S", [(self.do, ("do", t))] + [(p, ("s", t)) for p in self.s], self.tdq, None,
                             ("dq", t, 0), self.B, False)
            if self.dlows:
                if "first_full_early" in self.mut:
                    self.commit(who, self.bar["first_full"], t)
                yield from low(self.v, "v", "v dS low1", 1)
            if not (self.dlows and "first_full_early" in self.mut):
                self.commit(who, self.bar["first_full"], t)
            kd = parts
            if self.stream and self.hs:
                parts = 0
                for i in range(2):
                    yield from low([self.do], "do", f"do S low{i}", self.dlows + i)
                self.commit(who, self.bar["low_done"], t)
                kq = parts
            else:
                kq = 0
            yield self.w("s_free", t)
            if self.hd:
                self.product(who, "k dS", [(self.k, ("k", t)), (self.ds, ("ds", t))], self.ts, None, ("dv1", t), self.A,
                             False)
            self.commit(who, self.bar["dv1_full"], t)
            yield self.w("p_ready", t)
            self.product(who, "P do", [(p, ("P", t)) for p in self.p] + [(self.do, ("do", t))], self.tt, None,
                         ("dv", t), self.A, False)
            self.commit(who, self.bar["dv_full"], t)
            if "no_scaled_wait" not in self.mut:
                yield self.w("scaled", t)
            dp = [(p, ("dP", t)) for p in self.s]
            self.product(who, "dP k", dp + [(self.k, ("k", t))], self.tdq, ("dq", t, kq, "B0", "B1"), ("dq", t), self.B,
                         self.hs)
            self.commit(who, self.bar["dq_full"], t)
            self.product(who, "dP q", dp + [(self.q, ("q", t))], self.tdk, ("dk", t, kd, "B0", "B1"), ("dk", t), self.A,
                         self.hd)
            self.commit(who, self.bar["out_full"], t)
            yield STEP
        self.commit(who, self.bar["done"], 0)
        yield self.w("done", 0)

    # ---------------------------------------------------------------- group A
    def scores(self, who, i):
        for t in range(len(self.tails)):
            yield self.w("gates", t)
            yield self.w("first_full", t)
            if t and "no_dg_wait" not in self.mut:
                yield self.w("dg_done", t - 1)
            self.read(who, self.gates, ("G", t))
            self.gates.loaded.discard(who)          # ordinary stores come next here, not TMA
            self.read(who, self.ts, ("s", t), smem=False)
            self.read(who, self.tt, ("t", t), smem=False)
            self.bar["s_free"].arrive(t, who)
            yield STEP
            self.write(who, self.p[i], ("P", t), {"P do"})
            self.write(who, self.s[i], ("dP", t), {"dP k", "dP q"})
            self.write(who, self.rc[i], ("W", t), {"dg"})
            if "no_fence_p" not in self.mut:
                self.fence(who)
            self.bar["p_ready"].arrive(t, who)
            yield STEP
            yield self.w("dv_full", t)
            self.read(who, self.tt, ("dv", t), smem=False)
            if self.hd:
                self.read(who, self.ts, ("dv1", t), smem=False)
            self.bar["dv_read"].arrive(t, who)
            yield STEP
            yield self.w("out_full", t)
            self.read(who, self.tdk, ("dk", t), smem=False)
            self.bar["dk_read"].arrive(t, who)
            yield STEP

    # ---------------------------------------------------------------- group B
    def first_terms(self, who, i):
        tails = 0
        for t, tail in enumerate(self.tails):
            for b in ("gates", "full_qs", "full_k", "first_full"):
                yield self.w(b, t)
            if tail:
                yield self.w("tail", tails)
                tails += 1
            if t:
                yield self.w("dg_done", t - 1)
            self.read(who, self.gates, ("G", t))
            self.gates.loaded.discard(who)
            if self.hd:
                self._scale(who, self.tdk, "dk", t, self.dlows)
                self.read(who, self.k, ("k", t), zeroed=True)
            yield STEP
            if self.hs:
                if self.stream and "no_low_wait" not in self.mut:
                    yield self.w("low_done", t)
                self._scale(who, self.tdq, "dq", t, self.lows - self.dlows)
                self.read(who, self.q, ("q", t), zeroed=True)
            self.write(who, self.re[i], ("R", t), {"dg"})
            self.re[i].stored.discard(who)          # read by ordinary loads
            if "no_fence_b" not in self.mut:
                self.fence(who)
            self.bar["scaled"].arrive(t, who)
            yield STEP
            yield self.w("dq_full", t)
            self.read(who, self.tdq, ("dq", t), smem=False)
            self.bar["dq_read"].arrive(t, who)
            yield STEP

    def _scale(self, who, acc, name, t, lows):
        """Each of the group's agents rescales its rows; the tag collects who has."""
        want = (name, t, lows)
        tag = acc.tag if isinstance(acc.tag, tuple) else ()
        if tag[:3] != want or who in tag or acc.busy():
            raise ProtocolError(f"{who}: rescales {acc.name} holding {acc.tag}, wants {want}, at rest")
        acc.tag = want + tuple(sorted(tag[3:] + (who,)))
        acc.need.discard(who)

    def dg(self):
        for t in range(len(self.tails)):
            yield self.w("p_ready", t)
            yield self.w("scaled", t)
            for p in self.rc:
                self.read("dg", p, ("W", t))
                p.loaded.discard("dg")
                p.stored.clear()
            for p in self.re:
                self.read("dg", p, ("R", t))
                p.loaded.discard("dg")
            self.bar["dg_done"].arrive(t, "dg")
            yield STEP


class StateModel(Engine):
    """One (segment, head, slice) of ``nb`` blocks.  ``slots``: slices in shared memory at once (2 for the
    reverse scan at D = 128); ``through``: the reverse scan's reads of the forward snapshots."""

    ISSUERS = ("mma",)
    E, S = ("E0", "E1"), ("S0", "S1", "S2", "S3")

    def __init__(self, nb, tail=False, slots=3, through=False, snap=True, mutations=()):
        super().__init__(mutations)
        self.nb, self.tail, self.slots, self.through, self.snap = nb, tail, slots, through, snap
        self.places = []
        self.a = [[self.place(f"tile{i}.{u}") for u in range(4)] for i in range(3)]
        self.b = [[self.place(f"slice{i}.{u}") for u in range(4)] for i in range(slots)]
        self.parts = [self.place(f"parts.{u}") for u in range(4)]
        self.acc = [self.place(f"acc{i}") for i in range(2)]
        self.other = self.place("other")
        self.out = [self.place(f"out.{i}") for i in range(2)]
        self.g = [self.place(f"sums{i}") for i in range(2)]
        B = Barrier
        self.full, self.empty = [B(f"full{i}", 1) for i in range(3)], [B(f"empty{i}", 1) for i in range(3)]
        self.ready, self.pfree = [B(f"ready{u}", 1) for u in range(4)], [B(f"parts_free{u}", 1) for u in range(4)]
        self.afull, self.afree = [B(f"acc_full{i}", 1) for i in range(2)], [B(f"acc_free{i}", 2) for i in range(2)]
        self.ofull, self.ofree, self.done = B("other_full", 1), B("other_free", 2), B("done", 1)
        self.gready, self.gfree = [B(f"gates_ready{i}", 1) for i in range(2)], [B(f"gates_free{i}", 6) for i in range(2)]
        self.named = B("named", 2)
        self.roles = {"load": self.loader(), "mma": self.issuer(), "gates": self.gates()}
        if through:
            self.roles["other"] = self.others()
        self.roles.update({e: self.epilogue(e, i) for i, e in enumerate(self.E)})
        self.roles.update({s: self.scaling(s, u) for u, s in enumerate(self.S)})

    def partial(self, t):
        return self.tail and t == (0 if self.through else self.nb - 1)   # the reverse scan meets it first

    def loader(self):
        who = "load"
        for t in range(self.nb):
            if t >= 3:
                yield ("wait", self.empty[t % 3], t // 3 - 1)
            f = self.full[t % 3]
            f.arrive(t // 3, who, 8)
            for u, p in enumerate(self.a[t % 3]):
                self.load(who, p, ("a", t), f, t // 3, {f"product{u}"}, not self.partial(t))
            yield STEP
            if self.slots < 3 and t >= 2 and "slice_no_wait" not in self.mut:
                yield ("wait", self.empty[(t - 2) % 3], (t - 2) // 3)
            for u, p in enumerate(self.b[t % self.slots]):
                self.load(who, p, ("b", t), f, t // 3, {self.S[u]}, not self.partial(t))
            yield STEP
        for t in range(max(0, self.nb - 3), self.nb):
            yield ("wait", self.full[t % 3], t // 3)

    def issuer(self):
        who = "mma"
        for t in range(self.nb):
            yield ("wait", self.full[t % 3], t // 3)
            if t >= 2 and "no_acc_free" not in self.mut:
                yield ("wait", self.afree[t & 1], (t - 2) >> 1)
            for u in range(4):
                yield ("wait", self.ready[u], t)
                self.product(who, f"product{u}", [(self.a[t % 3][u], ("a", t)), (self.b[t % self.slots][u], ("part0", t)),
                                                  (self.parts[u], ("parts", t))],
                             self.acc[t & 1], ("acc", t, u), ("acc", t, u + 1), self.E, u > 0)
                self.commit(who, self.pfree[u], t)
            self.commit(who, self.empty[t % 3], t // 3)
            self.commit(who, self.afull[t & 1], t >> 1)
            yield STEP
        self.commit(who, self.done, 0)
        yield ("wait", self.done, 0)

    def gates(self):
        for t in range(self.nb):
            if t >= 2 and "gates_no_wait" not in self.mut:
                yield ("wait", self.gfree[t & 1], (t - 2) >> 1)
            self.write("gates", self.g[t & 1], ("G", t), set(self.E) | set(self.S))
            self.g[t & 1].stored.clear()
            self.gready[t & 1].arrive(t >> 1, "gates")
            yield STEP

    def _gate(self, who, t):
        self.read(who, self.g[t & 1], ("G", t))
        self.g[t & 1].loaded.discard(who)

    def others(self):
        who = "other"
        for t in range(self.nb):
            if t >= 1:
                yield ("wait", self.ofree, t - 1)
            self.ofull.arrive(t, who, 1)
            self.load(who, self.other, ("other", t), self.ofull, t, self.E)
            yield STEP
        if self.nb:
            yield ("wait", self.ofull, self.nb - 1)

    def epilogue(self, who, i):
        meet = 0
        for t in range(self.nb):
            yield ("wait", self.gready[t & 1], t >> 1)
            self._gate(who, t)
            self.gfree[t & 1].arrive(t >> 1, who)
            yield STEP
            if self.through:
                yield ("wait", self.ofull, t)
                self.read(who, self.other, ("other", t))
                if "no_fence_other" not in self.mut:
                    self.fence(who)
                self.ofree.arrive(t, who)
                yield STEP
            if self.snap:
                if i == 0 and "no_store_wait" not in self.mut:
                    yield from self.stores_read(who)
                self.named.arrive(meet, who)
                yield ("wait", self.named, meet)
                meet += 1
                self.write(who, self.out[i], ("snap", t), {"E0"})
                if "no_fence_snap" not in self.mut:
                    self.fence(who)
                self.named.arrive(meet, who)
                yield ("wait", self.named, meet)
                meet += 1
                if i == 0:
                    self.tma_store(who, self.out, ("snap", t))
                    yield STEP
            yield ("wait", self.afull[t & 1], t >> 1)
            self.read(who, self.acc[t & 1], ("acc", t, 4), smem=False)
            self.afree[t & 1].arrive(t >> 1, who)
            yield STEP
        if i == 0:
            yield from self.stores_read(who)

    def scaling(self, who, u):
        for t in range(self.nb):
            yield ("wait", self.gready[t & 1], t >> 1)
            yield ("wait", self.full[t % 3], t // 3)
            if t >= 1 and "no_parts_wait" not in self.mut:
                yield ("wait", self.pfree[u], t - 1)
            self._gate(who, t)
            self.read(who, self.b[t % self.slots][u], ("b", t))
            self.write(who, self.b[t % self.slots][u], ("part0", t), {f"product{u}"})
            self.write(who, self.parts[u], ("parts", t), {f"product{u}"})
            if self.partial(t):
                self.zero(who, self.a[t % 3][u], ("a", t))
            if "no_fence_parts" not in self.mut:
                self.fence(who)
            self.ready[u].arrive(t, who)
            self.gfree[t & 1].arrive(t >> 1, who)
            yield STEP


class PrefillModel(Engine):
    """One (segment, head, slice) of ``nb`` blocks of the prefill kernel."""

    ISSUERS = ("mma_s", "mma_o", "mma_kv")
    KV, P, O, V = ("KV0", "KV1"), ("P0", "P1"), ("O0", "O1"), ("V0", "V1", "V2", "V3")

    def __init__(self, nb, tail=False, mutations=()):
        super().__init__(mutations)
        self.nb, self.tail = nb, tail
        self.places = []

        def ring(n, k):
            return [[self.place(f"{n}{i}.{u}") for u in range(k)] for i in range(2)]
        self.q, self.k, self.v, self.s = ring("q", 1), ring("k", 4), ring("v", 2), ring("scores", 2)
        self.vp = [self.place(f"v'.{u}") for u in range(4)]
        self.snap = [self.place(f"snap{i}") for i in range(2)]
        self.g = [self.place(f"sums{i}") for i in range(2)]
        self.qs, self.pv, self.kv = self.place("qS"), self.place("Pv"), self.place("kv")
        B = Barrier

        def two(n, c):
            return [B(f"{n}{i}", c) for i in range(2)]
        self.full = {n: two(f"full_{n}", 1) for n in "qkv"}
        self.empty = {"q": two("empty_q", 2), "k": two("empty_k", 2), "v": two("empty_v", 2)}
        self.s_full, self.p_ready, self.o_free = two("s_full", 1), two("p_ready", 2), two("o_free", 2)
        self.v_split, self.g_ready, self.g_free = two("v_split", 4), two("gates_ready", 1), two("gates_free", 10)
        self.v_ready, self.v_free = [B(f"v_ready{u}", 1) for u in range(4)], [B(f"v_free{u}", 1) for u in range(4)]
        self.tailz, self.done = B("tail_zeroed", 4), B("done", 3)
        self.kv_full, self.kv_free = B("kv_full", 1), B("kv_free", 2)
        self.snap_ready, self.qs_done, self.o_full = B("snap_ready", 2), B("qs_done", 1), B("o_full", 1)
        self.roles = {"load": self.loader(), "mma_s": self.scores(), "mma_o": self.outputs(), "mma_kv": self.states()}
        self.roles.update({a: self.group_kv(a, i) for i, a in enumerate(self.KV)})
        self.roles.update({a: self.group_p(a, i) for i, a in enumerate(self.P)})
        self.roles.update({a: self.group_o(a, i) for i, a in enumerate(self.O)})
        self.roles.update({a: self.group_v(a, u) for u, a in enumerate(self.V)})

    def partial(self, b):
        return self.tail and b == self.nb - 1

    def _gate(self, who, b):
        self.read(who, self.g[b & 1], ("G", b))
        self.g[b & 1].loaded.discard(who)

    def loader(self):
        who = "load"
        for b in range(self.nb):
            i, n, z = b & 1, b >> 1, not self.partial(b)
            for name, ring, need in (("k", self.k, lambda u: {"s", f"kv{u}"}), ("q", self.q, lambda u: {"s", "qs"}),
                                     ("v", self.v, lambda u: {"pv", f"V{2 * u}", f"V{2 * u + 1}"})):
                if b >= 2 and f"{name}_no_wait" not in self.mut:
                    yield ("wait", self.empty[name][i], n - 1)
                self.full[name][i].arrive(n, who, len(ring[i]))
                for u, p in enumerate(ring[i]):
                    self.load(who, p, (name, b), self.full[name][i], n, need(u), z)
                yield STEP
            if b >= 2:
                yield ("wait", self.g_free[i], n - 1)
            self.write(who, self.g[i], ("G", b), set(self.KV + self.P + self.O + self.V))
            self.g[i].stored.clear()
            self.g_ready[i].arrive(n, who)
            yield STEP
        for name in "kqv":
            for b in range(max(0, self.nb - 2), self.nb):
                yield ("wait", self.full[name][b & 1], b >> 1)

    def scores(self):
        who = "mma_s"
        for b in range(self.nb):
            i, n = b & 1, b >> 1
            yield ("wait", self.full["k"][i], n)
            yield ("wait", self.full["q"][i], n)
            if b >= 2 and "no_o_free" not in self.mut:
                yield ("wait", self.o_free[i], n - 1)
            # (rows behind the sequence may hold anything: the mask drops what they give)
            reads = [(p, ("q", b)) for p in self.q[i]] + [(p, ("k", b)) for p in self.k[i]]
            for w in range(2):
                self._scores(who, reads if w == 0 else [], self.s[i][w], b, self.P[w])
            self.commit(who, self.s_full[i], n)
            self.commit(who, self.empty["q"][i], n)
            self.commit(who, self.empty["k"][i], n)
            yield STEP
        self.commit(who, self.done, 0)
        yield ("wait", self.done, 0)

    def _scores(self, who, reads, acc, b, reader):
        for p, _ in reads:
            p.stored_before = set(p.stored)
            p.stored.clear()                        # group V may be zeroing k's last rows meanwhile
        self.product(who, "s", reads, acc, None, ("S", b), {reader}, False, zeroed=False)
        for p, _ in reads:
            p.stored |= p.stored_before

    def outputs(self):
        who = "mma_o"
        for b in range(self.nb):
            i, n = b & 1, b >> 1
            yield ("wait", self.full["q"][i], n)
            yield ("wait", self.snap_ready, b)
            if b >= 1 and "no_o_free2" not in self.mut:
                yield ("wait", self.o_free[(b - 1) & 1], (b - 1) >> 1)
            self.product(who, "qs", [(p, ("q", b)) for p in self.q[i]] + [(p, ("snap", b)) for p in self.snap], self.qs,
                         None, ("qS", b), self.O, False, zeroed=False)
            self.commit(who, self.qs_done, b)
            self.commit(who, self.empty["q"][i], n)
            yield STEP
            yield ("wait", self.full["v"][i], n)
            yield ("wait", self.p_ready[i], n)
            if self.partial(b) and "no_tail_wait" not in self.mut:
                yield ("wait", self.tailz, 0)
            self.product(who, "pv", [(p, ("P", b)) for p in self.s[i]] + [(p, ("v", b)) for p in self.v[i]], self.pv, None,
                         ("Pv", b), self.O, False)
            self.commit(who, self.o_full, b)
            yield STEP
        self.commit(who, self.done, 0)
        yield ("wait", self.done, 0)

    def states(self):
        who = "mma_kv"
        for b in range(self.nb):
            i, n = b & 1, b >> 1
            yield ("wait", self.full["k"][i], n)
            if b >= 1 and "no_kv_free" not in self.mut:
                yield ("wait", self.kv_free, b - 1)
            for u in range(4):
                yield ("wait", self.v_ready[u], b)
                self.product(who, f"kv{u}", [(self.k[i][u], ("k", b)), (self.vp[u], ("v'", b))], self.kv, ("kv", b, u),
                             ("kv", b, u + 1), self.KV, u > 0)
                self.commit(who, self.v_free[u], b)
                yield STEP
            self.commit(who, self.kv_full, b)
            self.commit(who, self.empty["k"][i], n)
        self.commit(who, self.done, 0)
        yield ("wait", self.done, 0)

    def group_kv(self, who, i):
        def snapshot(b):
            self.write(who, self.snap[i], ("snap", b), {"qs"})
            if "no_fence_snap" not in self.mut:
                self.fence(who)
            self.snap_ready.arrive(b, who)
        if self.nb:
            snapshot(0)
            yield STEP
        for b in range(self.nb):
            yield ("wait", self.g_ready[b & 1], b >> 1)
            self._gate(who, b)
            self.g_free[b & 1].arrive(b >> 1, who)
            yield STEP
            yield ("wait", self.kv_full, b)
            self.read(who, self.kv, ("kv", b, 4), smem=False)
            self.kv_free.arrive(b, who)
            yield STEP
            if b + 1 < self.nb:
                if "no_qs_wait" not in self.mut:
                    yield ("wait", self.qs_done, b)
                snapshot(b + 1)
                yield STEP

    def group_p(self, who, w):
        for b in range(self.nb):
            yield ("wait", self.g_ready[b & 1], b >> 1)
            yield ("wait", self.s_full[b & 1], b >> 1)
            self._gate(who, b)
            p = self.s[b & 1][w]
            self.read(who, p, ("S", b), smem=False)
            self.write(who, p, ("P", b), {"pv"}, smem=False)
            self.p_ready[b & 1].arrive(b >> 1, who)
            self.g_free[b & 1].arrive(b >> 1, who)
            yield STEP

    def group_o(self, who, w):
        for b in range(self.nb):
            i, n = b & 1, b >> 1
            yield ("wait", self.g_ready[i], n)
            self._gate(who, b)
            self.g_free[i].arrive(n, who)
            yield STEP
            yield ("wait", self.o_full, b)
            if "no_split_wait" not in self.mut:
                yield ("wait", self.v_split[i], n)
            self.read(who, self.qs, ("qS", b), smem=False)
            self.read(who, self.pv, ("Pv", b), smem=False)
            p = self.v[i][w]
            self.write(who, p, ("o", b), {who})
            self.o_free[i].arrive(n, who)
            yield STEP
            if self.partial(b):
                self.read(who, p, ("o", b))         # the last rows leave by ordinary stores; no load follows
            else:
                if "no_fence_o" not in self.mut:
                    self.fence(who)
                self.tma_store(who, [p], ("o", b))
                if "no_read_wait" not in self.mut:
                    yield from self.stores_read(who)
            self.empty["v"][i].arrive(n, who)
            yield STEP
        yield from self.stores_read(who)

    def group_v(self, who, u):
        for b in range(self.nb):
            i, n = b & 1, b >> 1
            yield ("wait", self.g_ready[i], n)
            yield ("wait", self.full["v"][i], n)
            if b >= 1 and "no_v_free" not in self.mut:
                yield ("wait", self.v_free[u], b - 1)
            p = self.v[i][u >> 1]
            if self.partial(b):
                yield ("wait", self.full["k"][i], n)
                p.zeroed_by = getattr(p, "zeroed_by", 0) + 1
                self._holds(who, p, ("v", b), "zeroing", zeroed=False)
                p.stored.add(who)
                p.zeroed = p.zeroed_by == 2         # by the two warps whose rows these are
                self.zero(who, self.k[i][u], ("k", b))
                if "no_fence_tail" not in self.mut:
                    self.fence(who)
                self.tailz.arrive(0, who)
                yield STEP
            self._gate(who, b)
            self.read(who, p, ("v", b))
            self.write(who, self.vp[u], ("v'", b), {f"kv{u}"})
            if "no_fence_v" not in self.mut:
                self.fence(who)
            self.v_ready[u].arrive(b, who)
            self.g_free[i].arrive(n, who)
            self.v_split[i].arrive(n, who)
            yield STEP
