"""A randomized model of the synchronisation of the serving operators'
tensor-core kernel, attend_tc_kernel (csrc/serving_tc.cu), checked on the CPU
for what would hang or corrupt it on the GPU: a waiter that misses an mbarrier
phase, a deadlock, or a copy, MMA, softmax, guard or output step that touches
data out of order.

One block walks a list of pieces.  The roles and barriers follow the kernel one
to one (barriers and their parity rule are test_tc_sync_model.Bar):
  producer  publishes piece k (work_full) after piece k - 2 is done, loads its Q
            after the previous piece's last Q K^T (q_empty), then K and V tiles
            through two stages each; V tiles with masked keys complete on
            vg_full instead of v_full;
  guard     (two warps) checks those tiles in place, arrives v_ready; noted
            after a piece's last one;
  issuer    Q K^T and P V in the kernel's order (two row tiles share every key
            tile; one row tile: the warpgroups take alternate key tiles), the
            first P V of a piece after the piece before is done;
  softmax t waits S_t, writes P over it (p_full); after its last tile reads O
            (one row tile: both O's, after exchanging maxima through ml_full),
            then done.
Copy, MMA and role latencies are random; pieces have random tile counts, from
none on.  Planted mistakes must be caught.
"""
import heapq
import random

import pytest

from test_tc_sync_model import Bar


class Fail(AssertionError):
    pass


class Model:
    def __init__(self, seed, pieces, mutation=None):
        self.rng, self.pieces, self.mutation = random.Random(seed), pieces, mutation
        self.time, self.queue, self.n = 0, [], 0
        self.pipe_free = 0
        two = {"k_full": 1, "k_empty": 1, "v_full": 1, "v_empty": 1, "vg_full": 1, "v_ready": 2, "s_full": 1, "p_full": 4,
               "o_final": 1, "noted": 2, "done": 8, "work_full": 1}
        self.bars = {f"{b}{i}": Bar(f"{b}{i}", c) for b, c in two.items() for i in (0, 1)}
        self.bars |= {b: Bar(b, 1) for b in ("q_full", "q_empty")}
        self.bars |= {f"ml_full{i}{t}": Bar(f"ml_full{i}{t}", 4) for i in (0, 1) for t in (0, 1)}
        self.work = [None, None]
        self.q = None                      # piece whose Q is in shared memory
        self.k, self.v = [None, None], [None, None]    # (piece, tile) landed in each stage
        self.v_checked = [None, None]
        self.k_use, self.v_use, self.q_use = [0, 0], [0, 0], 0
        self.s = [None, None]              # ("S" or "P", piece, tile)
        self.o = [None, None]              # piece whose sum O_t holds
        self.o_left = [0, 0]               # warpgroups that have to read it yet
        self.o_busy = [0, 0]
        self.notes = [None, None]          # piece whose notes a buffer holds
        self.notes_read = [0, 0]
        self.ml = [[None, None], [None, None]]
        self.finished = 0

    def at(self, dt, fn):
        self.n += 1
        heapq.heappush(self.queue, (self.time + dt, self.n, fn))

    def check(self, ok, what):
        if not ok:
            raise Fail(what)

    def wait(self, bar, phase):
        while not self.bars[bar].ready(phase):
            yield self.rng.randint(1, 40)

    def arrive(self, bar, n=1):
        self.bars[bar].arrive(n)

    # ------------------------------------------------------------ hardware
    def copy(self, bar, land, busy):
        self.check(busy() == 0, f"copy into memory that {busy()} MMAs still read ({bar})")
        self.bars[bar].arrive(expect_tx=1)

        def done():
            land()
            self.bars[bar].complete_tx(1)
        self.at(self.rng.randint(1, 400), done)

    def mma(self, start, end):
        begin = max(self.time, self.pipe_free)
        self.pipe_free = begin + self.rng.randint(10, 60)
        self.at(begin - self.time, start)
        self.at(self.pipe_free - self.time, end)

    def commit(self, bar):
        self.at(max(self.time, self.pipe_free) - self.time + self.rng.randint(0, 3), lambda: self.arrive(bar))

    # --------------------------------------------------------------- roles
    def item(self, k):
        if k >= len(self.pieces):
            return None
        n, two, n0, g0 = self.pieces[k]
        return dict(n=n, two=two, nt=(n0, n) if two else ((n + 1) // 2, n // 2), g0=g0)

    def get(self, k, who):
        yield from self.wait(f"work_full{k & 1}", k >> 1)
        self.check(self.work[k & 1] == k, f"{who} reads piece {self.work[k & 1]} for {k}")

    def producer(self):
        tile = 0
        for k in range(len(self.pieces) + 1):
            if k >= 2 and self.mutation != "publish early":
                yield from self.wait(f"done{k & 1}", (k >> 1) - 1)
            self.work[k & 1] = k
            self.arrive(f"work_full{k & 1}")
            it = self.item(k)
            if it is None:
                return
            if k > 0 and self.mutation != "q early":
                yield from self.wait("q_empty", k - 1)
            self.q = None

            def q_land(k=k):
                self.q = k
            self.copy("q_full", q_land, lambda: self.q_use)
            for j in range(it["n"]):
                st = tile & 1
                for what, use, data in (("k", self.k_use, self.k), ("v", self.v_use, self.v)):
                    if tile >= 2:
                        yield from self.wait(f"{what}_empty{st}", (tile >> 1) - 1)
                    data[st] = None
                    if what == "v":
                        self.v_checked[st] = None
                    bar = f"k_full{st}" if what == "k" else (f"vg_full{st}" if j >= it["g0"] else f"v_full{st}")

                    def land(data=data, st=st, k=k, j=j):
                        data[st] = (k, j)
                    self.copy(bar, land, lambda use=use, st=st: use[st])
                    yield self.rng.randint(1, 20)
                tile += 1
            yield self.rng.randint(1, 60)

    def guard(self, w):
        tile, ph = 0, [0, 0]
        for k in range(len(self.pieces) + 1):
            yield from self.get(k, "guard")
            it = self.item(k)
            if it is None:
                return
            b = k & 1
            if self.notes[b] != k:
                self.check(self.notes[b] is None or self.notes_read[b] == 8, f"notes of piece {self.notes[b]} overwritten by {k}")
                self.notes[b], self.notes_read[b] = k, 0
            for j in range(it["g0"], it["n"]):
                st = (tile + j) & 1
                yield from self.wait(f"vg_full{st}", ph[st])
                ph[st] += 1
                self.check(self.v[st] == (k, j), f"guard sees {self.v[st]} for {(k, j)}")
                yield self.rng.randint(1, 80)
                self.v_checked[st] = (k, j)
                self.arrive(f"v_ready{st}")
            tile += it["n"]
            self.arrive(f"noted{b}")

    def qk(self, t, k, j, st):
        def start():
            self.check(self.k[st] == (k, j), f"Q K^T of {(k, j)} reads K {self.k[st]}")
            self.check(self.q == k, f"Q K^T of piece {k} reads Q of {self.q}")
            self.check(self.s[t] is None or self.s[t][0] == "free", f"S_{t} of {(k, j)} written over {self.s[t]}")
            self.s[t] = None

        def end():
            self.s[t] = ("S", k, j)
            self.k_use[st] -= 1
            self.q_use -= 1
        self.k_use[st] += 1
        self.q_use += 1
        self.mma(start, end)
        self.commit(f"s_full{t}")

    def pv(self, t, k, j, st, guarded, first):
        def start():
            self.check(self.v[st] == (k, j), f"P V of {(k, j)} reads V {self.v[st]}")
            self.check(not guarded or self.v_checked[st] == (k, j), f"P V of {(k, j)} before its guard")
            self.check(self.s[t] == ("P", k, j), f"P V of {(k, j)} reads {self.s[t]}")
            if first:
                self.check(self.o_left[t] == 0, f"O_{t} of piece {self.o[t]} overwritten by {k} before it was read")
                self.o[t], self.o_left[t] = k, 1 if self.item(k)["two"] else 2
            self.check(self.o[t] == k, f"O_{t}")

        def end():
            self.s[t] = ("free",)
            self.v_use[st] -= 1
            self.o_busy[t] -= 1
        self.v_use[st] += 1
        self.o_busy[t] += 1
        self.mma(start, end)

    def issuer(self):
        tile, pp, pv_, pg = 0, [0, 0], [0, 0], [0, 0]
        for k in range(len(self.pieces) + 1):
            yield from self.get(k, "issuer")
            it = self.item(k)
            if it is None:
                return
            n, nt, g0 = it["n"], it["nt"], it["g0"]
            yield from self.wait("q_full", k)

            def wait_k(x):
                yield from self.wait(f"k_full{x & 1}", x >> 1)

            def wait_v(j):
                st = (tile + j) & 1
                c, bar = (pv_, "v_full") if j < g0 else (pg, "v_ready")
                yield from self.wait(f"{bar}{st}", c[st])
                c[st] += 1

            def wait_p(t):
                yield from self.wait(f"p_full{t}", pp[t])
                pp[t] += 1

            def wait_o():
                if k > 0 and self.mutation != "no wait for O":
                    yield from self.wait(f"done{(k - 1) & 1}", (k - 1) >> 1)
            if n == 0:
                self.commit("q_empty")
            elif it["two"]:
                yield from wait_k(tile)
                for t in (0, 1):
                    if nt[t] > 0:
                        self.qk(t, k, 0, tile & 1)
                self.commit(f"k_empty{tile & 1}")
                if n == 1:
                    self.commit("q_empty")
                for j in range(n):
                    st, st1 = (tile + j) & 1, (tile + j + 1) & 1
                    yield from wait_v(j)
                    if j + 1 < n:
                        yield from wait_k(tile + j + 1)
                    if j == 0:
                        yield from wait_o()
                    for t in (0, 1):
                        if j < nt[t]:
                            yield from wait_p(t)
                            self.pv(t, k, j, st, j >= g0, j == 0)
                            if j == nt[t] - 1:
                                self.commit(f"o_final{t}")
                        if t == 1:
                            self.commit(f"v_empty{st}")
                        if j + 1 < nt[t]:
                            self.qk(t, k, j + 1, st1)
                        yield self.rng.randint(1, 30)
                    if j + 1 < n:
                        self.commit(f"k_empty{st1}")
                        if j + 2 == n:
                            self.commit("q_empty")
            else:
                for j in range(min(n, 2)):
                    yield from wait_k(tile + j)
                    self.qk(j, k, j, (tile + j) & 1)
                    self.commit(f"k_empty{(tile + j) & 1}")
                if n <= 2:
                    self.commit("q_empty")
                for j in range(n):
                    t, st = j & 1, (tile + j) & 1
                    yield from wait_v(j)
                    if j + 2 < n:
                        yield from wait_k(tile + j + 2)
                    if j == 0:
                        yield from wait_o()
                    yield from wait_p(t)
                    self.pv(t, k, j, st, j >= g0, j < 2)
                    if j + 2 >= n:
                        self.commit(f"o_final{t}")
                    if self.mutation != "no v_empty" or k < 12:
                        self.commit(f"v_empty{st}")
                    if j + 2 < n:
                        self.qk(t, k, j + 2, st)
                        self.commit(f"k_empty{st}")
                        if j + 3 == n:
                            self.commit("q_empty")
                    yield self.rng.randint(1, 30)
            tile += n

    def softmax(self, t):
        ns, own, oth, nml = 0, 0, 0, [0, 0]
        for k in range(len(self.pieces) + 1):
            yield from self.get(k, f"softmax {t}")
            it = self.item(k)
            if it is None:
                return
            my, other = it["nt"][t], it["nt"][1 - t]
            for i in range(my):
                j = i if it["two"] else 2 * i + t
                yield from self.wait(f"s_full{t}", ns)
                ns += 1
                self.check(self.s[t] == ("S", k, j), f"softmax {t} reads {self.s[t]} for {(k, j)}")
                yield self.rng.randint(1, 300)
                self.check(self.o_busy[t] == 0, f"O_{t} rescaled while a P V adds to it")
                self.s[t] = ("P", k, j)
                self.arrive(f"p_full{t}", 4)
            yield from self.wait(f"noted{k & 1}", k >> 1)
            self.check(self.notes[k & 1] == k, "notes of another piece")
            self.check(self.work[k & 1] == k, f"the slot of piece {k} was taken early")
            if not it["two"]:
                b = 0 if self.mutation == "one exchange" else k & 1
                self.ml[b][t] = k
                self.arrive(f"ml_full{b}{t}", 4)
                yield from self.wait(f"ml_full{b}{1 - t}", nml[b])
                nml[b] += 1
                self.check(self.ml[b][1 - t] == k, "maxima of another piece")
            if my:
                yield from self.wait(f"o_final{t}", own)
            if not it["two"] and other:
                yield from self.wait(f"o_final{1 - t}", oth)
            own += my > 0
            oth += other > 0
            for u in ((t,) if it["two"] else (0, 1)):
                if it["nt"][u]:
                    self.check(self.o[u] == k and self.o_busy[u] == 0, f"O_{u} read for {k} holds {self.o[u]}")
            yield self.rng.randint(1, 400)
            for u in ((t,) if it["two"] else (0, 1)):
                if it["nt"][u]:
                    self.check(self.o[u] == k, f"O_{u} changed while it was read")
            self.notes_read[k & 1] += 4
            self.finished += 1
            for u in ((t,) if it["two"] else (0, 1)):
                if it["nt"][u]:
                    self.o_left[u] -= 1
            self.arrive(f"done{k & 1}", 4)

    def run(self):
        def drive(gen):
            def step():
                try:
                    dt = next(gen)
                except StopIteration:
                    self.left -= 1
                    return
                self.at(dt, step)
            return step
        roles = [self.producer(), self.issuer(), self.guard(0), self.guard(1), self.softmax(0), self.softmax(1)]
        self.left = len(roles)
        for g in roles:
            self.at(self.rng.randint(0, 50), drive(g))
        for _ in range(400000):
            if not self.queue:
                break
            self.time, _, fn = heapq.heappop(self.queue)
            fn()
            if self.left == 0 and not self.queue:
                break
        self.check(self.left == 0, "deadlock")
        self.check(self.finished == 2 * len(self.pieces), "pieces left")


def random_pieces(rng):
    out = []
    for _ in range(rng.randint(1, 7)):
        n, two = rng.choice([0, 1, 1, 2, 3, 4, 7]), rng.random() < 0.5
        out.append((n, two, rng.randint(max(0, n - 3), n), rng.randint(0, n)))
    return out


@pytest.mark.parametrize("seed", range(120))
def test_protocol_holds(seed):
    Model(seed, random_pieces(random.Random(1000 + seed))).run()


def test_many_short_pieces():
    for seed in range(20):
        Model(seed, [(seed % 3, bool((seed + i) % 2), seed % 3, 0) for i in range(25)]).run()


@pytest.mark.parametrize("mutation", ["publish early", "q early", "no wait for O", "no v_empty", "one exchange"])
def test_planted_mistakes_are_caught(mutation):
    caught = 0
    for seed in range(60):
        pieces = [(0, False, 0, 0)] * 12 + [(3, False, 3, 1)] + random_pieces(random.Random(seed)) + [(1, True, 1, 0), (2, True, 2, 0), (4, False, 4, 2)]
        try:
            Model(seed, pieces, mutation).run()
        except AssertionError:
            caught += 1
    assert caught > 0
