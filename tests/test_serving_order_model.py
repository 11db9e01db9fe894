"""Memory order in the serving operators' tensor-core kernel, attend_tc_kernel
(csrc/serving_tc.cu): a race detector over the randomized protocol model of
test_serving_sync_model.

Every role has a vector clock.  An ordinary mbarrier arrival releases it (into
the phase that the arrival counts for) and a wait acquires that phase's; a
relaxed arrival, the completion of a copy and the commit of MMAs carry none.
The locations are those that roles read and write as ordinary memory and use
again for a later piece: `work` (a piece as its roles see it), the notes of
non-finite V (`first`, `odd`), the exchanged maxima and sums (`ml`), and the rows
to which a long piece's O is folded (here with every tile).  A write must come after all earlier reads and writes of the location
by other roles in the order that the clocks give, a read after its last write.
"""
import heapq
import os
import random
import re

import pytest

from test_serving_sync_model import Fail, Model, random_pieces

SRC = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "long_context_blockwise_max_b200", "csrc", "serving_tc.cu")).read()


def kernel_hands_reads_back():
    """Whether the kernel's roles return what they have read by ordinary
    arrivals (the eight softmax warps, and the issuer) that the producer waits for."""
    return (re.search(r"mbar_init\(&bars->read\[s\], 9\);", SRC) is not None
            and SRC.count("mbar_arrive(&bars->read[k & 1]);") == 2
            and "wait(&bars->read[k & 1], (k >> 1) - 1)" in SRC)


class Slots(list):
    """A list whose assignments are writes by the role at work."""

    def __init__(self, model, name, n):
        super().__init__([None] * n)
        self.model, self.name = model, name

    def __setitem__(self, i, value):
        self.model.wrote((self.name, i))
        super().__setitem__(i, value)


class OrderModel(Model):
    def __init__(self, seed, pieces, hands_back=True, mutation=None):
        super().__init__(seed, pieces)
        self.hands_back, self.plant = hands_back, mutation
        self.work, self.notes = Slots(self, "work", 2), Slots(self, "notes", 2)
        self.ml = [Slots(self, f"ml{b}", 2) for b in (0, 1)]
        self.fold = [Slots(self, f"fold{b}", 2) for b in (0, 1)]
        Bar = type(self.bars["q_full"])
        for i in (0, 1):
            self.bars[f"read{i}"] = Bar(f"read{i}", 8 if mutation == "issuer not counted" else 9)
        self.role = None
        self.clock = {}          # role -> {role: time}
        self.phase = {}          # (barrier, phase) -> {role: time}
        self.last_write, self.reads = {}, {}
        self.checked = 0

    # ------------------------------------------------------------- the clocks
    def now(self):
        return self.clock.setdefault(self.role, {})

    def tick(self):
        c = self.now()
        c[self.role] = c.get(self.role, 0) + 1
        return c[self.role]

    def merge(self, into, other):
        for r, t in other.items():
            into[r] = max(into.get(r, 0), t)

    def after(self, role, t):
        return role == self.role or self.now().get(role, 0) >= t

    def wrote(self, where):
        t = self.tick()
        for role, at in self.reads.pop(where, {}).items():
            self.check(self.after(role, at), f"{self.role} writes {where}, and nothing orders that behind {role}'s read")
        if where in self.last_write:
            self.check(self.after(*self.last_write[where]), f"{self.role} and {self.last_write[where][0]} both write {where}")
        self.last_write[where] = (self.role, t)
        self.checked += 1

    def saw(self, where):
        self.check(where in self.last_write, f"{self.role} reads {where} before it is written")
        self.check(self.after(*self.last_write[where]), f"{self.role} reads {where}: not ordered behind its write")
        self.reads.setdefault(where, {})[self.role] = self.tick()

    # --------------------------------------------------------- the operations
    def release(self, bar, n=1):
        self.tick()
        self.merge(self.phase.setdefault((bar, self.bars[bar].done), {}), self.now())
        self.bars[bar].arrive(n)

    def acquire(self, bar, phase):
        self.merge(self.now(), self.phase.get((bar, phase), {}))

    def wait(self, bar, phase):
        yield from super().wait(bar, phase)
        self.acquire(bar, phase)
        if self.role == "producer" and bar.startswith("done") and self.hands_back:
            yield from super().wait(f"read{bar[-1]}", phase)
            self.acquire(f"read{bar[-1]}", phase)

    def arrive(self, bar, n=1):
        if self.role is None:                 # a commit: no order of ordinary memory
            self.bars[bar].arrive(n)
        elif bar.startswith("done"):          # the softmax warps, a piece's output behind them
            b, k = int(bar[-1]), self.piece[self.role]
            self.saw(("work", b))
            self.saw(("notes", b))
            it, t = self.item(k), int(self.role[-1])
            if not it["two"]:
                self.saw((f"ml{b}", 1 - t))
            for u in (t,) if it["two"] else (0, 1):
                if it["nt"][u]:
                    self.saw((f"fold{self.fold_of(k)}", u))
            if self.hands_back:
                if self.plant == "handed back relaxed":
                    self.bars[f"read{b}"].arrive(n)
                else:
                    self.release(f"read{b}", n)
            self.bars[bar].arrive(n)          # relaxed
        else:
            if bar.startswith("p_full"):
                self.fold[self.fold_of(self.piece[self.role])][int(self.role[-1])] = True
            self.release(bar, n)

    def fold_of(self, k):
        return 0 if self.plant == "one row for all pieces" else k & 1

    def get(self, k, who):
        yield from super().get(k, who)
        self.saw(("work", k & 1))
        self.piece[self.role] = k
        if who == "issuer" and self.item(k) is not None and self.hands_back and self.plant != "issuer not counted":
            self.release(f"read{k & 1}")

    def run(self):
        self.piece = {}
        roles = {"producer": self.producer(), "issuer": self.issuer(), "guard 0": self.guard(0), "guard 1": self.guard(1),
                 "softmax 0": self.softmax(0), "softmax 1": self.softmax(1)}
        left = set(roles)

        def step(name):
            self.role = name
            try:
                dt = next(roles[name])
            except StopIteration:
                left.discard(name)
                return
            finally:
                self.role = None
            self.at(dt, lambda: step(name))
        for name in roles:
            self.at(self.rng.randint(0, 50), lambda name=name: step(name))
        for _ in range(400000):
            if not self.queue:
                break
            self.time, _, fn = heapq.heappop(self.queue)
            fn()
        self.check(not left, "deadlock")
        self.check(self.finished == 2 * len(self.pieces), "pieces left")


def pieces_of(seed):
    rng = random.Random(2000 + seed)
    return [p for _ in range(4) for p in random_pieces(rng)]


@pytest.mark.parametrize("seed", range(60))
def test_every_reuse_of_shared_memory_is_ordered(seed):
    m = OrderModel(seed, pieces_of(seed), hands_back=kernel_hands_reads_back())
    m.run()
    assert m.checked > len(m.pieces)


@pytest.mark.parametrize("kw", [dict(hands_back=False), dict(mutation="handed back relaxed"), dict(mutation="issuer not counted"),
                                dict(mutation="one row for all pieces")],
                         ids=lambda kw: str(*kw.values()))
def test_planted_mistakes_are_caught(kw):
    for seed in range(10):
        with pytest.raises(Fail, match="nothing orders|not ordered behind"):
            OrderModel(seed, pieces_of(seed) + [(2, True, 2, 0)] * 4 + [(4, False, 4, 0)] * 12, **kw).run()
