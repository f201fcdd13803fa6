"""The barrier protocol of the CTA-pair kernel, as a model that runs on the CPU.

The model has what the kernel has: `full` on the leader only, on which each CTA
announces and delivers its own bytes; `empty`, `acc_full` and `drain`, which the
MMA threads' commits complete in both CTAs; `acc_empty` on the leader.  Steps of
all agents, copies in flight and MMAs in flight are taken in random order, and in
some runs a wait gives up, at random, after which the CTA's others give up at
their next wait.  Checked: an MMA reads a stage only when both CTAs' copies of
that block are there; a copy overwrites only what both halves' MMAs have read; an
MMA overwrites only a partial that all epilogue warps have read; each phase of
the final waits completes; nobody leaves while a copy, an MMA or a signal is
under way to it.
"""

import random
import re
from pathlib import Path

import pytest

SRC = (Path(__file__).resolve().parent.parent / "weight_only_quantized_prologue_b200" / "csrc" / "dq_block.cuh").read_text()
CFG = SRC[SRC.index("struct PairCfg"):]
ST, PB = (int(re.search(rf"\b{n} = (\d+);", CFG).group(1)) for n in ("ST", "PB"))
KERNEL = SRC[SRC.index("block_pair_kernel(const"):SRC.index("// weight packing, checking")]


class Bar:
    """An mbarrier: pending arrivals and bytes of the phase under way."""

    def __init__(self, count):
        self.count, self.pending, self.tx, self.phase = count, count, 0, 0

    def arrive(self, tx=0):
        assert self.pending > 0, "more arrivals than the phase takes"
        self.tx += tx
        self.pending -= 1
        self._turn()

    def complete(self, n):
        self.tx -= n
        self._turn()

    def _turn(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def done(self, parity):
        return self.phase % 2 != parity


class Pair:
    def __init__(self, rng, blocks, quit_rate):
        self.rng, self.blocks, self.quit_rate = rng, blocks, quit_rate
        self.full = [Bar(2) for _ in range(ST)]
        self.empty = [[Bar(2) for _ in range(ST)] for _ in range(2)]
        self.acc_full = [[[Bar(1) for _ in range(PB)] for _ in range(2)] for _ in range(2)]    # [cta][half][buffer]
        self.acc_empty = [[Bar(8) for _ in range(PB)] for _ in range(2)]                       # [half][buffer]
        self.drain = [[Bar(1) for _ in range(2)] for _ in range(2)]                            # [cta][half]
        self.abort = [False, False]
        self.filled = [0, 0]
        self.issued = [False, False]
        self.flights = []                                   # in any order: landings of copies, threads' arrivals
        self.signals = [[[], []], [[], []]]                 # [half][cta]: commits' arrivals, in order
        self.mma = [[], []]                                 # in order, per half
        self.stage = [[None] * ST for _ in range(2)]        # [cta][stage]: block that is there
        self.reading = [[0] * ST for _ in range(2)]
        self.partial = [[[(-1, set()) for _ in range(PB)] for _ in range(2)] for _ in range(2)]
        self.summed = {}

    # a wait as a generator: yields until the phase is complete; False = it gave up
    def wait(self, cta, bar, parity):
        while not bar.done(parity):
            if self.abort[cta] or self.rng.random() < self.quit_rate:
                self.abort[cta] = True
                return False
            yield
        return True

    def sure_wait(self, bar, parity):
        while not bar.done(parity):
            yield

    def copies(self, cta):
        i, ok = 0, True
        while i < self.blocks:
            s = i % ST
            if i >= ST:
                ok = yield from self.wait(cta, self.empty[cta][s], (i // ST + 1) % 2)
                if not ok:
                    break
            assert self.reading[cta][s] == 0, "a stage is overwritten while it is read"
            self.stage[cta][s] = None

            def land(s=s, i=i):
                self.stage[cta][s] = i
                self.full[s].complete(2)

            def announce(s=s):
                self.full[s].arrive(2)

            # the announcement travels too, and may arrive behind the bytes
            self.flights += [(0, announce), (cta, land)]
            i += 1
            yield
        self.filled[cta] = i
        for j in range(max(0, i - ST), i):
            if ok:
                ok = yield from self.wait(cta, self.empty[cta][j % ST], (j // ST) % 2)

    def commit(self, h, bars):
        self.mma[h].append(("commit", bars))

    def mmas(self, h):
        ok = True
        for i in range(self.blocks):
            s, pb = i % ST, i % PB
            ok = yield from self.wait(0, self.full[s], (i // ST) % 2)
            if ok:
                ok = yield from self.wait(0, self.acc_empty[h][pb], (i // PB + 1) % 2)
            if not ok:
                break
            for c in range(2):
                assert self.stage[c][s] == i, "an MMA reads a stage before its copies are there"
                self.reading[c][s] += 1
                before, seen = self.partial[c][h][pb]
                assert before == i - PB if i >= PB else before == -1
                assert i < PB or len(seen) == 4, "a partial is overwritten before all have read it"
            self.mma[h].append(("mma", i))
            self.commit(h, [self.empty[0][s], self.empty[1][s]])
            self.commit(h, [self.acc_full[0][h][pb], self.acc_full[1][h][pb]])
            self.issued[h] = True
            yield
        if self.issued[h]:
            self.commit(h, [self.drain[0][h], self.drain[1][h]])
            yield from self.sure_wait(self.drain[0][h], 0)

    def epilogue(self, cta, h, w):
        for i in range(self.blocks):
            pb = i % PB
            ok = yield from self.wait(cta, self.acc_full[cta][h][pb], (i // PB) % 2)
            if not ok:
                self.abort[cta] = True
                return
            at, seen = self.partial[cta][h][pb]
            assert at == i, "a partial is read before it is there"
            seen.add(w)
            self.summed[cta, h, w] = i + 1
            self.flights.append((0, lambda pb=pb: self.acc_empty[h][pb].arrive()))
            yield

    def engine(self):
        """One landing, signal or MMA step, if there is any."""
        kinds = [k for k in (0, 1) if self.mma[k]] + (["f"] if self.flights else [])
        kinds += [q for h in self.signals for q in h if q]
        if not kinds:
            return False
        k = self.rng.choice(kinds)
        if isinstance(k, list):
            k.pop(0)()
            return True
        if k == "f":
            self.flights.pop(self.rng.randrange(len(self.flights)))[1]()
            return True
        what, arg = self.mma[k].pop(0)
        if what == "mma":
            for c in range(2):
                self.reading[c][arg % ST] -= 1
                self.partial[c][k][arg % PB] = (arg, set())
        else:
            for c, b in enumerate(arg):
                self.signals[k][c].append(b.arrive)
        return True

    def run(self, agents):
        """Until all agents have ended; a state that nobody can leave is a hang."""
        agents, idle = list(agents), 0
        while agents:
            if self.rng.random() < 0.5 and self.engine():
                idle = 0
                continue
            a = self.rng.choice(agents)
            try:
                next(a)
                idle += 1
            except StopIteration:
                agents.remove(a)
                idle = 0
            assert idle < 20000 or self.engine(), "a wait that never ends"

    def end(self, cta, gave_up):
        """What a CTA does behind the first cluster barrier."""
        if gave_up:
            for i in range(self.filled[cta], self.filled[1 - cta]):
                self.flights.append((0, self.full[i % ST].arrive))
            last = max(self.filled)
            if cta == 0:
                for i in range(max(0, last - ST), last):
                    yield from self.sure_wait(self.full[i % ST], (i // ST) % 2)
        if cta == 1:
            for h in range(2):
                if self.issued[h]:
                    yield from self.sure_wait(self.drain[1][h], 0)
        assert gave_up or not any(h[cta] for h in self.signals), "a CTA leaves before its signals have arrived"


@pytest.mark.parametrize("quit_rate", [0.0, 0.0002, 0.002, 0.02, 0.3])
@pytest.mark.parametrize("blocks", [0, 1, ST, ST + 1, 3 * ST + 1])
def test_copies_sums_and_ends(blocks, quit_rate):
    gave_up = 0
    for seed in range(60):
        p = Pair(random.Random(seed), blocks, quit_rate)
        p.run([p.copies(c) for c in range(2)] + [p.mmas(h) for h in range(2)] +
              [p.epilogue(c, h, w) for c in range(2) for h in range(2) for w in range(4)])
        # the first cluster barrier
        assert abs(p.filled[0] - p.filled[1]) <= ST
        gave_up += any(p.abort)
        p.run([p.end(c, any(p.abort)) for c in range(2)])
        assert not any(k == "mma" for q in p.mma for k, _ in q)
        assert not any(q for h in p.signals for q in h), "a CTA leaves before its signals have arrived"
        if not any(p.abort):
            assert p.filled == [blocks, blocks]
            assert all(p.summed.get((c, h, w), 0) == blocks for c in range(2) for h in range(2) for w in range(4))
            assert not p.mma[0] and not p.mma[1]
        landings = [c for c, f in p.flights if "land" in f.__name__]
        assert not landings, "a CTA leaves before its copies have landed"
    assert gave_up or quit_rate < 0.02 or blocks == 0
    assert quit_rate or not gave_up


def test_waits_of_the_pair_are_of_its_scope():
    """A barrier that the other CTA completes is waited for at the scope of the
    cluster, no thread passes a CTA's landed copies on, and copies count on the
    leader's barrier."""
    for bar in ("full", "empty", "acc_full", "acc_empty"):
        waits = re.findall(rf"(\w+)(?:<\w+>)?\(&{bar}\[", KERNEL)
        assert all(w.endswith("_pair") or w in ("mbar_init", "pair_ready") for w in waits), (bar, waits)
    assert "peer_full" not in KERNEL and "tma_load_2d(" not in KERNEL
    assert re.search(r"acquire\.cluster", SRC[SRC.index("bool pair_ready("):SRC.index("struct PairCfg")])
