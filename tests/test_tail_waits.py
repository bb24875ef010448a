"""The roles of the tile kernel of linear_logprob.cu and the kernel before it, which it overlaps, on
the model of tests/_barrier_model.py: under every schedule nothing of that kernel is read early,
and no bounded wait stands while that kernel runs on.  Its limit is for this kernel's own work: a
predecessor of any length must not use it up.  The placement that the kernel had before, with
waits for the predecessor only where its results are read, must be rejected."""
import pytest

from tests._barrier_model import Sim, Violation

STAGES, SLOTS = 3, 2
MODES = ["forward", "forward-copied", "dz", "dz-copied", "grad"]


class Behind(Sim):
    """Sim with a kernel before: ('previous',) waits until it is done, ('needs', what) uses what it
    makes.  It ends when nothing else can move any more, the slowest there is."""
    done = False

    def _ready(self, a):
        if a["act"][0] == "previous":
            return self.done
        if a["act"][0] == "end":
            return (not self.copies and not any(self.queues.values())
                    and not any(not b["done"] and b is not a and self._ready(b) for b in self.agents))
        return super()._ready(a)

    def _perform(self, a):
        kind = a["act"][0]
        if kind == "needs" and not self.done:
            self.fail(f"{a['act'][1]} used before it is made")
        if kind == "end":
            stands = [b["act"] for b in self.agents if not b["done"] and b["act"][0] == "wait"]
            if stands:
                self.fail(f"bounded waits stand while the kernel before runs: {stands}")
            self.done = True
        super()._perform(a)


def tile_kernel(sim, mode, tiles, steps, bounded=True):
    """One block's warps, as the source has them; bounded=False places the waits as before."""
    copied, dz, grad = mode.endswith("copied"), mode.startswith("dz"), mode == "grad"
    output = dz or grad
    ahead = dz and not copied
    full = [sim.bar(f"full{i}", 2) for i in range(STAGES)]
    empty = [sim.bar(f"empty{i}") for i in range(STAGES)]
    acc_full = [sim.bar(f"acc_full{i}") for i in range(2)]
    acc_empty = [sim.bar(f"acc_empty{i}", 2, tagged=True) for i in range(2)]
    out_full = [sim.bar(f"out_full{i}") for i in range(SLOTS)]
    out_free = [sim.bar(f"out_free{i}") for i in range(SLOTS)]

    def predecessor():
        yield ("end",)

    def feed(name):
        is_b = name == "B"
        it = 0
        if grad or (not is_b and (copied if not bounded else not ahead)):
            yield ("previous",)
        for n in range(tiles):
            if bounded and ahead and n == 2:
                yield ("previous",)
            for k in range(steps):
                s, use = it % STAGES, it // STAGES
                if bounded and it == STAGES and not ahead:
                    yield ("previous",)
                if use > 0:
                    yield ("wait", empty[s], use - 1)
                if grad or (copied and not is_b):
                    yield ("needs", f"{name} of tile {n}")
                yield ("copy", full[s], it, f"{name}{s}", (name, it))
                it += 1
        if bounded:
            yield ("previous",)
        for i in range(min(it, STAGES)):
            uses = (it - i + STAGES - 1) // STAGES
            yield ("wait", empty[i], uses - 1)

    def issue():
        it = 0
        if bounded and not ahead:
            yield ("previous",)
        for n in range(tiles):
            if bounded and ahead and n == 2:
                yield ("previous",)
            if n >= 2:
                yield ("wait", acc_empty[n & 1], n // 2 - 1)
            for k in range(steps):
                s = it % STAGES
                yield ("wait", full[s], it // STAGES)
                last = [(f"D{n & 1}", n)] if k == steps - 1 else []
                yield ("mma", "T", [(f"A{s}", ("A", it)), (f"B{s}", ("B", it))], last)
                yield ("commit", "T", empty[s], it)
                it += 1
            yield ("commit", "T", acc_full[n & 1], n)

    def epilogue(half):
        if bounded or dz:
            yield ("previous",)
        for n in range(tiles):
            yield ("wait", acc_full[n & 1], n // 2)
            yield ("read", f"D{n & 1}", n)
            if dz:
                yield ("needs", "the rows' terms")
            if output:                              # a slot each, filled by the two halves in turn
                slot = (2 * n + half) % SLOTS
                use = (2 * n + half) // SLOTS
                if use > 0:
                    yield ("wait", out_free[slot], use - 1)
                yield ("write", f"O{slot}", 2 * n + half)
                yield ("arrive", out_full[slot], n)
            yield ("arrive", acc_empty[n & 1], n)

    def store(mine):
        if not output:
            return
        if bounded:
            yield ("previous",)
        for g in range(mine, 2 * tiles, 2):
            yield ("wait", out_full[g % SLOTS], g // SLOTS)
            yield ("read", f"O{g % SLOTS}", g)
            yield ("needs", "the output's last contents")
            yield ("arrive", out_free[g % SLOTS], g)

    for g in (predecessor(), feed("A"), feed("B"), issue(), epilogue(0), epilogue(1), store(0), store(1)):
        sim.agent(g)


def _violations(mode, bounded):
    found = []
    for seed in range(120):
        sim = Behind(seed, qmax=1 + seed % 3)
        tile_kernel(sim, mode, 1 + seed % 5, 1 + seed % 4, bounded)
        try:
            sim.run()
        except Violation as e:
            found.append(str(e))
    return found


@pytest.mark.parametrize("mode", MODES)
def test_no_bounded_wait_stands_before_the_predecessor_ends(mode):
    if mode == "forward":                           # the first kernel of its call: nothing runs before it
        sim = Behind(0)
        sim.done = True
        tile_kernel(sim, mode, 5, 3)
        sim.run()
        return
    assert _violations(mode, True) == []


@pytest.mark.parametrize("mode", MODES[1:])
def test_rejects_waits_only_where_results_are_read(mode):
    found = _violations(mode, False)
    assert found and all("bounded waits stand" in m for m in found)
