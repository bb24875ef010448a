"""The roles of the scan's blocks and of the projection's tile kernel on the model of
tests/_barrier_model.py: under every schedule no deadlock, no wait that returns on another phase, no
buffer read before it is written or after it is overwritten.  What the kernels did while they were
built, and must not do again, is rejected: tiles dealt out with a group's later ones first, a tile's own map
kept back until the others' are there, slots for z and y asked for before either is filled."""
import pytest

from tests._barrier_model import Sim, Violation

WARPS = 3                                       # of eight


class Published(Sim):
    """Sim with values that blocks leave for one another: ('publish', key), ('await', key); and a ticket
    counter."""

    def __init__(self, seed, qmax=2):
        super().__init__(seed, qmax)
        self.there, self.tickets = set(), 0

    def draw(self):
        self.tickets += 1
        return self.tickets - 1

    def _ready(self, a):
        if a["act"][0] == "await":
            return a["act"][1] in self.there
        return super()._ready(a)

    def _perform(self, a):
        if a["act"][0] == "publish":
            self.there.add(a["act"][1])
        super()._perform(a)


def scan_block(sim, name, tiles, stages, own_map_last=False):
    """One block.  tiles: (index, place in its group, the group's tiles, its group, the group before or
    None), in the order in which tickets are drawn."""
    b = lambda kind, i, count=1: sim.bar(f"{name}.{kind}{i}", count)
    known, full, empty = ([b(k, i, c) for i in range(stages)] for k, c in (("known", 1), ("full", 1), ("empty", WARPS + 1)))
    maps, carry = ([b(k, i, c) for i in range(2)] for k, c in (("maps", WARPS), ("carry", 1)))
    meta = {}

    def copy():
        it, drawn = 0, sim.draw()
        while True:
            tile = tiles[drawn] if drawn < len(tiles) else None
            if tile:
                drawn = sim.draw()              # ahead of the stage's wait
            s = it % stages
            if it >= stages:
                yield ("wait", empty[s], it // stages - 1)
            meta[it] = tile
            yield ("write", f"{name}.meta{s}", it)
            yield ("arrive", known[s], it)
            if tile is None:
                yield ("arrive", full[s], it)
                return
            yield ("copy", full[s], it, f"{name}.rows{s}", it)
            it += 1

    def carries():
        it = 0
        while True:
            s, par = it % stages, it & 1
            yield ("wait", known[s], it // stages)
            yield ("read", f"{name}.meta{s}", it)
            tile = meta[it]
            if tile is None:
                return
            index, at, count, group, before = tile

            def others():
                for k in range(at):
                    yield ("await", ("map", index - at + k))
                if before is not None:
                    yield ("await", ("state", before))
                yield ("write", f"{name}.carry{par}", it)
                yield ("arrive", carry[par], it)

            def own():
                yield ("wait", maps[par], it // 2)
                for w in range(WARPS):
                    yield ("read", f"{name}.map{par}.{w}", it)
                yield ("publish", ("map", index))
            # whichever comes first in the kernel; here the order that is hardest for the others
            for part in ((others(), own()) if own_map_last else (own(), others())):
                yield from part
            if at == count - 1:
                yield ("publish", ("state", group))
            yield ("arrive", empty[s], it)
            it += 1

    def consumer(w):
        it = 0
        while True:
            s, par = it % stages, it & 1
            yield ("wait", full[s], it // stages)
            if meta[it] is None:
                return
            yield ("read", f"{name}.rows{s}", it)
            yield ("write", f"{name}.map{par}.{w}", it)
            yield ("arrive", maps[par], it)
            yield ("wait", maps[par], it // 2)
            yield ("wait", carry[par], it // 2)
            yield ("read", f"{name}.carry{par}", it)
            for v in range(w):
                yield ("read", f"{name}.map{par}.{v}", it)
            yield ("read", f"{name}.rows{s}", it)
            yield ("arrive", empty[s], it)
            it += 1

    for g in [copy(), carries()] + [consumer(w) for w in range(WARPS)]:
        sim.agent(g)



def scan_block_ahead(sim, name, tiles, stages=3):
    """One block of the kernel for long trajectories: a tile's map before the results of the one before
    it, published by the warp that is last with its rows."""
    b = lambda kind, i, count=1: sim.bar(f"{name}.{kind}{i}", count)
    known, full, empty, maps, carry = ([b(k, i, c) for i in range(stages)] for k, c in (
        ("known", 1), ("full", 1), ("empty", WARPS + 1), ("maps", WARPS), ("carry", 1)))
    meta, mapped = {}, {}

    def copy():
        it, drawn = 0, sim.draw()
        while True:
            tile = tiles[drawn] if drawn < len(tiles) else None
            if tile:
                drawn = sim.draw()
            s = it % stages
            if it >= stages:
                yield ("wait", empty[s], it // stages - 1)
            meta[it] = tile
            yield ("write", f"{name}.meta{s}", it)
            yield ("arrive", known[s], it)
            if tile is None:
                yield ("arrive", full[s], it)
                return
            yield ("copy", full[s], it, f"{name}.rows{s}", it)
            it += 1

    def carries():
        it = 0
        while True:
            s = it % stages
            yield ("wait", known[s], it // stages)
            yield ("read", f"{name}.meta{s}", it)
            if meta[it] is None:
                return
            index, at, count, group, before = meta[it]
            for k in range(at):
                yield ("await", ("map", index - at + k))
            if before is not None:
                yield ("await", ("state", before))
            yield ("write", f"{name}.carry{s}", it)
            yield ("arrive", carry[s], it)
            yield ("wait", maps[s], it // stages)
            for w in range(WARPS):
                yield ("read", f"{name}.map{s}.{w}", it)
            if at == count - 1:
                yield ("publish", ("state", group))
            yield ("arrive", empty[s], it)
            it += 1

    def consumer(w):
        def map_tile(it):
            s = it % stages
            yield ("wait", full[s], it // stages)
            yield ("read", f"{name}.meta{s}", it)
            if meta[it] is None:
                return
            yield ("read", f"{name}.rows{s}", it)
            yield ("write", f"{name}.map{s}.{w}", it)
            yield ("arrive", maps[s], it)
            mapped[it] = mapped.get(it, 0) + 1
            if mapped[it] == WARPS and meta[it][1] < meta[it][2] - 1:
                for v in range(WARPS):
                    yield ("read", f"{name}.map{s}.{v}", it)
                yield ("publish", ("map", meta[it][0]))

        def results(it):
            s = it % stages
            yield ("wait", maps[s], it // stages)
            yield ("wait", carry[s], it // stages)
            yield ("read", f"{name}.carry{s}", it)
            for v in range(w):
                yield ("read", f"{name}.map{s}.{v}", it)
            yield ("read", f"{name}.rows{s}", it)
            yield ("arrive", empty[s], it)

        it = 0
        yield from map_tile(0)
        while meta[it] is not None:
            yield from map_tile(it + 1)
            yield from results(it)
            it += 1

    for g in [copy(), carries()] + [consumer(w) for w in range(WARPS)]:
        sim.agent(g)


def _chain(n, group, backwards_in_group=False):
    tiles = []
    for i in range(n):
        g = i // group
        tiles.append((i, i % group, min(group, n - g * group), g, g - 1 if g else None))
    if backwards_in_group:
        tiles.sort(key=lambda t: (t[3], -t[1]))
    return tiles


def _found(make, seeds=60):
    out = []
    for seed in range(seeds):
        sim = Published(seed, qmax=1 + seed % 3)
        make(sim, seed)
        try:
            sim.run()
        except Violation as e:
            out.append(str(e))
    return out


@pytest.mark.parametrize("blocks", [1, 2, 4])
@pytest.mark.parametrize("n,group", [(1, 4), (7, 3), (12, 4), (9, 1), (16, 8)])
def test_scan_blocks_wait_only_for_what_comes(n, group, blocks):
    def make(sim, seed):
        for k in range(blocks):
            scan_block(sim, f"b{k}", _chain(n, group), 2 + seed % 2)
    assert _found(make) == []



@pytest.mark.parametrize("blocks", [1, 2, 4])
@pytest.mark.parametrize("n,group", [(1, 4), (2, 1), (7, 3), (12, 4), (9, 1), (24, 8)])
def test_scan_blocks_a_map_ahead(n, group, blocks):
    def make(sim, seed):
        for k in range(blocks):
            scan_block_ahead(sim, f"b{k}", _chain(n, group))
    assert _found(make) == []


def test_scan_a_map_ahead_wants_a_stage_of_its_own():
    """In one stage, the map would wait for the results before it, and they come after the map."""
    def make(sim, seed):
        scan_block_ahead(sim, "b", _chain(4, 2), stages=1)
    assert all("deadlock" in m.lower() for m in _found(make, 5)) and len(_found(make, 5)) == 5


def test_scan_rejects_a_group_dealt_out_backwards():
    def make(sim, seed):
        for k in range(2):
            scan_block(sim, f"b{k}", _chain(16, 8, backwards_in_group=True), 2)
    found = _found(make, 20)
    assert len(found) == 20 and all("deadlock" in m.lower() for m in found)


def test_scan_maps_do_not_wait_for_one_another():
    """A tile's own map goes out although the maps before it are not there: with it last, a group's
    maps would follow one another across blocks, right but one at a time.  Here the map before never
    comes; what counts is whether the tile's own has been published when nothing can move any more."""
    for last, published in ((False, True), (True, False)):
        sim = Published(1)
        scan_block(sim, "b", [(1, 1, 3, 0, None)], 2, own_map_last=last)   # tile 0's map never comes
        with pytest.raises(Violation, match="(?i)deadlock"):
            sim.run()
        assert (("map", 1) in sim.there) == published


def output_slots(sim, keep, units, both_first=False, together=True):
    """The two halves' epilogue warps (one stands for four) and their storing threads: every unit leaves
    z, where it is kept, and y in the half's two slots in turn.  together: both are given back behind y,
    otherwise each behind the next store."""
    full = [sim.bar(f"full{i}") for i in range(4)]
    free = [sim.bar(f"free{i}") for i in range(4)]

    def epilogue(half):
        q = 0
        for u in range(half, units, 2):
            asked = []
            for k in (0, 1) if keep else (1,):
                s, use = half + 2 * (q & 1), q >> 1
                q += 1
                if use > 0:
                    yield ("wait", free[s], use - 1)
                asked.append((s, use, k))
                if both_first and k == 0:
                    continue
                for s, use, k in asked:
                    yield ("write", f"slot{s}", (u, k))
                    yield ("arrive", full[s], use)
                asked = []

    def store(half):
        q = 0
        last = None
        for u in range(half, units, 2):
            for k in (0, 1) if keep else (1,):
                s, use = half + 2 * (q & 1), q >> 1
                yield ("wait", full[s], use)
                yield ("read", f"slot{s}", (u, k))
                q += 1
                if keep and together:
                    if k == 1:
                        yield ("arrive", free[half], use)
                        yield ("arrive", free[half + 2], use)
                elif last is not None:                  # all but the last store have been read
                    yield ("arrive", free[last[0]], last[1])
                last = (s, use)

    for half in (0, 1):
        sim.agent(epilogue(half))
        sim.agent(store(half))


@pytest.mark.parametrize("units", [1, 2, 3, 8, 13])
@pytest.mark.parametrize("together", [False, True])
@pytest.mark.parametrize("keep", [False, True])
def test_output_slots(keep, together, units):
    for seed in range(60):
        sim = Sim(seed)
        output_slots(sim, keep, units, together=together)
        sim.run()


def test_output_slots_reject_both_asked_for_before_either_is_filled():
    """Where a slot is given back behind the next store, y's comes free only behind the z that follows it."""
    with pytest.raises(Violation, match="(?i)deadlock"):
        for seed in range(20):
            sim = Sim(seed)
            output_slots(sim, True, 8, both_first=True, together=False)
            sim.run()
