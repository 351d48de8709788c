"""Model checks of the linear kernels' protocols on the CPU (the simulator is that of
test_pipeline_model.py): the ring, accumulators and residual copies of the pair kernel over
tiles and parts of a split reduction, the ring of the tile kernel, the staging slots of the
epilogue against stores that are read as late as the waits allow, and the tile kernel's
exchange, whose every partial sum has to land on a place of its own inside the buffer."""
import itertools

import pytest

from test_pipeline_model import Sim

WARPS = 16


def pair_roles(sim, units, stages=5, res=False, pre=False):
    """units: k-steps of each unit of this pair, in order. One epilogue warp per CTA stands
    for the sixteen (each arrives for its own share). Its residual copy is asked for before
    the wait for the products, or, with a pre-activation, after its store."""
    FULL = [sim.bar(f"full{i}", 3) for i in range(stages)]                 # CTA 0's
    EMPTY = [[sim.bar(f"empty{c}.{i}") for i in range(stages)] for c in range(2)]
    AFULL = [[sim.bar(f"afull{c}.{i}") for i in range(2)] for c in range(2)]
    AEMPTY = [sim.bar(f"aempty{i}", 2 * WARPS) for i in range(2)]          # CTA 0's
    DRAIN = [sim.bar(f"drain{c}") for c in range(2)]
    RES = [sim.bar(f"res{c}", 2) for c in range(2)]
    members = [f"{r}{c}" for c in range(2) for r in ("producer", "mma", "epilogue")]

    def producer(c):
        it = 0
        for ks in itertools.chain.from_iterable(range(n) for n in units):
            st, use = it % stages, it // stages
            if use > 0:  # the kernel's first waits, for the phase before the first, pass at once
                yield ('wait', EMPTY[c][st], use - 1)
            if c == 0:
                yield ('arrive', FULL[st], 1, use)
            yield ('tma', FULL[st], use)
            it += 1
        for st in range(min(stages, it)):
            yield ('wait', EMPTY[c][st], (it - 1 - st) // stages)
        yield ('named', 'cluster', members)

    def mma(c):
        if c == 0:
            it = 0
            for lt, n in enumerate(units):
                acc, use = lt & 1, lt >> 1
                if use > 0:
                    yield ('wait', AEMPTY[acc], use - 1)
                for ks in range(n):
                    st = it % stages
                    yield ('wait', FULL[st], it // stages)
                    yield ('mma',)
                    yield ('commit', [EMPTY[0][st], EMPTY[1][st]])
                    if ks == n - 1:
                        yield ('commit', [AFULL[0][acc], AFULL[1][acc]])
                    it += 1
            yield ('commit', [DRAIN[0], DRAIN[1]])
            for acc in range(2):
                uses = (len(units) + 1 - acc) // 2
                if uses > 0:
                    yield ('wait', AEMPTY[acc], uses - 1)
        yield ('wait', DRAIN[c], 0)
        yield ('named', 'cluster', members)

    def epilogue(c):
        for lt in range(len(units)):
            load = [('arrive', RES[c], 1, lt), ('tma', RES[c], lt)]
            if res and not pre:
                yield from load
            yield ('wait', AFULL[c][lt & 1], lt >> 1)
            if res:
                if pre:
                    yield from load
                yield ('wait', RES[c], lt)
            yield ('arrive', AEMPTY[lt & 1], WARPS)
        yield ('named', 'cluster', members)

    roles = {}
    for c in range(2):
        roles[f"producer{c}"], roles[f"mma{c}"] = producer(c), mma(c)
        roles[f"epilogue{c}"] = epilogue(c)
    return roles


@pytest.mark.parametrize("units", [[1], [16] * 3, [4] * 5, [2] * 9, [9, 8, 9, 8], [1, 1, 1, 1, 1]])
@pytest.mark.parametrize("res,pre", [(False, False), (True, False), (True, True)])
def test_pair_kernel_protocol(units, res, pre):
    for seed in range(20):
        sim = Sim(seed * 100 + len(units))
        sim.run(pair_roles(sim, units, res=res, pre=pre))


def test_model_detects_a_residual_loaded_before_its_slot_is_used_up():
    """Two residual copies ahead with one slot: the second lands in the phase of the first."""
    def roles(sim):
        r = sim.bar("res", 2)

        def epilogue():
            for k in range(4):
                if k == 0:
                    yield ('arrive', r, 1, 0)
                    yield ('tma', r, 0)
                if k < 3:  # the next one before this one has been waited for
                    yield ('arrive', r, 1, k + 1)
                    yield ('tma', r, k + 1)
                yield ('wait', r, k)
        return {"epilogue": epilogue()}

    with pytest.raises(AssertionError, match="arrival for phase|phase skipped|stale|more"):
        for seed in range(40):
            sim = Sim(seed)
            sim.run(roles(sim))


def tile_roles(sim, ksteps, stages):
    FULL = [sim.bar(f"full{i}", 2) for i in range(stages)]
    EMPTY = [sim.bar(f"empty{i}") for i in range(stages)]
    ACC = sim.bar("acc")

    def producer():
        for it in range(ksteps):
            st = it % stages
            if it >= stages:
                yield ('wait', EMPTY[st], it // stages - 1)
            yield ('arrive', FULL[st], 1, it // stages)
            yield ('tma', FULL[st], it // stages)
        for st in range(min(stages, ksteps)):
            yield ('wait', FULL[st], (ksteps - 1 - st) // stages)
        yield ('wait', ACC, 0)

    def mma():
        for it in range(ksteps):
            yield ('wait', FULL[it % stages], it // stages)
            yield ('mma',)
            yield ('commit', EMPTY[it % stages])
        yield ('commit', ACC)
        yield ('wait', ACC, 0)

    def epilogue():
        yield ('wait', ACC, 0)

    return {"producer": producer(), "mma": mma(), "epilogue": epilogue()}


@pytest.mark.parametrize("ksteps,stages", [(1, 5), (5, 5), (6, 5), (23, 7), (40, 10)])
def test_tile_kernel_protocol(ksteps, stages):
    for seed in range(20):
        sim = Sim(seed * 50 + ksteps)
        sim.run(tile_roles(sim, ksteps, stages))


@pytest.mark.parametrize("res,pre", list(itertools.product([False, True], repeat=2)))
def test_staging_slot(res, pre):
    """The order of an epilogue warp's waits, residual loads, writes and stores over tiles
    inside and outside, with every store read from the slot as late as the waits allow."""
    unread = False  # a store that may still read the slot

    def write():
        assert not unread, "the slot written while a store still reads it"

    for inside in (True, True, False, True, False, False, True, True):
        if not inside:
            continue
        if res and not pre:
            unread = False  # wait_group.read 0
            write()         # the residual copy
        if pre:
            unread = False
            write()
            unread = True   # the pre-activation's store
            if res:
                unread = False
                write()
        if not res:
            unread = False
        write()             # the output, in place of the residual
        unread = True


def swizzle(row, units):
    return row & 7 if units >= 8 else (row >> 1) & 3 if units == 4 else (row >> 2) & 1


@pytest.mark.parametrize("bn", [64, 128])
@pytest.mark.parametrize("split", [1, 2, 4, 8])
def test_exchange_places(bn, split):
    """Tiles with the rows on the 128 side: 16-byte units of rank r's partial sums in owner
    q's buffer of 128 bn floats are distinct, inside, and where the owner reads them."""
    per, units = bn // split, bn // split // 4
    for owner in range(split):
        seen = {}
        for rank in range(split):
            for m in range(128):
                for col in range(owner * per, (owner + 1) * per, 4):
                    u = (col % per) // 4
                    at = (rank * 128 + m) * units + (u ^ swizzle(m, units))
                    assert 0 <= at < 128 * bn // 4 and at not in seen
                    assert rank * 128 * units <= at < (rank + 1) * 128 * units
                    assert at // units == rank * 128 + m, "the unit leaves its row"
                    seen[at] = (rank, m, col)
        for row in range(128):
            for c8 in range(per // 8):
                z = swizzle(row, units)
                for q in range(split):
                    for k in range(2):
                        at = (q * 128 + row) * units + ((2 * c8 + k) ^ z)
                        assert seen[at] == (q, row, owner * per + 8 * c8 + 4 * k)


@pytest.mark.parametrize("bn", [16, 32, 64])
@pytest.mark.parametrize("split", [1, 2, 4, 8])
def test_exchange_places_of_few_rows(bn, split):
    """Tiles with the columns on the 128 side: floats [rank][row][128]."""
    per = bn // split
    for owner in range(split):
        seen = set()
        for rank in range(split):
            for r in range(owner * per, (owner + 1) * per):
                for m in range(128):
                    at = (rank * per + r % per) * 128 + m
                    assert 0 <= at < 128 * bn and at not in seen
                    seen.add(at)
        assert len(seen) == 128 * bn
