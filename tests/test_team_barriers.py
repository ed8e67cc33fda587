"""The barrier protocol of k_selective_teams (csrc/ssd_selective_scan.cuh) under random schedules, on the CPU.

Three teams of warps (operands, recurrence, output) share two buffers through four named barriers, FULL + k and
DONE + k.  A barrier opens when every warp of the block has taken part, waiting ("s") or only arriving ("a").  The
teams below take the steps of the kernel's loops; checked are that no schedule stops, that no warp takes part twice
in one phase, that no buffer is written or read out of turn, and that every phase is complete at the end."""
import random

import pytest


def recurrence(tiles):
    for t in range(tiles):
        yield "s", ("FULL", t & 1)
        yield "x", ("scan", t)
        yield "a", ("DONE", t & 1)


def operands(tiles):
    for t in range(tiles):
        if t >= 2:
            yield "s", ("DONE", t & 1)
        yield "x", ("put", t)
        yield "a", ("FULL", t & 1)
    for t in range(max(0, tiles - 2), tiles):
        yield "a", ("DONE", t & 1)


def output(tiles):
    for k in range(min(2, tiles)):
        yield "a", ("FULL", k)
    for t in range(tiles):
        yield "s", ("DONE", t & 1)
        yield "x", ("take", t)
        if t + 2 < tiles:
            yield "a", ("FULL", t & 1)


def run(tiles, rng, outputs=2):
    warps = [recurrence(tiles) for _ in range(4)] + [operands(tiles) for _ in range(2)] + [output(tiles) for _ in range(outputs)]
    alive, blocked, phase, did = set(range(len(warps))), set(), {}, {}
    while alive:
        ready = sorted(alive - blocked)
        assert ready, "every warp waits"
        w = rng.choice(ready)
        step = next(warps[w], None)
        if step is None:
            alive.discard(w)
            continue
        kind, what = step
        if kind == "x":
            do, t = what
            if do == "put":    # the buffer's last tile has been scanned
                assert t < 2 or did.get(("scan", t - 2)) == 4
            elif do == "scan":  # its operands are there, and the sums that it writes over have been taken
                assert did.get(("put", t)) == 2 and (t < 2 or not outputs or did.get(("take", t - 2)) == 2)
            else:
                assert did.get(("scan", t)) == 4
            did[what] = did.get(what, 0) + 1
            continue
        here, waiting = phase.setdefault(what, (set(), set()))
        assert w not in here, "twice in one phase"
        here.add(w)
        if kind == "s":
            waiting.add(w)
            blocked.add(w)
        if len(here) == len(warps):
            blocked -= waiting
            del phase[what]
    assert not phase, "a phase is left open"


@pytest.mark.parametrize("outputs", [2, 0])  # 0: blocks for a segment's end state have no output team
@pytest.mark.parametrize("tiles", [0, 1, 2, 3, 4, 5, 8, 31])
def test_no_schedule_stops_or_mixes_buffers(tiles, outputs):
    rng = random.Random(tiles)
    for _ in range(100):
        run(tiles, rng, outputs)


def test_a_missing_arrival_is_seen(monkeypatch):
    """The check itself: an operand team that does not arrive for the last tiles leaves the output team waiting."""
    whole = operands

    def short(tiles):
        for step in whole(tiles):
            if step[0] == "a" and step[1][0] == "DONE":
                return
            yield step

    monkeypatch.setitem(globals(), "operands", short)
    with pytest.raises(AssertionError, match="every warp waits|left open"):
        run(3, random.Random(0))
