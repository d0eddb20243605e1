"""The paged attention kernel's rings of tiles, checked on a randomised model (CPU only).

Tile n of a CTA's run goes to warp n % W.  Every warp has a ring of its own: it fills the stages with its first
tiles, and refills a stage with its next tile when it has read it; copies land in any order, and the warps
meet at the end of each segment while their rings run on into the next.  The model (scheduler and barriers of
protocol_model.py, which reject any wait whose parity is ambiguous) shows this to be safe and planted mistakes
to be caught, among them one ring shared by all warps: there a stage's tiles belong to different warps, and a warp
could wait for a stage whose previous tile has not landed yet, so that its parity wait passes a phase early.
"""
import random

import pytest

import protocol_model as pm


def rings_model(segments, seed, W, depth, mistake=None):
    sim = pm.Sim(seed)
    for w in range(W):
        for s in range(depth):
            sim.bar(f"full{w}.{s}")
    total = sum(segments)
    stage = {(w, s): None for w in range(W) for s in range(depth)}
    met, eaten = [0] * len(segments), []

    def land(at, n):
        def put():
            if stage[at] is not None:
                raise pm.Hazard(f"tile {n} written over tile {stage[at]}")
            stage[at] = n
        return put

    def warp(w):
        mine = list(range(w, total, W))
        issued = taken = base = 0

        def issue():
            nonlocal issued
            if issued < len(mine):
                s = issued % depth
                sim.tma.append((f"full{w}.{s}", land((w, s), mine[issued])))
                issued += 1

        for _ in range(depth):
            issue()
            yield pm.STEP
        for i, count in enumerate(segments):
            while taken < len(mine) and mine[taken] < base + count:
                s, phase = taken % depth, taken // depth
                if mistake == "refilled before it is read":
                    issue()
                yield pm.wait(f"full{w}.{s}", phase + (mistake == "phase counted from one"))
                if stage[w, s] != mine[taken]:
                    raise pm.Hazard(f"warp {w} read tile {stage[w, s]} for tile {mine[taken]}")
                yield pm.STEP
                stage[w, s] = None
                eaten.append(mine[taken])
                taken += 1
                if mistake is None:
                    issue()
            base += count
            met[i] += 1
            while met[i] < W:  # the warps' sums are joined here
                yield pm.STEP

    sim.run({f"warp{w}": warp(w) for w in range(W)})
    assert sorted(eaten) == list(range(total))


def shared_ring_model(segments, seed, W, S):
    """One ring for all warps, filled in order by a warp of its own."""
    sim = pm.Sim(seed)
    for s in range(S):
        sim.bar(f"full{s}")
        sim.bar(f"empty{s}")
    total = sum(segments)

    def producer():
        for n in range(total):
            if n >= S:
                yield pm.wait(f"empty{n % S}", n // S - 1)
            sim.tma.append((f"full{n % S}", lambda: None))
            yield pm.STEP

    def consumer(w):
        for n in range(w, total, W):
            yield pm.wait(f"full{n % S}", n // S)
            yield pm.STEP
            sim.arrive(f"empty{n % S}")

    sim.run({"producer": producer(), **{f"warp{w}": consumer(w) for w in range(W)}})


def segments_of(rng):
    return [rng.randrange(0, 30) for _ in range(rng.randrange(1, 5))]


@pytest.mark.parametrize("W,depth", [(4, 2), (4, 4), (5, 2), (6, 2), (6, 3), (8, 2), (8, 4), (12, 2)])
def test_rings_are_safe(W, depth):
    rng = random.Random(W * 100 + depth)
    for seed in range(150):
        rings_model(segments_of(rng), seed, W, depth)


def _caught(model, *args):
    for seed in range(400):
        try:
            model([20, 30], seed, *args)
        except pm.Hazard:
            return True
    return False


@pytest.mark.parametrize("mistake", ["refilled before it is read", "phase counted from one", "never refilled"])
def test_planted_mistake_is_caught(mistake):
    assert _caught(rings_model, 6, 2, mistake)


@pytest.mark.parametrize("W,S", [(8, 11), (7, 10), (4, 9)])
def test_ring_whose_stages_change_owners_is_caught(W, S):
    assert _caught(shared_ring_model, W, S)
