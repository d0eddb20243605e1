"""The paged attention kernel's ring of tiles, checked on a randomised model (CPU only).

The producer fills stages in order, tile n goes to consumer warp n % W, copies land in any order, and the
warps meet at the end of each segment.  The ring's length is a multiple of W, so a stage's tiles all go to
one warp: otherwise a warp could wait for a stage whose previous tile, another warp's, has not landed yet,
and its parity wait would pass a phase early.  The model (scheduler and barriers of protocol_model.py, which
reject any wait whose parity is ambiguous) shows the kernel's rings to be safe and each planted mistake to be caught.
"""
import random

import pytest

import protocol_model as pm


def ring_model(segments, seed, W, S, mistake=None):
    sim = pm.Sim(seed)
    for s in range(S):
        sim.bar(f"full{s}")
        sim.bar(f"empty{s}")
    stage = [None] * S
    total = sum(segments)
    met = [0] * len(segments)
    eaten = []

    def land(s, n):
        def put():
            if stage[s] is not None:
                raise pm.Hazard(f"tile {n} written over tile {stage[s]} in stage {s}")
            stage[s] = n
        return put

    def producer():
        for n in range(total):
            s, k = n % S, n // S
            if k > 0 and mistake != "no wait for the stage":
                yield pm.wait(f"empty{s}", k - 1)
            sim.tma.append((f"full{s}", land(s, n)))
            yield pm.STEP

    def consumer(w):
        base = 0
        for i, count in enumerate(segments):
            n = base + (w + W - base % W) % W
            while n < base + count:
                s, k = n % S, n // S
                yield pm.wait(f"full{s}", k)
                if mistake == "released before it is read":
                    sim.arrive(f"empty{s}")
                    yield pm.STEP
                if stage[s] != n:
                    raise pm.Hazard(f"warp {w} read tile {stage[s]} for tile {n}")
                yield pm.STEP
                if stage[s] != n:
                    raise pm.Hazard(f"tile {n} changed under warp {w}")
                stage[s] = None
                eaten.append(n)
                if mistake != "released before it is read":
                    sim.arrive(f"empty{s}")
                n += W
            base += count
            met[i] += 1
            while met[i] < W:  # the warps' sums are joined here
                yield pm.STEP

    roles = {"producer": producer()}
    roles.update({f"warp{w}": consumer(w) for w in range(W)})
    sim.run(roles)
    assert sorted(eaten) == list(range(total))


def segments_of(rng):
    return [rng.randrange(0, 30) for _ in range(rng.randrange(1, 5))]


# (warps, stages) of the kernel's variants
RINGS = [(6, 12), (5, 10), (4, 8), (4, 16), (8, 16), (8, 32), (7, 14), (7, 28)]


@pytest.mark.parametrize("W,S", RINGS)
def test_ring_is_safe(W, S):
    rng = random.Random(W * 100 + S)
    for seed in range(150):
        ring_model(segments_of(rng), seed, W, S)


def _caught(W, S, mistake=None):
    for seed in range(400):
        try:
            ring_model([20, 30], seed, W, S, mistake)
        except pm.Hazard:
            return True
    return False


@pytest.mark.parametrize("mistake", ["no wait for the stage", "released before it is read"])
def test_planted_mistake_is_caught(mistake):
    assert _caught(6, 12, mistake)


@pytest.mark.parametrize("W,S", [(8, 11), (7, 10), (4, 9)])
def test_ring_that_changes_owners_is_caught(W, S):
    assert _caught(W, S)
