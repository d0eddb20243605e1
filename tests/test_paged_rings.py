"""The rings of the paged attention kernel as its warps run them, checked on a randomised model (CPU only).

A warp walks its share alone: segments (tiles of one item) one after another, without meeting the other warps, its ring
running on into the next segment (runs of tiles, and whole items); or it takes every W-th tile of its CTA's one item, and
the warps meet once, at the item's end, to join their sums in the memory of the rings.  Pages are looked up in batches
that end at a segment's end: the ring is filled from the current batch alone, so it may be partly full while tiles are
read.  Tiles come by TMA on a barrier per stage, in any order (bf16), or by groups of asynchronous copies, of which
a warp can only wait for all but the newest n (4 bits): for the oldest of a full ring, for all of a partly full one.

The loop restates attend() and Issuer of csrc/paged_attention.cu; a change there needs the same change here.
"""
import random

import pytest

import protocol_model as pm


class Groups:
    """Copy groups of one warp, committed in order; waiting for the first k of them."""

    def __init__(self):
        self.landed = []

    def arrive(self):
        pass

    def ready(self, k):
        return all(self.landed[:k])


class Issuer:
    """Walks a warp's segments ahead of their reader, in batches."""

    def __init__(self, segments, first, step, batch):
        self.segments, self.step, self.size = segments, step, batch
        self.seg, self.k = 0, first
        self.tiles, self.issued = [], 0

    def look_up(self):
        while self.seg < len(self.segments) and self.k >= self.segments[self.seg]:
            self.k -= self.segments[self.seg]
            self.seg += 1
        if self.seg < len(self.segments):
            n = min(self.size, -(-(self.segments[self.seg] - self.k) // self.step))
            self.tiles = [(self.seg, self.k + i * self.step) for i in range(n)]
            self.k += n * self.step


def rings_model(shares, seed, depth, batch, copies, one_item=False, mistake=None):
    """shares: the segments of every warp (one_item: the CTA's one segment, W warps)."""
    sim = pm.Sim(seed)
    W = len(shares)
    stage = {(w, s): None for w in range(W) for s in range(depth)}   # tile whose copy was asked for last
    there = {(w, s): False for w in range(W) for s in range(depth)}  # and whether it has landed
    eaten, met = [[] for _ in shares], [0]
    for w in range(W):
        for s in range(depth):
            sim.bar(f"full{w}.{s}")
        sim.bars[f"groups{w}"] = Groups()

    def warp(w):
        segments, first, step = shares[w], w if one_item else 0, W if one_item else 1
        iss, groups = Issuer(segments, first, step, batch), sim.bars[f"groups{w}"]
        k, ahead, taken, seg, looked = first, 0, 0, 0, False
        room = depth + (mistake == "refilled before it is read")

        def issue():
            at, tile = (w, iss.issued % depth), iss.tiles.pop(0)
            if stage[at] is not None:
                raise pm.Hazard(f"{tile} asked for over {stage[at]}")
            stage[at], there[at] = tile, False
            n = len(groups.landed)
            groups.landed.append(False)

            def land():
                there[at] = groups.landed[n] = True
            sim.tma.append((f"full{w}.{at[1]}" if copies == "tma" else f"groups{w}", land))
            iss.issued += 1

        while seg < len(segments):
            if not iss.tiles and not (looked and mistake == "pages looked up once"):
                iss.look_up()
                looked = True
            if ahead and k < segments[seg]:
                s = taken % depth
                if copies == "tma":
                    phase = taken // depth + (mistake == "phase counted from one")
                    if mistake == "phase counted by segment":
                        phase = (k // step) // depth
                    yield pm.wait(f"full{w}.{s}", phase)
                else:
                    newest = depth - 1 if ahead == depth or mistake == "newest left whatever the ring holds" else 0
                    yield pm.wait(f"groups{w}", len(groups.landed) - newest)
                if stage[w, s] != (seg, k) or not there[w, s]:
                    raise pm.Hazard(f"warp {w} read {stage[w, s]} (landed: {there[w, s]}) for {(seg, k)}")
                yield pm.STEP
                stage[w, s] = None
                eaten[w].append((seg, k))
                taken, ahead, k = taken + 1, ahead - 1, k + step
            while ahead < room and iss.tiles:
                issue()
                ahead += 1
                yield pm.STEP
            yield pm.STEP
            if k < segments[seg]:
                continue
            k -= segments[seg]
            seg += 1
        if one_item:
            met[0] += 1
            while met[0] < W and mistake != "joined before all have read":
                yield pm.STEP
            for at, tile in stage.items():
                if tile is not None:
                    raise pm.Hazard(f"warp {w} joins over tile {tile} of warp {at[0]}")

    # a loop that makes no progress ends at the bound
    sim.run({f"warp{w}": warp(w) for w in range(W)}, max_steps=30000)
    for w, segments in enumerate(shares):
        first, step = (w, W) if one_item else (0, 1)
        want = [(i, t) for i, n in enumerate(segments) for t in range(first, n, step)]
        if eaten[w] != want:
            raise pm.Hazard(f"warp {w} took {eaten[w]} of {want}")


def runs(rng, W):
    """Segments of every warp: empty items among them."""
    return [[rng.choice([0, 1, 2, 3, rng.randrange(20)]) for _ in range(rng.randrange(1, 6))] for _ in range(W)]


@pytest.mark.parametrize("copies", ["tma", "groups"])
@pytest.mark.parametrize("W,depth,batch", [(4, 3, 32), (6, 2, 32), (6, 4, 5), (8, 3, 7), (12, 2, 3), (12, 4, 1)])
def test_runs_without_a_meeting_are_safe(copies, W, depth, batch):
    rng = random.Random(W * 100 + depth)
    for seed in range(60):
        rings_model(runs(rng, W), seed, depth, batch, copies)


@pytest.mark.parametrize("copies", ["tma", "groups"])
@pytest.mark.parametrize("W,depth,batch", [(4, 3, 32), (6, 2, 32), (6, 4, 2), (8, 3, 3), (12, 2, 32)])
def test_one_item_with_its_join_is_safe(copies, W, depth, batch):
    rng = random.Random(W * 100 + depth)
    for seed in range(60):
        n = rng.choice([0, 1, W - 1, W, rng.randrange(8 * W)])
        rings_model([[n]] * W, seed, depth, batch, copies, one_item=True)


def _caught(shares, depth, batch, copies, one_item, mistake):
    for seed in range(100):
        try:
            rings_model(shares, seed, depth, batch, copies, one_item, mistake)
        except pm.Hazard:
            return True
    return False


@pytest.mark.parametrize("copies,mistake", [
    ("tma", "refilled before it is read"), ("tma", "phase counted from one"), ("tma", "phase counted by segment"),
    ("tma", "pages looked up once"), ("groups", "refilled before it is read"),
    ("groups", "newest left whatever the ring holds"), ("groups", "pages looked up once"),
])
def test_planted_mistake_in_a_run_is_caught(copies, mistake):
    assert _caught([[5, 0, 9], [3, 11]], 3, 4, copies, False, mistake)


@pytest.mark.parametrize("copies", ["tma", "groups"])
def test_joining_before_all_have_read_is_caught(copies):
    assert _caught([[17]] * 4, 2, 32, copies, True, "joined before all have read")
