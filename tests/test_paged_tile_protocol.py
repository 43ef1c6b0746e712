"""A model of how a producer warp of the paged attention kernel fills a K or V
tile, run under random interleavings of its lanes: runs that lie whole in the
block's keys come by TMA (bytes announced to the tile's barrier), the rows of
the others as 16-byte cp.async pieces, each lane's its own.  A lane's wait and
proxy fence order the lane's own copies alone, so the barrier may complete its
phase (all 32 arrivals, no bytes outstanding) only when every lane has waited.

The form in which lane 0 announces and arrives in one, before its copies, lets
the phase end with lane 0's pieces still on their way."""
import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LANES = 32


def _fill(partial, seed, early):
    """One tile: `partial` of its 8 runs are copied piece by piece; with `early` lane 0 arrives as it announces."""
    rnd = random.Random(seed)
    pending, tx = LANES, 0                 # arrivals and bytes that the phase still waits for
    flying = {l: 0 for l in range(LANES)}  # pieces on their way
    bulk = 0                               # TMA runs on their way
    prog = {l: ["sync", "copy", "wait", "arrive"] for l in range(LANES)}
    prog[0].insert(0, "announce")
    if early:
        prog[0].remove("arrive")
    at_sync, done = set(), []
    slow = rnd.randrange(LANES)            # a lane that moves, behind the warp's meeting, only when no other can

    def check():
        if pending == 0 and tx == 0 and not done:
            done.append(True)
            left = [l for l in range(LANES) if flying[l] or "copy" in prog[l]]
            assert not left and not bulk, f"read with pieces of lanes {left} outstanding"

    while True:
        acts = [("lane", l) for l in range(LANES) if prog[l] and not (prog[l][0] == "sync" and l in at_sync)
                and not (prog[l][0] == "wait" and flying[l])]
        acts += [("land", l) for l in range(LANES) if flying[l]] + [("bulk", -1)] * (bulk > 0)
        if not acts:
            break
        kind, l = rnd.choice([a for a in acts if a[1] != slow or len(at_sync) < LANES] or acts)
        if kind == "land":
            flying[l] -= 1
        elif kind == "bulk":
            bulk, tx = bulk - 1, tx - 1
        else:
            op = prog[l][0]
            if op == "sync":
                at_sync.add(l)
                if len(at_sync) == LANES:  # __syncwarp, then the leaders issue the whole runs
                    for k in prog:
                        prog[k].pop(0)
                    bulk = 8 - partial
                continue
            prog[l].pop(0)
            if op == "announce":
                tx += 8 - partial
                pending -= early
            elif op == "copy":
                flying[l] += partial
            elif op == "arrive":
                pending -= 1
        check()
    assert done, "the phase never ends"


@pytest.mark.parametrize("partial", [0, 1, 5, 8])
def test_tile_is_whole_when_its_phase_ends(partial):
    for seed in range(200):
        _fill(partial, seed, early=False)


def test_an_early_arrival_leaves_a_lanes_pieces_outstanding():
    with pytest.raises(AssertionError, match="lanes \\[0\\]"):
        for seed in range(200):
            _fill(1, seed, early=True)


def test_the_kernels_producer_announces_without_arriving():
    src = open(os.path.join(ROOT, "sliding_window_attention_tcgen05_b200", "csrc", "paged_attn_tc.cu")).read()
    body = src[src.index("if (tma) {"):src.index("} else {", src.index("if (tma) {"))]
    assert "mbar_expect_tx(full" in body and "arrive_expect_tx" not in body
    assert re.findall(r"[^\n]*mbar_arrive\(full\);", body) == ["          mbar_arrive(full);"]   # every lane, after its wait
    assert body.index("cp_async_wait<0>()") < body.index("mbar_arrive(full)")


@pytest.mark.parametrize("D", [64, 128])
def test_the_barriers_fit_behind_the_tiles(D):
    # The dynamic shared memory may start on any 16-byte boundary, so the 1024 bytes for the tiles' alignment are no room.
    src = open(os.path.join(ROOT, "sliding_window_attention_tcgen05_b200", "csrc", "paged_attn_tc.cu")).read()
    names = dict(NST=int(re.search(r"kStages = D == 128 \? (\d+) : (\d+)", src)[1 if D == 128 else 2]), kTile=256 * D)
    names["kStages"] = names["NST"]
    for part in re.search(r"constexpr int (FULL = 0.*?);", src)[1].split(","):
        name, value = part.split("=")
        names[name.strip()] = eval(value, {}, names)
    for name in ("kBars", "kTail", "kSmem"):
        if found := re.search(rf"constexpr int {name} = (.*?);", src):
            names[name] = eval(found[1], {}, names)
    tiles = (2 + names["NST"]) * names["kTile"]
    assert tiles + 1008 + names["NBAR"] * 8 + 8 <= names["kSmem"] <= 227 * 1024
