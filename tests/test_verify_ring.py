"""The V half of tree attention's shared-memory ring as a state machine, every interleaving of its roles.

A role waits for a slot's phase by the phase's parity, so it must never be two phases away from it.  The roles: the
producer fills a slot once its `empty` barrier says that its last contents are used; the issuer of the products takes
each tile in order and arrives on `empty`; the watcher (which mends the tiles that need care) waits for every tile.  A tile
that needs care is taken only after the watcher has been there."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_hybrid_layer_b200", "csrc")


def explore(tiles, slots, care, watcher_arrives):
    """What goes wrong in some interleaving: "early" (the watcher passes a wait for contents that are not its tile's) or
    "stuck" (nobody can go on); an empty set where nothing does."""
    def before(x, s):                                    # tiles below x that lie in slot s
        return (x - s + slots - 1) // slots if x > s else 0

    def passes(completed, parity):                       # mbarrier try_wait.parity
        return completed & 1 != parity

    bad, seen, todo = set(), {(0, 0, 0)}, [(0, 0, 0)]
    while todo:
        p, c, w = todo.pop()
        used = lambda s: (before(c, s) + before(w, s)) // 2 if watcher_arrives else before(c, s)   # noqa: E731
        nxt = []
        if p < tiles and passes(used(p % slots), p // slots & 1 ^ 1):
            nxt.append((p + 1, c, w))
        if c < tiles and passes(before(p, c % slots), c // slots & 1) and (c not in care or w > c):
            assert before(p, c % slots) == c // slots + 1
            nxt.append((p, c + 1, w))
        if w < tiles and passes(before(p, w % slots), w // slots & 1):
            if before(p, w % slots) != w // slots + 1:
                bad.add("early")
            nxt.append((p, c, w + 1))
        if not nxt and (p, c, w) != (tiles, tiles, tiles):
            bad.add("stuck")
        for n in nxt:
            if n not in seen:
                seen.add(n)
                todo.append(n)
    return bad


@pytest.mark.parametrize("slots", [3, 6])                # V slots at 128 and 256 dimensions, at 64
@pytest.mark.parametrize("tiles", [1, 5, 13, 26])
def test_no_role_of_the_ring_is_two_phases_away(slots, tiles):
    for care in (set(), {tiles - 1}, {tiles // 2, tiles - 1}):
        assert explore(tiles, slots, care, watcher_arrives=True) == set()


def test_the_model_finds_a_watcher_that_the_ring_does_not_wait_for():
    assert explore(13, 3, {12}, watcher_arrives=False) == {"early", "stuck"}


def test_the_kernel_waits_for_every_role_that_looks_at_a_slot():
    """V slots (the odd ones) count the issuer and the watcher, and the watcher arrives before it goes on to the next tile."""
    with open(os.path.join(CSRC, "tree_attention.cu")) as f:
        src = f.read()
    assert re.search(r"mbar_init\(bar\(bars\.empty\[i\]\), i & 1 \? 2 : 1\)", src)
    watcher = src[src.index("} else if (warp == 11) {"):src.index("} else {\n    // ------------------------------------------------------------- softmax")]
    loop = watcher[watcher.index("for (int tile = w.t0"):]
    skipped, cared = loop.split("continue;", 1)
    for part in (skipped, cared):
        assert "mbar_arrive(bar(bars.empty[s]))" in part
