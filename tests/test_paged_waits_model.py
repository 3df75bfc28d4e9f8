"""How warps that wait on one another leave the attention kernel of chunks when a wait
gives up, as a model: every interleaving of the warps' steps, every wait that is not
over free to give up.  A barrier has no limit of its own, so none may be left with a warp
in it and another gone."""
import pytest

TILES = 2


def meet(warps=2):
    """What the kernel does: every warp comes to a barrier at the end of each tile,
    and once more when there is no tile (or it gave up looking for one); all go on, or
    all leave.  Behind it, barriers of the tile's join.

    A warp is (step, tile, go); the steps of a tile:
      info   the tile is known: go, or give up
      work   its products are done: go, or give up
      meet   the barrier
      join   the barrier of the join
    """

    def moves(state):
        for w, (step, tile, go) in enumerate(state):
            if step == "info":
                if tile == TILES:
                    yield w, ("meet", tile, False)  # no more tiles
                else:
                    yield w, ("work", tile, True)
                yield w, ("meet", tile, False)
            elif step == "work":
                yield w, ("meet", tile, True)
                yield w, ("meet", tile, False)

    def barriers(state):
        if all(s[0] == "meet" for s in state):
            on = all(s[2] for s in state)
            return tuple(("join", s[1], True) if on else ("left", s[1], False) for s in state)
        if all(s[0] == "join" for s in state):
            return tuple(("info", s[1] + 1, True) for s in state)
        return None

    return tuple(("info", 0, True) for _ in range(warps)), moves, barriers


def arrive_and_wait(warps=2):
    """A planted mistake: the end of a tile is an arrival and a wait that may give
    up on its own, and barriers follow for those whose wait did not.  (go: whether the
    warp has arrived.)"""

    def moves(state):
        for w, (step, tile, arrived) in enumerate(state):
            if step == "info":
                if tile < TILES:
                    yield w, ("work", tile, False)
                yield w, ("left", tile, False)
            elif step == "work":
                yield w, ("ended", tile, True)
                yield w, ("left", tile, False)
            elif step == "ended":
                if all(s[1] > tile or s[2] for s in state):
                    yield w, ("join", tile, True)
                else:
                    yield w, ("left", tile, True)

    def barriers(state):
        if all(s[0] == "join" for s in state):
            return tuple(("info", s[1] + 1, False) for s in state)
        return None

    return tuple(("info", 0, False) for _ in range(warps)), moves, barriers


def stuck(model):
    """A state with a warp in a barrier that the others will not reach, or None."""
    start, moves, barriers = model
    seen, todo = {start}, [start]
    while todo:
        state = todo.pop()
        after = [tuple(new if i == w else s for i, s in enumerate(state))
                 for w, new in moves(state)]
        met = barriers(state)
        if met is not None:
            after.append(met)
        if not after and any(s[0] != "left" for s in state):
            return state
        for x in after:
            if x not in seen:
                seen.add(x)
                todo.append(x)
    return None


@pytest.mark.parametrize("warps", [2, 3])
def test_no_warp_is_left_in_a_barrier(warps):
    assert stuck(meet(warps)) is None


def test_the_model_finds_a_warp_that_is_left_behind():
    state = stuck(arrive_and_wait())
    assert state is not None and {s[0] for s in state} == {"join", "left"}


def test_every_warp_leaves_after_the_last_tile():
    """Without a wait that gives up, the meetings of all warps are as many."""
    start, moves, barriers = meet()
    state = start
    while any(s[0] != "left" for s in state):
        met = barriers(state)
        if met is not None:
            state = met
            continue
        w, new = next(iter(moves(state)))
        state = tuple(new if i == w else s for i, s in enumerate(state))
    assert all(s[1] == TILES for s in state)
