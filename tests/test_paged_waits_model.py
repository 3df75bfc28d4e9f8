"""How warps that wait on one another leave the attention kernel of chunks when a wait
gives up, as a model: every interleaving of the warps' steps, every wait that is not
over free to give up.  A barrier has no limit of its own, so none may be left with a warp
in it and another gone; and a CTA waits for the copies that it has asked for (again with a
limit) before it leaves, whoever gave up."""
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


def left_with_copies(blocks, ring, drain):
    """Whether a CTA can leave with a copy in flight for which no wait was begun.  A
    producer asks for `blocks` copies into `ring` places, a consumer takes them in order;
    any wait that is not over may give up, and sets the CTA's word of failure.
    drain(producer_failed, failed): whether the last `ring` copies are waited for before
    the CTA leaves."""
    # asked, landed, taken, producer: go / failed / done, consumer: the same
    start = (0, 0, 0, "go", "go")
    seen, todo = {start}, [start]
    while todo:
        asked, landed, taken, prod, cons = todo.pop()
        failed = "failed" in (prod, cons)
        after = []
        if landed < asked:
            after.append((asked, landed + 1, taken, prod, cons))
        if prod == "go":
            if asked == blocks:
                after.append((asked, landed, taken, "done", cons))
            elif asked - taken < ring:
                after.append((asked + 1, landed, taken, prod, cons))
            else:
                after.append((asked, landed, taken, "failed", cons))
        if cons == "go":
            if taken == blocks:
                after.append((asked, landed, taken, prod, "done"))
            elif landed > taken:
                after.append((asked, landed, taken + 1, prod, cons))
            else:
                after.append((asked, landed, taken, prod, "failed"))
        if prod != "go" and cons != "go" and landed < asked:
            if not drain(prod == "failed", failed):
                return True
        for x in after:
            if x not in seen:
                seen.add(x)
                todo.append(x)
    return False


@pytest.mark.parametrize("blocks,ring", [(1, 3), (3, 3), (7, 3), (9, 5)])
def test_copies_in_flight_are_waited_for(blocks, ring):
    assert not left_with_copies(blocks, ring, lambda producer, anyone: True)
    # the planted mistake: only where the producer itself gave up
    assert left_with_copies(blocks, ring, lambda producer, anyone: producer)
