"""A CTA of the serving step that gives up waits for every copy that is still on
its way into its shared memory: the walk is replayed here with one phase counter
a stage, as the barriers have, and nothing may be left behind."""
import pytest


@pytest.fixture(scope="module")
def R():
    from bwd_persistent_cta_gb300 import build
    build.build()
    import bwd_persistent_cta_gb300 as R
    R.lib()
    return R


@pytest.mark.parametrize("turns", [1, 2, 3, 4, 5, 6, 7, 8, 9, 13, 40])
def test_give_up_waits_for_every_copy_under_way(R, turns):
    depth = 4
    for turn in range(turns):
        # before turn 0 the first ``depth`` fills start; each finished turn starts the one ``depth`` later
        started = range(min(turns, turn + depth))
        under_way = {}
        for t in started:
            if t >= turn:
                stage, fills_before = t % depth, t // depth
                under_way[stage] = fills_before & 1       # a wait for this parity ends with this fill, not the last one
        got = R.rnn_debug_step_drain(turn, turns)
        assert len(got) == len(under_way) and dict(got) == under_way, (turn, turns)


def test_turns_outside_the_walk(R):
    for turn, turns in ((-1, 3), (3, 3), (0, 0)):
        assert R.rnn_debug_step_drain(turn, turns) == []
