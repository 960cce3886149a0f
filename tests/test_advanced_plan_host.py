"""What a call works out from a plan's lengths follows the host copy when the plan advances."""
import pytest

from launch_fakes import consecutive, fakes  # noqa: F401

STEPS = 1500


def pair(fakes, lens, now, shared=0):  # noqa: F811
    """A plan advanced from `lens` to `now`, and one built there."""
    table, pool = consecutive(now, 16, shared)
    built = [fakes.plan(n, table, [(s, x - 1) for s, x in enumerate(n)], 16, pool) for n in (lens, now)]
    fakes.reset()
    for _ in range(now[0] - lens[0]):
        assert fakes.lib.pa_plan_advance(built[0], None) == 0
    return built


def launches(fakes, call):  # noqa: F811
    fakes.reset()
    assert call() == 0
    return [e for e in fakes.events() if e.name not in ("record", "wait")]


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("queries,start,hq", [(4, 30, 32), (20, 400, 32), (24, 1, 32), (24, 400, 64)])
def test_splits_of_the_8_bit_cache(fakes, queries, start, hq, causal):  # noqa: F811
    lens = [start + 7 * s % 50 for s in range(queries)]
    lens[0] = max(lens)
    moved, fresh = pair(fakes, lens, [n + STEPS for n in lens])
    for splits in (2, 19, 64):
        a, b = (launches(fakes, lambda p=p: fakes.forward_q8(p, hq, 8, splits=splits, causal=causal)) for p in (moved, fresh))
        assert a == b


def test_share_behind_a_prefix(fakes):  # noqa: F811
    lens = [16384 + 1] * 64
    moved, fresh = pair(fakes, lens, [n + STEPS for n in lens], 16384)
    for splits in ((2, 1), (4, 1), (9, 2)):
        a, b = (launches(fakes, lambda p=p: fakes.forward_shared(p, 32, 8, 16384, splits)) for p in (moved, fresh))
        assert a == b
