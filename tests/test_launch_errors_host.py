"""A launch that fails leaves nothing in flight beside the caller's stream."""
import pytest

from launch_fakes import STREAM, consecutive, fakes  # noqa: F401

CUDA = 9


def mixed(fakes):
    """Prompt chunks and decode items that are worth a stream each."""
    lens = [4600] * 8 + [4000] * 120
    table, pool = consecutive(lens, 16)
    return fakes.plan(lens, table, [(s, p) for s in range(8) for p in range(4088, 4600)] + [(s, 3999) for s in range(8, 128)], 16, pool)


def behind_a_prefix(fakes):
    lens = [16384 + 400] * 64
    table, pool = consecutive(lens, 16, 16384)
    return fakes.plan(lens, table, [(s, 16384 + 399) for s in range(64)], 16, pool)


CALLS = {
    "8-bit": (mixed, lambda f, p: f.forward_q8(p, 32, 8, splits=2), ["q8_places", "q8_load", "prefill", "q8_decode_tc", "merge"]),
    "16-bit": (mixed, lambda f, p: f.forward(p, 32, 8, splits=2), ["prefill", "decode", "merge"]),
    "shared": (behind_a_prefix, lambda f, p: f.forward_shared(p, 32, 8, 16384, (4, 1)), ["prefix", "decode", "merge"]),
}


def beside(events):
    """Streams that hold work which the caller's stream has not been made to wait for."""
    open_, recorded = set(), {}
    for e in events:
        if e.name == "record":
            recorded[e.event] = e.stream
        elif e.name == "wait":
            if e.stream == STREAM:
                open_.discard(recorded[e.event])
            else:
                open_.add(e.stream)                   # a side stream in the caller's order (or capture)
        elif e.stream != STREAM:
            open_.add(e.stream)
    return open_


@pytest.mark.parametrize("capturing", [False, True])
@pytest.mark.parametrize("name", CALLS)
def test_side_stream_is_joined(fakes, name, capturing):  # noqa: F811
    build, call, launches = CALLS[name]
    plan = build(fakes)
    fakes.reset()
    assert call(fakes, plan) == 0
    fakes.reset(capturing=capturing)
    assert call(fakes, plan) == 0
    events = fakes.events()
    assert [e.name for e in events if e.stream not in (STREAM, 0)].count("wait") == 1          # it does use a second stream
    assert sorted(e.name for e in events if e.name not in ("record", "wait")) == sorted(launches) and not beside(events)
    for fails in launches:
        fakes.reset(fails, capturing)
        assert call(fakes, plan) == CUDA
        assert not beside(fakes.events()), fails
        assert b"a fake's error" in fakes.lib.pa_last_error()


@pytest.mark.parametrize("name", CALLS)
def test_calls_during_a_capture_of_another_stream(fakes, name):  # noqa: F811
    """The second stream stays with the capture that it joined until that ends; other calls of the thread do without it."""
    build, call, launches = CALLS[name]
    plan = build(fakes)
    fakes.reset()
    assert call(fakes, plan) == 0                     # (it is there)
    fakes.reset(capturing=True)
    assert call(fakes, plan) == 0
    for stream, capture in ((78, 0), (79, 2), (STREAM, 1), (78, 0)):
        seen = len(fakes.events())
        fakes.lib.fake_capture(stream, capture)
        fakes.stream = stream
        assert call(fakes, plan) == 0
        events = fakes.events()[seen:]
        assert sorted(e.name for e in events if e.name not in ("record", "wait")) == sorted(launches)
        beside_it = {e.stream for e in events} - {stream}
        assert bool(beside_it) == (stream == STREAM)
    fakes.reset()                                     # the captures have ended
    fakes.stream = 78
    assert call(fakes, plan) == 0 and {e.stream for e in fakes.events()} != {78}
