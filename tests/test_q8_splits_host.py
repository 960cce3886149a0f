"""How many of the splits that a caller allows the 8-bit attention takes."""
import pytest

from launch_fakes import consecutive, fakes  # noqa: F401

F32, BF16 = 0, 2


def taken(fakes, lens, queries, hq=32, hkv=8, splits=16, tensor_cores=True, capturing=False, width=None, **kw):  # noqa: F811
    """The splits of the decode launch and of the merge (None: no merge)."""
    table, pool = consecutive(lens, 16)
    if width:
        table = [row[:width] + [-1] * (width - len(row)) for row in table]
    plan = fakes.plan(lens, table, queries, 16, pool)
    fakes.reset(capturing=capturing, tensor_cores=tensor_cores)
    assert fakes.forward_q8(plan, hq, hkv, splits=splits, **kw) == 0
    events = {e.name: e for e in fakes.events()}
    decode = events.get("q8_decode_tc") or events["q8_decode_any"]
    return decode.splits, events["merge"].splits if "merge" in events else None


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_window_without_a_causal_end(fakes, dtype):  # noqa: F811
    """A query at a low position of a long history sees from its window's start to the history's end."""
    kw = dict(splits=16, dtype=dtype, tensor_cores=dtype == BF16)
    whole = taken(fakes, [100000], [(0, 99999)], **kw)
    assert whole[0] > 8 and whole[1] == whole[0]
    assert taken(fakes, [100000], [(0, 50)], causal=0, window=100, **kw) == whole
    # at the history's end the window is all there is, and with a causal end always
    for pos, causal in ((99999, 0), (99999, 1), (50, 1), (5000, 1)):
        assert taken(fakes, [100000], [(0, pos)], causal=causal, window=100, **kw) == (1, None)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_keys_behind_the_query_do_not_count(fakes, dtype):  # noqa: F811
    """Early positions of long histories (a prompt checked again, say) are short."""
    kw = dict(splits=16, dtype=dtype, tensor_cores=dtype == BF16)
    assert taken(fakes, [100000], [(0, 120)], **kw) == taken(fakes, [121], [(0, 120)], **kw) == (1, None)
    assert taken(fakes, [100000, 300], [(0, 4000), (1, 20)], **kw) == taken(fakes, [4001, 21], [(0, 4000), (1, 20)], **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_captured_calls_may_see_longer_histories(fakes, dtype):  # noqa: F811
    """As many splits as for histories that fill the block table, whatever the lengths at the capture."""
    kw = dict(splits=16, dtype=dtype, tensor_cores=dtype == BF16)
    long = taken(fakes, [32768], [(0, 32767)], **kw)
    assert long[0] > 8
    for now in (1, 200, 5000, 32768):
        assert taken(fakes, [32768], [(0, now - 1)], capturing=True, **kw) == long
    # one table row grown from 200 keys to what it can hold
    table = [list(range(2048))]
    plan = fakes.plan([200], table, [(0, 199)], 16, 2048)
    fakes.reset(capturing=True, tensor_cores=dtype == BF16)
    assert fakes.forward_q8(plan, 32, 8, splits=16, dtype=dtype) == 0
    assert fakes.events()[0].splits == long[0]
    fakes.reset(tensor_cores=dtype == BF16)
    assert fakes.forward_q8(plan, 32, 8, splits=16, dtype=dtype) == 0
    assert fakes.events()[0].splits == 1                      # not captured: by the lengths it has
    # a window is all that a causal query ever sees
    assert taken(fakes, [32768], [(0, 199)], capturing=True, window=100, **kw) == (1, None)
    assert taken(fakes, [32768], [(0, 199)], capturing=True, window=100, causal=0, **kw) == long


def test_captured_at_full_length_is_as_not_captured(fakes):  # noqa: F811
    for lens in ([131072], [8000] * 64, [2000] * 4, [500] * 16, [32768, 50000, 90000, 131072]):
        queries = [(s, n - 1) for s, n in enumerate(lens)]
        for hq in (32, 64):
            assert taken(fakes, lens, queries, hq=hq, splits=64) == taken(fakes, lens, queries, hq=hq, splits=64, capturing=True)


def test_no_more_than_allowed(fakes):  # noqa: F811
    for lens in ([131072], [300, 9000, 40000], [200] * 4, [8000] * 64):
        queries = [(s, n - 1) for s, n in enumerate(lens)]
        for splits in (1, 2, 5, 64):
            s, merged = taken(fakes, lens, queries, splits=splits)
            assert 1 <= s <= splits and merged == (s if s > 1 else None)


def test_a_stream_that_cannot_be_asked(fakes):  # noqa: F811
    """The legacy stream while another thread captures, say: taken for a captured one, and no error is left behind."""
    plan = fakes.plan([200], [list(range(2048))], [(0, 199)], 16, 2048)
    fakes.reset("is_capturing")
    assert fakes.forward_q8(plan, 32, 8, splits=16) == 0
    assert fakes.events()[0].splits > 8 and fakes.lib.cudaGetLastError() == 0
