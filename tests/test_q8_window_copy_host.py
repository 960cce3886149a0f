"""Prompt chunks over the 8-bit cache under a window: only what the window lets them see is copied."""
import pytest

import paged_kv_attention_20_gb300 as pka
from launch_fakes import consecutive, fakes  # noqa: F401

PAGE = 128 * 8 * 128 * 2          # bytes of a page of the copy, one tensor


def chunk(lens, chunks):
    table, pool = consecutive(lens, 16)
    return table, [(s, p) for s, r in chunks for p in r], pool


def up(n):
    return -(-n // 256) * 256


@pytest.mark.parametrize("window", [0, 1, 100, 1000, 1 << 20])
@pytest.mark.parametrize("lens,chunks", [([32768], [(0, range(32256, 32768))]), ([5000, 700, 300], [(0, range(4000, 4020)), (2, range(100, 300))]),
                                         ([2000] * 3, [(0, range(0, 2000)), (1, range(1500, 1516)), (1, range(1800, 1900))])])
def test_workspace_and_rows_read(fakes, window, lens, chunks):  # noqa: F811
    table, queries, pool = chunk(lens, chunks)
    first = {}
    for s, r in chunks:
        first[s] = min(first.get(s, r[0]), r[0])
    start = {s: max(0, p - window + 1) // 128 * 128 if window else 0 for s, p in first.items()}
    blocks = sum(-(-lens[s] // 128) - j // 128 for s, j in start.items())
    longest = max(lens[s] - j for s, j in start.items())
    host = pka.paged_attn_plan(lens, table, [s for s, _ in queries], [p for _, p in queries], 16, pool, upload=False)
    lists = up(8 * len(lens)) + up(4 * len(lens) * -(-len(table[0]) * 16 // 128))
    need = pka.q8_workspace_bytes(host, 32, 8, 128, 128, 1, window=window)
    assert need == lists + 2 * blocks * PAGE
    assert pka.q8_workspace_bytes(host, 32, 8, 128, 128, 1, window=window, max_keys=10 ** 6) == lists + 2 * PAGE * (-(-10 ** 6 // 128) + len(first))
    assert pka.q8_workspace_bytes(host, 32, 8, 128, 128, 1, window=-1) == 0
    plan = fakes.plan(lens, table, queries, 16, pool)
    for given in (need, need + 2 * 5 * PAGE):
        fakes.reset()
        assert fakes.forward_q8(plan, 32, 8, window=window, ws_bytes=given) == 0
        events = {e.name: e for e in fakes.events()}
        room = blocks + (given - need) // (2 * PAGE)
        assert (events["q8_places"].a, events["q8_places"].b) == (room, window)
        assert events["q8_load"].a == longest and events["prefill"].a == room
    assert fakes.forward_q8(plan, 32, 8, window=window, ws_bytes=need - 1) == 6


def test_share_of_the_decode_items(fakes):  # noqa: F811
    """The copy that comes before the tiles is what the model of both streams counts: without it the tiles get more time."""
    lens = [60000] * 4 + [8000] * 100
    table, queries, pool = chunk(lens, [(s, range(59488, 60000)) for s in range(4)] + [(s, range(7999, 8000)) for s in range(4, 104)])
    plan = fakes.plan(lens, table, queries, 16, pool)
    share = {}
    for window in (0, 8000):
        fakes.reset()
        assert fakes.forward_q8(plan, 32, 8, window=window) == 0
        share[window] = next(e.max_ctas for e in fakes.events() if e.name == "q8_decode_tc")
    # eight thousand keys a query for both: what differs is 4 x 60000 copied keys or 4 x 8600
    short = [8511] * 4 + [8000] * 100
    table, queries, pool = chunk(short, [(s, range(7999, 8511)) for s in range(4)] + [(s, range(7999, 8000)) for s in range(4, 104)])
    plan = fakes.plan(short, table, queries, 16, pool)
    fakes.reset()
    assert fakes.forward_q8(plan, 32, 8, window=8000) == 0
    assert abs(next(e.max_ctas for e in fakes.events() if e.name == "q8_decode_tc") - share[8000]) <= 1
