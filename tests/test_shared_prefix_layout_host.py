"""The SMs that attention behind a shared prefix gives to the prefix belong to the splits of the call."""
import pytest

import paged_kv_attention_20_gb300 as pka
from launch_fakes import consecutive, fakes  # noqa: F401

SMS = 152


def call(fakes, queries, shared, own, hq, splits):  # noqa: F811
    lens = [shared + own] * queries
    table, pool = consecutive(lens, 16, shared)
    plan = fakes.plan(lens, table, [(s, n - 1) for s, n in enumerate(lens)], 16, pool)
    fakes.reset()
    assert fakes.forward_shared(plan, hq, 8, shared, splits) == 0
    launches = {e.name: e for e in fakes.events() if e.name not in ("record", "wait")}
    assert launches["prefix"].splits == splits[0] and launches["decode"].splits == splits[1] and launches["decode"].a == shared
    assert launches["merge"].splits == sum(splits)
    return launches["prefix"].max_ctas, launches["decode"].max_ctas


# (queries, shared, own, query heads, prefix splits): the prefix's SMs, those that a sweep over the share found best or within
# a few per cent of it (0: one after the other).  Eight KV heads.
CASES = [
    (64, 16384, 1, 32, 9, 144), (64, 16384, 1, 32, 4, 64), (64, 16384, 500, 32, 4, 64), (64, 16384, 500, 32, 9, 72),
    (64, 16384, 2048, 32, 4, 64), (64, 16384, 2048, 32, 3, 48), (64, 16384, 2048, 32, 2, 32),
    (64, 16384, 1, 64, 2, 64), (64, 16384, 1, 64, 3, 96), (64, 16384, 1, 64, 4, 0),
    (64, 16384, 2048, 64, 2, 32), (16, 16384, 1, 64, 12, 96), (16, 16384, 1, 64, 18, 0), (16, 4096, 1, 32, 12, 96),
]


@pytest.mark.parametrize("queries,shared,own,hq,prefix_splits,share", CASES)
def test_share(fakes, queries, shared, own, hq, prefix_splits, share):  # noqa: F811
    assert call(fakes, queries, shared, own, hq, (prefix_splits, 1)) == (share, SMS - share if share else 0)


@pytest.mark.parametrize("hq", [32, 56, 64, 128])
@pytest.mark.parametrize("own", [1, 300, 1500, 6000])
def test_share_fits_the_units(fakes, hq, own):  # noqa: F811
    """No SM of the share is without a unit, none of the prefix's rounds is all but empty, and the own keys keep eight SMs."""
    for queries in (3, 16, 48, 100):
        for splits in ((1, 1), (2, 1), (5, 2), (9, 1), (16, 3), (31, 8)):
            units = -(-queries // (128 // (hq // 8))) * 8 * splits[0]
            share, rest = call(fakes, queries, 8192, own, hq, splits)
            assert (share, rest) == (0, 0) or (rest == SMS - share >= 8 and share <= units
                                               and any(share == -(-units // r) for r in range(1, 9)))


def test_splits_chosen(fakes):  # noqa: F811
    """As many as end soonest for the share that the call then takes: single rounds of groups of 8 leave the own keys' persistent
    kernel SMs enough."""
    for hq, queries, own, most in ((64, 16, 1, 16), (64, 64, 1, 3), (32, 64, 2048, 6)):
        lens = [16384 + own] * queries
        table, pool = consecutive(lens, 16, 16384)
        p = pka.paged_attn_plan(lens, table, list(range(queries)), [n - 1 for n in lens], 16, pool, upload=False)
        a, b = pka.paged_attn_shared_splits(p, hq, 8, 16384, num_sms=SMS)
        assert 2 <= a <= most and b == 1, (a, b)
