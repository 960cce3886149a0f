"""Bounds of the operators around a bounded cache that the host checks before it looks at a device pointer.

Plans are built on the host and bound to made-up device addresses, which nothing dereferences: each call ends with the
status of the first check that fails, or with PA_ERR_STATE for a plan that no upload followed.
"""
import numpy as np

import paged_kv_attention_20_gb300 as pka
from test_cache_ops_host import CONFLICT, FAKE, LIMIT, SHAPE, STATE, WORKSPACE, plan


def evict(lib, a, b, stride=100, sink=0, recent=0, hkv=2, d=64, dv=64, dt=2):
    return lib.paged_kv_evict(a.handle, b.handle, FAKE, FAKE, FAKE, FAKE, stride, sink, recent, hkv, d, dv, dt, None)


def test_evict_leaves_reserved_pages_alone(built_lib):
    """A plan's queries can advance on the device past the host's lengths, onto the pages its rows reserve: keys may live
    there when the eviction runs, so no kept row may be moved onto them from elsewhere."""
    src = plan([21, 30], [[0, 1, 2, 3], [4, 5, -1, -1]], [(0, 20), (1, 29)], pages=12)
    call = lambda lens, table, a=src, **kw: evict(built_lib, a, plan(lens, table, pages=12), **kw)   # noqa: E731
    assert call([12, 10], [[2], [4]]) == CONFLICT               # the sequence's own reserve, as a fresh page
    assert call([12, 10], [[0], [3]]) == CONFLICT               # another sequence's
    assert call([12, 10], [[0], [4]]) == STATE
    assert call([12, 10], [[8], [9]]) == STATE
    # a reserve ends where the advance does: at the first entry that names no page
    gap = plan([21, 30], [[0, 1, -1, 3], [4, 5, -1, -1]], [(0, 20), (1, 29)], pages=12)
    assert call([12, 10], [[3], [4]], gap) == STATE
    # without queries, or with prefill tiles, nothing advances
    assert call([12, 10], [[2], [4]], plan([21, 30], [[0, 1, 2, 3], [4, 5, -1, -1]], pages=12)) == STATE
    tile = [(0, i) for i in range(21)]
    assert call([12, 10], [[2], [4]], plan([21, 30], [[0, 1, 2, 3], [4, 5, -1, -1]], tile, pages=12)) == STATE
    # a sequence that no query names stays as it is
    assert call([12, 10], [[2], [4]], plan([21, 30], [[0, 1, 2, 3], [4, 5, -1, -1]], [(1, 29)], pages=12)) == STATE
    # padding that names a page in use reserves nothing
    zeros = plan([21, 30], [[1, 2, 0, 0], [0, 3, 0, 0]], [(0, 20), (1, 29)], pages=12)
    assert call([12, 17], [[1, 0], [0, 3]], zeros) == STATE


def test_evict_budget_above_the_host_length(built_lib):
    """A budget up to what the sequence's pages hold: the device's length may have reached it."""
    src = plan([21, 30], [[0, 1, 2, 3], [4, 5, -1, -1]], [(0, 20), (1, 29)], pages=12)
    call = lambda lens, table, a=src: evict(built_lib, a, plan(lens, table, pages=12))   # noqa: E731
    rows = [[0, 1, 2, 3], [4, 5, -1, -1]]
    assert call([30, 30], rows) == STATE and call([64, 32], rows) == STATE
    assert call([30, 30], [[8, 9], [10, 11]]) == STATE
    assert call([40, 30], [[0, 1, 8], [4, 5, -1]]) == STATE
    assert call([64, 33], [[0, 1, 2, 3], [4, 5, 6, -1]]) == SHAPE       # its pages hold 32
    still = plan([21, 30], [[0, 1, 2, 3], [4, 5, -1, -1]], pages=12)
    assert call([22, 30], rows, still) == SHAPE                         # nothing can have advanced
    # a reserved page is moved into in place, and another row reserves it too
    both = plan([16, 16], [[0, 2], [1, 2]], [(0, 15), (1, 15)], pages=12)
    assert call([20, 10], [[0, 2], [1, -1]], both) == CONFLICT


def forward_mass(lib, p, hq=4, hkv=2, d=64, dv=64, window=0, dt=2, nbytes=2 ** 63, splits=1):
    return lib.paged_attn_forward_mass(p.handle, FAKE, FAKE, FAKE, FAKE, FAKE, hq, hkv, d, dv, 0.1, 1, window, dt, FAKE, nbytes,
                                       splits, None)


def test_forward_mass_rows_past_32_bits(built_lib):
    """(query, head, split) rows are counted in 32 bits: more of them are refused, and their score rows, whose bytes can
    leave 64 bits, ask for no workspace."""
    def ones(n):
        return plan([1] * n, [[i] for i in range(n)], [(i, 0) for i in range(n)], ps=1, pages=n)
    few, more, many = ones(512), ones(513), ones(1 << 17)
    call = lambda p, **kw: forward_mass(built_lib, p, **{**dict(hq=65535, hkv=1, d=1, dv=1), **kw})   # noqa: E731
    assert call(few, splits=64) == STATE               # 2147450880 rows
    assert call(more, splits=64) == LIMIT
    assert call(many) == LIMIT and call(many, hq=16383) == STATE
    size = lambda p, heads, **kw: pka.mass_workspace_bytes(p, heads, 1, 1, **{**dict(splits=1), **kw})   # noqa: E731
    assert size(more, 65535, splits=64) == 0 and size(few, 65535, splits=64) > 64 * 512 * 65535 * 8
    assert size(many, 65535) == 0
    far = 2 ** 31 - 1
    assert size(many, 65535, max_keys=far) == 0        # 2^66 bytes of scores
    assert size(many, 16383, max_keys=far) == 0        # just below 2^64
    assert size(many, 16, max_keys=far) > 2 ** 17 * 16 * far * 4


def test_forward_mass_scores_past_any_workspace(built_lib):
    """32768 items of one history of 2^30 keys with 65535 heads: 2^63 bytes of scores, and no workspace is that large."""
    n = 1 << 15
    queries = [(0, (1 << 30) - 1 - 2 * i) for i in range(n)]
    p = plan([1 << 30], [list(range(1024))], queries, ps=1 << 20, pages=1024)
    assert pka.mass_workspace_bytes(p, 65535, 1, 1, 1) == 0
    for nbytes in (2 ** 62, 2 ** 63, 2 ** 64 - 1):
        assert forward_mass(built_lib, p, hq=65535, hkv=1, d=1, dv=1, nbytes=nbytes) == WORKSPACE


def test_forward_mass_long_chunks(built_lib):
    """Histories above 2^30 keys are refused for prompt chunks too: the kernels step through keys in 32 bits."""
    def chunk(n, extra=()):
        return plan([n], [list(range(1025))], [(0, n - 16 + i) for i in range(16)] + list(extra), ps=1 << 20, pages=1025)
    at, above = chunk(1 << 30), chunk((1 << 30) + 1)
    for kw in (dict(dt=2, d=128, dv=128), dict(dt=0, d=8, dv=8)):       # (neither has tensor-core tiles at this page size)
        assert forward_mass(built_lib, at, **kw) == STATE
        assert forward_mass(built_lib, above, **kw) == LIMIT


def test_evict_sizes_past_32_bits(built_lib):
    """kept rows and histories above 2^30 keys, which the kernels would step through past 32 bits."""
    src, kept = plan([40, 30], [[0, 1, 2], [3, 4, -1]]), plan([20, 10], [[0, 1], [3, -1]])
    assert evict(built_lib, src, kept, stride=1 << 30) == STATE
    assert evict(built_lib, src, kept, stride=(1 << 30) + 1) == LIMIT
    assert evict(built_lib, src, kept, stride=2 ** 31 - 1) == LIMIT
    long = lambda n: plan([n], [list(range(1025))], ps=1 << 20, pages=1025)   # noqa: E731
    short = plan([100], [[0]], ps=1 << 20, pages=1025)
    assert evict(built_lib, long(1 << 30), short, hkv=1, d=8, dv=8) == STATE
    assert evict(built_lib, long((1 << 30) + 1), short, hkv=1, d=8, dv=8) == LIMIT


def test_evict_lists_past_the_grid(built_lib):
    """So many (sequence, head) lists and column slices that a launch cannot number them: refused before any launch."""
    n = 1 << 21
    table = np.full((n, 1), -1, np.int32)
    lens = np.zeros(n, np.int32)
    table[0], lens[0] = 3, 9
    src = plan(lens, table)
    kept = plan(lens, table)
    assert evict(built_lib, src, kept, hkv=8, d=1024, dv=1024, dt=0) == STATE
    assert evict(built_lib, src, kept, hkv=64, d=1024, dv=1024, dt=0) == LIMIT      # 2^27 lists of 32 slices or more
    assert evict(built_lib, src, kept, hkv=256, d=8, dv=8) == LIMIT                 # 2^29 lists
