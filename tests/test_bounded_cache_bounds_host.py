"""Bounds of the operators around a bounded cache that the host checks before it looks at a device pointer.

Plans are built on the host and bound to made-up device addresses, which nothing dereferences: each call ends with the
status of the first check that fails, or with PA_ERR_STATE for a plan that no upload followed.
"""
from test_cache_ops_host import CONFLICT, FAKE, SHAPE, STATE, plan


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
