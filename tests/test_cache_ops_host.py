"""Refusals of the operators around a bounded cache that need no GPU.

Every status below comes before the call looks at a device pointer.
"""
import ctypes

import pytest

import paged_kv_attention_20_gb300 as pka

OK, ARG, SHAPE, DTYPE, RANGE, CONFLICT, WORKSPACE, SPLITS, LIMIT, CUDA, STATE = range(11)
FAKE = 0x10000          # bound to plans, never dereferenced


def plan(lens, table, queries=(), ps=16, pages=8, staged=False):
    p = pka.paged_attn_plan(lens, table, [s for s, _ in queries], [i for _, i in queries], ps, pages, upload=False)
    if staged:
        buf = (ctypes.c_int32 * (p.device_bytes() // 4))()
        assert pka.load().pa_plan_stage(p.handle, ctypes.addressof(buf), p.device_bytes(), FAKE, p.device_bytes()) == 0
    return p


def test_norm_rope_store(built_lib):
    base = dict(q=FAKE, qs=512, k=FAKE, ks=512, v=FAKE, vs=512, out=FAKE, kc=FAKE, vc=FAKE, mass=None, table=FAKE, far=64,
                rot=64, inter=0, pos=None, qw=None, kw=None, eps=1e-6, hq=4, hkv=2, d=128, dv=128, dt=2)
    one = plan([5], [[0]], [(0, 4)])

    def call(p=one, **kw):
        a = {**base, **kw}
        return built_lib.paged_qk_norm_rope_store(
            p.handle if p else None, a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["out"], a["kc"], a["vc"], a["mass"],
            a["table"], a["far"], a["rot"], a["inter"], a["pos"], a["qw"], a["kw"], a["eps"], a["hq"], a["hkv"], a["d"],
            a["dv"], a["dt"], None)

    assert call(None) == ARG and call(dt=3) == DTYPE
    for kw in (dict(hq=0), dict(hkv=0), dict(d=0), dict(dv=0), dict(rot=63), dict(rot=0), dict(rot=130), dict(far=0),
               dict(qs=-1), dict(ks=-1), dict(vs=-1), dict(qw=FAKE, eps=float("inf")), dict(kw=FAKE, eps=-1e-6)):
        assert call(**kw) == SHAPE, kw
    assert call(d=1025) == LIMIT and call(dv=1025) == LIMIT and call(hq=65536) == LIMIT
    assert call(inter=2) == ARG and call(table=None, pos=FAKE) == ARG
    assert call(qs=2 ** 41) == RANGE
    assert call() == STATE
    assert call(plan([5], [[0]])) == OK                       # no queries: nothing to do
    assert call(plan([5], [[0]], [(0, 4)], staged=True), q=None) == ARG


def test_forward_mass(built_lib):
    base = dict(q=FAKE, k=FAKE, v=FAKE, out=FAKE, mass=FAKE, hq=4, hkv=2, d=64, dv=64, scale=0.1, causal=1, window=0, dt=2,
                ws=FAKE, bytes=1 << 30, splits=1)
    one = plan([5], [[0]], [(0, 4)])

    def call(p=one, **kw):
        a = {**base, **kw}
        return built_lib.paged_attn_forward_mass(
            p.handle if p else None, a["q"], a["k"], a["v"], a["out"], a["mass"], a["hq"], a["hkv"], a["d"], a["dv"],
            a["scale"], a["causal"], a["window"], a["dt"], a["ws"], a["bytes"], a["splits"], None)

    assert call(None) == ARG and call(dt=9) == DTYPE and call(hq=5) == SHAPE and call(scale=0.0) == SHAPE
    assert call(window=-1) == ARG and call(causal=2) == ARG and call(d=2000) == LIMIT
    assert call(mass=None) == ARG and call(mass=FAKE + 2) == ARG
    assert call(splits=0) == SPLITS and call(splits=65) == SPLITS
    assert call(ws=None) == WORKSPACE and call(ws=FAKE + 8) == WORKSPACE and call(bytes=64) == WORKSPACE
    need = built_lib.pa_mass_workspace_bytes(one.handle, 4, 2, 64, 1, 0, 0)
    assert call(bytes=need - 1) == WORKSPACE and call(bytes=need) == STATE
    assert call(plan([20, 20], [[0, 1], [0, 2]], [(0, 19)])) == CONFLICT      # a page with two holders
    assert call(plan([20], [[3, 3]], [(0, 19)])) == CONFLICT                  # twice in one row
    assert call(plan([5], [[0]])) == OK


def test_mass_workspace_bytes(built_lib):
    p = plan([300, 40], [list(range(19)), [19, 20, 21] + [-1] * 16], [(0, 299), (1, 39)], pages=30)
    up = lambda n: -(-n // 256) * 256                                          # noqa: E731
    rows = 2 * 8
    lists = up((2 + 1 + 2) * 4)
    assert pka.mass_workspace_bytes(p, 8, 2, 128, 1) == up(rows * 4) + lists + up(rows * 320 * 4)
    assert pka.mass_workspace_bytes(p, 8, 2, 128, 3) == up(3 * rows * 128 * 4) + up(3 * rows * 4) + lists + up(rows * 320 * 4)
    assert pka.mass_workspace_bytes(p, 8, 2, 128, 1, window=50) == up(rows * 4) + lists + up(rows * 64 * 4)
    assert pka.mass_workspace_bytes(p, 8, 2, 128, 1, window=64) == up(rows * 4) + lists + up(rows * 96 * 4)   # + 3 keys
    assert pka.mass_workspace_bytes(p, 8, 2, 128, 1, window=300) == pka.mass_workspace_bytes(p, 8, 2, 128, 1)
    assert pka.mass_workspace_bytes(p, 8, 2, 128, 1, max_keys=1000) == up(rows * 4) + lists + up(rows * 1024 * 4)
    for bad in (dict(heads=0), dict(heads=7), dict(kv_heads=0), dict(value_dim=0), dict(splits=0), dict(splits=65),
                dict(window=-1), dict(max_keys=-1)):
        assert pka.mass_workspace_bytes(p, **{**dict(heads=8, kv_heads=2, value_dim=64, splits=1), **bad}) == 0


def test_evict(built_lib):
    src = plan([40, 30], [[0, 1, 2], [3, 4, -1]])
    same = [[0, 1, 2], [3, 4, -1]]

    def call(a, b, stride=100, sink=0, recent=0, hkv=2, d=64, dv=64, dt=2, mass=FAKE):
        return built_lib.paged_kv_evict(a.handle if a else None, b.handle if b else None, mass, FAKE, FAKE, FAKE, stride,
                                        sink, recent, hkv, d, dv, dt, None)

    kept = plan([20, 10], same)
    assert call(src, kept) == STATE
    assert call(None, kept) == ARG and call(src, None) == ARG and call(src, kept, dt=5) == DTYPE
    assert call(src, kept, hkv=0) == SHAPE and call(src, kept, d=0) == SHAPE and call(src, kept, dv=1025) == LIMIT
    assert call(src, kept, sink=-1) == ARG and call(src, kept, recent=-1) == ARG
    assert call(src, kept, sink=2 ** 31 - 1, recent=5) == RANGE
    assert call(src, plan([20], [[0, 1, 2]])) == SHAPE                          # another number of sequences
    assert call(src, plan([20, 10], same, pages=9)) == SHAPE
    assert call(src, plan([20, 10], [[0] * 5 + [1] * 0 + [1, 2], [3] * 5 + [4, 5]], ps=8)) == SHAPE
    assert call(src, plan([41, 10], same)) == SHAPE                             # more than it has
    assert call(src, kept, sink=8, recent=4) == SHAPE                           # a budget below sink + recent
    assert call(src, plan([40, 12], same), sink=8, recent=4) == STATE           # (an untouched sequence may be)
    assert call(src, kept, stride=19) == SHAPE
    assert call(src, plan([20, 10], [[1, 0, 2], [3, 4, -1]])) == CONFLICT       # its own pages in another order
    assert call(src, plan([20, 10], [[0, 4, 2], [3, 4, -1]])) == CONFLICT       # another sequence's page
    assert call(src, plan([20, 10], [[5, 6, -1], [6, -1, -1]])) == CONFLICT     # one fresh page twice
    assert call(src, plan([20, 10], [[5, 6, -1], [7, -1, -1]])) == STATE
    assert call(src, plan([20, 10], [[0, 6, -1], [7, -1, -1]])) == STATE        # in place and fresh, page by page
    shared = plan([40, 30], [[0, 1, 2], [0, 4, -1]])
    assert call(shared, plan([20, 16], [[0, 1, 2], [0, 4, -1]]), sink=15) == CONFLICT
    assert call(shared, plan([20, 17], [[0, 1, 2], [0, 4, -1]]), sink=16) == STATE     # the shared page stays
    assert call(shared, plan([20, 10], [[5, 6, -1], [7, -1, -1]])) == STATE            # and may be copied from
    assert call(shared, plan([40, 30], [[0, 1, 2], [0, 4, -1]])) == CONFLICT           # the device copy may be longer
    assert call(src, plan([40, 30], same)) == STATE
    staged = plan([40, 30], same, staged=True), plan([20, 10], same, staged=True)
    assert call(*staged, mass=None) == ARG
    none = plan([], [])
    assert call(none, none, stride=0) == OK


def test_evict_after_advance(built_lib):
    """The facts kept about a plan's pages follow its lengths (pa_plan_advance is refused without a device copy)."""
    p = plan([16], [[0, 0]], [(0, 15)])
    assert built_lib.pa_plan_advance(p.handle, None) == STATE


@pytest.mark.parametrize("name", ["paged_qk_norm_rope_store", "paged_attn_forward_mass", "paged_kv_evict",
                                  "make_mass_workspace", "mass_workspace_bytes"])
def test_public_names(name):
    assert callable(getattr(pka, name)) and name in pka.__all__
