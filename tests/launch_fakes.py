"""The library's entry points over fakes of its kernels and of the CUDA runtime (native/launch_fakes.cpp), on the CPU."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess
from collections import namedtuple

import pytest

import paged_kv_attention_20_gb300 as pka

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_attention_20_gb300", "csrc")
FAKE = 1 << 40          # operands: an address for each, far apart, never dereferenced
SIZE = 1 << 40
STREAM = 77

Event = namedtuple("Event", "name stream event splits max_ctas a b")


class Fakes:
    def __init__(self, so: str):
        self.lib = ctypes.CDLL(so)
        real = pka.load()
        for name in pka.EXPORTED:
            f, r = getattr(self.lib, name), getattr(real, name)
            f.argtypes, f.restype = r.argtypes, r.restype
        i64 = ctypes.c_int64
        self.lib.fake_event.argtypes = [ctypes.c_int, ctypes.POINTER(i64), ctypes.POINTER(i64), ctypes.POINTER(i64)]
        self.lib.fake_event.restype = ctypes.c_char_p
        self.lib.fake_capture.argtypes = [i64, i64]
        self.stream = STREAM

    def reset(self, fails: str = "", capturing: bool = False, tensor_cores: bool = True) -> None:
        self.lib.fake_reset(fails.encode(), int(tensor_cores))
        self.lib.fake_capture(STREAM, int(capturing))
        self.stream = STREAM

    def events(self) -> list[Event]:
        found = []
        for i in range(self.lib.fake_events()):
            stream, event, value = ctypes.c_int64(), ctypes.c_int64(), (ctypes.c_int64 * 4)()
            name = self.lib.fake_event(i, ctypes.byref(stream), ctypes.byref(event), value).decode()
            found.append(Event(name, stream.value, event.value, *value))
        return found

    def plan(self, lens, table, queries, ps, pages):
        """A plan bound to a made-up device buffer; queries: (sequence, position)."""
        arr = lambda a: (ctypes.c_int32 * max(1, len(a)))(*a)                       # noqa: E731
        flat = [x for row in table for x in row]
        handle = ctypes.c_void_p()
        assert self.lib.paged_attn_plan(arr(lens), len(lens), arr(flat), len(table[0]), arr([s for s, _ in queries]),
                                        arr([p for _, p in queries]), len(queries), ps, pages, ctypes.byref(handle)) == 0
        assert self.lib.pa_plan_upload(handle, FAKE, SIZE, None) == 0
        return handle

    def operands(self, n: int) -> list[int]:
        return [FAKE + (i + 1) * SIZE for i in range(n)]

    def forward_q8(self, plan, hq, hkv, d=128, splits=1, causal=1, window=0, dtype=2, ws_bytes=SIZE):
        q, k, v, ks, vs, out, ws = self.operands(7)
        return self.lib.paged_attn_forward_q8(plan, q, k, v, ks, vs, out, hq, hkv, d, d, 0.1, causal, window, dtype, ws, ws_bytes,
                                              splits, self.stream)

    def forward_shared(self, plan, hq, hkv, shared, splits, d=128, causal=1, dtype=2):
        q, k, v, out, ws = self.operands(5)
        return self.lib.paged_attn_forward_shared(plan, q, k, v, out, hq, hkv, d, d, 0.1, causal, shared, dtype, ws, SIZE,
                                                  splits[0], splits[1], self.stream)

    def forward(self, plan, hq, hkv, d=128, splits=1, causal=1, window=0, dtype=2):
        q, k, v, out, ws = self.operands(5)
        return self.lib.paged_attn_forward_split(plan, q, k, v, out, hq, hkv, d, d, 0.1, causal, window, dtype, ws, SIZE, splits,
                                                 self.stream)


@pytest.fixture(scope="session")
def fakes(built_lib, tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    cxx = shutil.which("g++")
    if not os.path.exists(nvcc) or cxx is None:
        pytest.skip("nvcc's headers or g++ not found")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    so = str(tmp_path_factory.mktemp("fakes") / "entry_points.so")
    files = [os.path.join(CSRC, f) for f in ("plan.cpp", "cache_ops.cpp", "q8_ops.cpp", "shared_ops.cpp")]
    subprocess.run([cxx, "-O1", "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", cuda, *files,
                    os.path.join(ROOT, "tests", "native", "launch_fakes.cpp"), "-o", so, "-Wl,--no-undefined,-Bsymbolic"], check=True)
    return Fakes(so)


def consecutive(lens, ps, shared=0):
    """A block table of pages of their own behind `shared` common ones, and the pool's size."""
    first = shared // ps
    used = [-(-n // ps) - first for n in lens]
    at, rows, width = first, [], first + max(used + [0])
    for u in used:
        rows.append(list(range(first)) + list(range(at, at + u)) + [-1] * (width - first - u))
        at += u
    return rows, at
