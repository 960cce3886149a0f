"""What the library sets up once holds for one device: every device a process uses gets its own.

A kernel's shared-memory attribute counts for the device that was current when it was set, and so do resident CTAs and SM
counts; a guard that is set once a process leaves every other device's launches to fail.  The class that keeps such values is
compiled for the host here and driven with device numbers; the sources are searched for guards of the other kind.
"""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_attention_20_gb300", "csrc")


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    so = str(tmp_path_factory.mktemp("probe") / "per_device_probe.so")
    subprocess.run([nvcc, "-O2", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", CSRC,
                    os.path.join(ROOT, "tests", "native", "per_device_probe.cu"), "-o", so], check=True)
    return ctypes.CDLL(so)


def test_each_device_has_its_value(probe):
    setups = ctypes.c_int(0)
    call = lambda dev, fresh: probe.probe_per_device(dev, fresh, ctypes.byref(setups))   # noqa: E731
    assert call(0, 152) == 152 and setups.value == 1
    assert call(1, 148) == 148 and setups.value == 2           # another device: set up too
    assert call(0, 7) == 152 and call(1, 7) == 148 and setups.value == 2
    assert call(2, 0) == -1 and call(2, 5) == 5 and setups.value == 4       # a failure is not kept
    assert call(64, 9) == 9 and call(64, 10) == 10 and setups.value == 6    # past the table: every time
    assert probe.probe_per_device_threads(8) == 0


def test_no_guard_for_the_whole_process():
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            found = re.findall(r"^\s+static (?:int|bool|int32_t \*)\s*\w+(?:\[\w+\])? = .*$", f.read(), re.M)
        assert not found, (name, found)
