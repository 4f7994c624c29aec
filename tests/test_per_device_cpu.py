"""What the launches set up once, they set up once on each device (the library's own header, with a
stand-in for the CUDA call)."""
import ctypes as C
import glob
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dropless_moe_expert_router_gb300", "csrc")
SOURCE = """
#include "per_device.h"
static moe_host::PerDevice smem, wave;
static int calls = 0;
extern "C" int count() { return calls; }
extern "C" int reach(int device, int value, int works) {
    return smem.reach(device, value, [&](int) { calls++; return works != 0; });
}
extern "C" int get(int device, int value) { return wave.get(device, [&] { calls++; return value; }); }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("per_device")
    src, so = str(d / "t.cpp"), str(d / "t.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.check_call([cxx, "-std=c++17", "-O2", "-shared", "-fPIC", "-I", CSRC, src, "-o", so])
    return C.CDLL(so)


def test_each_device_is_set_up(lib):
    n = lib.count()
    for device in (0, 1, 0, 1, 1):
        assert lib.reach(device, 1000, 1) == 1
    assert lib.count() == n + 2                       # once on either
    assert lib.reach(0, 900, 0) == 1 and lib.count() == n + 2
    assert lib.reach(0, 2000, 1) == 1 and lib.reach(1, 1500, 1) == 1 and lib.count() == n + 4
    assert lib.reach(0, 2000, 0) == 1 and lib.count() == n + 4


def test_a_failure_is_told_and_tried_again(lib):
    n = lib.count()
    assert lib.reach(5, 10, 0) == 0 and lib.reach(5, 10, 0) == 0 and lib.count() == n + 2
    assert lib.reach(5, 10, 1) == 1 and lib.reach(5, 10, 0) == 1 and lib.count() == n + 3


def test_devices_beyond_the_table_are_set_up_each_time(lib):
    n = lib.count()
    for device in (64, 1000, -1):
        assert lib.reach(device, 10, 1) == 1 and lib.reach(device, 10, 1) == 1 and lib.reach(device, 10, 0) == 0
        assert lib.get(device, 7) == 7 and lib.get(device, 8) == 8
    assert lib.count() == n + 15


def test_numbers_by_device(lib):
    n = lib.count()
    assert lib.get(0, 152) == 152 and lib.get(1, 304) == 304 and lib.get(0, 9) == 152 and lib.get(1, 9) == 304
    assert lib.count() == n + 2
    assert lib.get(2, 0) == 0 and lib.get(2, 6) == 6 and lib.count() == n + 4


def test_no_launch_remembers_for_the_whole_process():
    """No static flag or number of a launch is shared by the devices."""
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        with open(path) as f:
            assert not re.findall(r"^\s+static (?:bool|int|unsigned|size_t) \w+ = .*", f.read(), re.M), path
