"""How the shared-prefix attention cuts its units over lanes (csrc/sp_lanes.h),
compiled for the host: the lane that the merge looks a unit up in has to be the
lane whose range holds it, for unit counts on both sides of 2^32."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = """
#include "sp_lanes.h"
extern "C" long long begin_of(long long units, int lanes, int l) { return thd::lane_begin(units, lanes, l); }
extern "C" int lane_of(long long units, int lanes, long long x) { return thd::lane_of(units, lanes, x); }
"""


@pytest.fixture(scope="module")
def lanes_lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("lanes")
    (d / "lanes.cpp").write_text(SOURCE)
    so = d / "lanes.so"
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-I", os.path.join(ROOT, "sliding_window_gqa_cu_b200", "csrc"),
                    "-o", str(so), str(d / "lanes.cpp")], check=True)
    lib = ctypes.CDLL(str(so))
    i64 = ctypes.c_int64
    lib.begin_of.argtypes, lib.begin_of.restype = [i64, ctypes.c_int, ctypes.c_int], i64
    lib.lane_of.argtypes, lib.lane_of.restype = [i64, ctypes.c_int, i64], ctypes.c_int
    return lib


# (1,048,576 own tokens of a request with 131,072 queries on 8 kv heads: 8,192
# row tiles x 8 heads x 65,537 units are just above 2^32)
UNITS = [1, 5, 1776, 1777, 100003, 2 ** 31 - 1, 2 ** 31, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + 1, 2 ** 32 + 1775,
         8192 * 8 * 65537, 3 * 2 ** 32, 2 ** 40 + 12345]


@pytest.mark.parametrize("units,lanes", [(u, n) for u in UNITS for n in (1, 2, 37, 148, 1775, 1776) if n <= u])
def test_the_lane_of_a_unit_is_the_one_whose_range_holds_it(lanes_lib, units, lanes):
    begin, lane_of = lanes_lib.begin_of, lanes_lib.lane_of
    assert begin(units, lanes, 0) == 0 and begin(units, lanes, lanes) == units
    some = set(range(min(units, 50))) | {units - 1, units // 2, units // 3}
    for l in range(lanes):                              # both sides of every border
        at = begin(units, lanes, l)
        assert at == units * l // lanes
        some |= {x for x in (at - 1, at, at + 1) if 0 <= x < units}
    for x in some:
        l = lane_of(units, lanes, x)
        assert 0 <= l < lanes and begin(units, lanes, l) <= x < begin(units, lanes, l + 1), (units, lanes, x, l)
