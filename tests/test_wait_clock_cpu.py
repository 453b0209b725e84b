"""The rule by which a bounded wait of the packed attention gives up, in a host build."""
import ctypes
import os
import subprocess

import pytest

from cem_search_transformer_gb300 import build_lib

LIMIT = 2_000_000_000


@pytest.fixture(scope="module")
def ends_at(tmp_path_factory):
    """Time at which a wait that begins at `start` ends, polled every `poll`, for work that moves every
    `step` until `stands`; -1 where it is not over at `horizon`."""
    d = tmp_path_factory.mktemp("wait_clock")
    src, so = str(d / "clock.cpp"), str(d / "clock.so")
    with open(src, "w") as f:
        f.write('#include "wait_clock.h"\n'
                'typedef unsigned long long u64;\n'
                'extern "C" long long ends_at(u64 start, u64 poll, u64 step, u64 stands, u64 horizon, u64 limit,\n'
                '                             unsigned count0) {\n'
                '  jepa::WaitClock c(start);\n'
                '  for (u64 t = start; t <= horizon; t += poll)\n'
                '    if (c.due(t, limit) && c.stuck(t, count0 + (unsigned)((t < stands ? t : stands) / step)))\n'
                '      return (long long)t;\n'
                '  return -1;\n'
                '}\n')
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-shared", "-fPIC", "-I", build_lib.CSRC, src,
                    "-o", so], check=True)
    fn = ctypes.CDLL(so).ends_at
    fn.argtypes, fn.restype = [ctypes.c_ulonglong] * 6 + [ctypes.c_uint], ctypes.c_longlong
    return lambda start, poll, step, stands, horizon, count0=0: fn(start, poll, step, stands, horizon, LIMIT, count0)


@pytest.mark.parametrize("step", [800, 300_000, 1_900_000_000])
@pytest.mark.parametrize("count0", [0, 0xffffff00])
def test_a_wait_lasts_as_long_as_the_work_moves(ends_at, step, count0):
    assert ends_at(0, 100_000, step, 60 * LIMIT, 60 * LIMIT, count0) == -1


@pytest.mark.parametrize("stands", [0, 1, 3 * LIMIT, 7 * LIMIT + 12345])
def test_a_wait_ends_two_limits_after_the_work_stood(ends_at, stands):
    over = ends_at(0, 50_000, 800, stands, 60 * LIMIT)
    assert stands < over <= stands + 2 * LIMIT + 200_000
    assert over > LIMIT


def test_a_wait_that_begins_late_has_its_whole_limit(ends_at):
    start = 5 * LIMIT
    assert ends_at(start, 50_000, 800, 0, 60 * LIMIT) > start + LIMIT
