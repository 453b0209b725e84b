"""Which packed sequences the 8-bit cache's kernels take, in a host build of their index arithmetic."""
import ctypes
import os
import subprocess

import pytest

from cem_search_transformer_gb300 import build_lib


@pytest.fixture(scope="module")
def span_ok(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv8_span")
    src, so = str(d / "span.cpp"), str(d / "span.so")
    with open(src, "w") as f:
        f.write('#include "kv8_index.h"\n'
                'extern "C" int span_ok(int b, int e, int n) { return jepa::kv8_span_ok(b, e, n); }\n')
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-shared", "-fPIC", "-I", build_lib.CSRC, src,
                    "-o", so], check=True)
    return ctypes.CDLL(so).span_ok


@pytest.mark.parametrize("begin,end,ok", [
    (0, 0, 1), (0, 10, 1), (10, 10, 1), (3, 7, 1),
    (0, 11, 0), (10, 11, 0), (11, 11, 0), (-1, 5, 0), (-1, -1, 0), (7, 6, 0), (10, 9, 0),
    (-2 ** 31, 5, 0), (0, 2 ** 31 - 1, 0), (2 ** 31 - 1, -2 ** 31, 0), (-2 ** 31, 2 ** 31 - 1, 0),
])
def test_sequences_within_ten_tokens(span_ok, begin, end, ok):
    assert span_ok(begin, end, 10) == ok
