"""The 8-bit paged cache without a GPU: the kernels' index arithmetic (compiled for the host)
over its whole range, the oracle's block quantisation, and the refusals of the entry points."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from cem_search_transformer_gb300 import binding, build_lib, synthetic
from oracle import paged, quant

CSRC = build_lib.CSRC


@pytest.fixture(scope="module")
def index(tmp_path_factory):
    """kv8_index.h behind a C interface, built with the host compiler."""
    d = tmp_path_factory.mktemp("kv8_index")
    src, so = str(d / "index.cpp"), str(d / "index.so")
    with open(src, "w") as f:
        f.write('#include "kv8_index.h"\n'
                'extern "C" int page_at(const int* t, int mp, int np, int lg, long long s, int pos)'
                '{ return jepa::kv8_page_at(t, mp, np, lg, s, pos); }\n'
                'extern "C" int exponent(uint32_t b) { return jepa::kv8_exponent(b); }\n'
                'extern "C" long long share(long long n, int w, int i) { return jepa::kv8_share(n, w, i); }\n'
                'extern "C" int worker_of(long long n, int w, long long u)'
                '{ return jepa::kv8_worker_of(n, w, u); }\n')
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, src, "-o", so],
                   check=True)
    lib = ctypes.CDLL(so)
    lib.page_at.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_longlong,
                            ctypes.c_int]
    lib.exponent.argtypes = [ctypes.c_uint32]
    lib.share.argtypes, lib.share.restype = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int], ctypes.c_longlong
    lib.worker_of.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_longlong]
    return lib


def test_pages_out_of_range_are_never_followed(index):
    table = np.array([[3, 0, 7], [-1, 8, 2]], np.int32)   # a pool of 8 pages: -1 and 8 are bad
    at = lambda s, pos: index.page_at(table.ctypes.data, 3, 8, 4, s, pos)
    assert [at(0, p) for p in (0, 15, 16, 47)] == [3, 3, 0, 7]
    assert [at(1, p) for p in (0, 16, 32)] == [-1, -1, 2]
    assert [at(0, p) for p in (-1, 48, 2 ** 31 - 1, -2 ** 31)] == [-1, -1, -1, -1]


def test_exponents_are_the_least_that_hold_the_block(index):
    values = [0.0, 1e-45, 448 * 2.0 ** -41, 448.0, 448.00003, 449.0, 447.9, 1.75, 1.7500001, 3.5, 2.0 ** 60, np.inf]
    values += [float(np.float32(448 * 2.0 ** e * f)) for e in range(-45, 46) for f in (1 - 2 ** -23, 1, 1 + 2 ** -23)]
    for v in values:
        bits = int(np.array(v, np.float32).view(np.uint32))
        assert index.exponent(bits) == paged.block_exponent(float(np.float32(v))), v


@pytest.mark.parametrize("total,workers", [(1, 1), (7, 3), (456, 456), (457, 456), (100003, 455), (5, 5), (1 << 40, 456)])
def test_shares_cover_the_line_once(index, total, workers):
    edges = [index.share(total, workers, w) for w in range(workers + 1)]
    assert edges[0] == 0 and edges[-1] == total
    sizes = np.diff(edges)
    assert sizes.min() >= 1 and sizes.max() - sizes.min() <= 1
    for w in range(workers):
        assert index.worker_of(total, workers, edges[w]) == w
        assert index.worker_of(total, workers, edges[w + 1] - 1) == w


def test_oracle_block_keeps_earlier_values_and_never_shrinks():
    rng = np.random.default_rng(0)
    held = quant.round_to_e4m3(rng.standard_normal((5, 64)) * 100)
    same, s = paged.append_block(held, 0.5, rng.standard_normal((3, 64)) * 0.01)
    assert s == 0.5 and np.array_equal(same[:5], held)
    grown, s = paged.append_block(held, 0.5, np.full((1, 64), 448 * 4.0))
    assert s == 4.0 and np.all(grown[5] == 448)
    assert np.max(np.abs(grown[:5] * 4.0 - held * 0.5)) <= 4.0 * 2.0 ** -10 + 0.5 * np.abs(held).max() * 2.0 ** -4
    # a value is at most half a step off: 2^-4 relative, 2^-10 of the scale where subnormal
    x = rng.standard_normal((16, 64)) * np.exp2(rng.uniform(-12, 3, (16, 1)))
    codes, s = paged.append_block(np.zeros((0, 64)), 1.0, x)
    assert np.all(np.abs(codes * s - x) <= np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10))


# ---- refusals: nothing invalid reaches the library ----

class _Unreachable:
    def __getattr__(self, name):
        def call(*args):
            raise AssertionError(f"{name} was called although an argument was invalid")
        return call


class _NoLibrary:
    lib = _Unreachable()
    h = None
    device = 0
    _dims = binding.Planner._dims

    def _check(self, status, what):
        raise AssertionError(f"{what} returned {status} although an argument was invalid")


def _cache_tensors(pages=4, heads=2, page=16, dim=64, batch=2, most=3):
    return (torch.zeros(pages, heads, page, dim, dtype=torch.uint8), torch.zeros(pages, heads, page, dim, dtype=torch.uint8),
            torch.zeros(pages, heads), torch.zeros(pages, heads), torch.zeros(batch, most, dtype=torch.int32))


@pytest.mark.parametrize("change,match", [
    (dict(), "CUDA"),                                                       # host tensors
    ({1: torch.zeros(4, 2, 16, 128, dtype=torch.uint8)}, "shape"),
    ({2: torch.zeros(4, 3)}, "k_scale"),
    ({0: torch.zeros(4, 2, 24, 64, dtype=torch.uint8), 1: torch.zeros(4, 2, 24, 64, dtype=torch.uint8)}, "page_size"),
    ({0: torch.zeros(4, 2, 16, 80, dtype=torch.uint8), 1: torch.zeros(4, 2, 16, 80, dtype=torch.uint8)}, "head_dim"),
    ({4: torch.zeros(3, dtype=torch.int32)}, "page_table"),
])
def test_cache_handle_refuses(change, match):
    t = list(_cache_tensors())
    for i, x in change.items():
        t[i] = x
    with pytest.raises(binding.JepaError, match=match):
        binding.KvCache8(*t)


def test_token_rows_refuse():
    with pytest.raises(binding.JepaError, match="tokens, heads, head_dim"):
        binding._rows(torch.zeros(4, 8), "q")
    with pytest.raises(binding.JepaError, match="dtype"):
        binding._rows(torch.zeros(4, 2, 64), "q")
    with pytest.raises(binding.JepaError, match="contiguous"):
        binding._rows(torch.zeros(2, 4, 64, dtype=torch.bfloat16).transpose(0, 1), "q")
    with pytest.raises(binding.JepaError, match="CUDA"):
        binding._rows(torch.zeros(4, 2, 64, dtype=torch.bfloat16), "q")


def test_packed_attention_refuses_before_the_call():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(binding.JepaError, match="CUDA"):
        binding.Planner.attention_packed(_NoLibrary(), q, q, q, cu, cu, q, 0.125)
    with pytest.raises(binding.JepaError, match="q must be"):
        cache = type("C", (), dict(batch=2, head_dim=64, check=lambda self, d: None))()
        binding.Planner.attention_kv8(_NoLibrary(), q, cache, cu, q, 0.125, None)


def test_null_contexts_are_refused_by_the_library():
    build_lib.build()
    lib = binding.load()
    c = binding.Kv8Struct()
    n = ctypes.c_size_t()
    assert lib.jepa_rope_table(None, 1, 16, 1e4, 1.0, None, None) == 1
    assert lib.jepa_rope_append_kv8(None, ctypes.byref(c), *([None, 0] * 3), 1, 1, None, None, 0.0, None, 0, 0, 0,
                                    None, None, None, None, None) == 1
    assert lib.jepa_kv8_read(None, ctypes.byref(c), None, None, 1, None, None, None) == 1
    assert lib.jepa_attention_kv8_workspace(None, ctypes.byref(c), ctypes.byref(n)) == 1
    assert lib.jepa_attention_kv8(None, ctypes.byref(c), None, 1, 1, None, 1.0, 1, None, None, None, 0, None) == 1
    assert lib.jepa_attention_packed(None, None, 0, None, 0, None, 0, 1, 1, 1, 1, 1, 64, None, None, 1.0, 1, None,
                                     None, None) == 1


def test_struct_matches_the_header():
    assert ctypes.sizeof(binding.Kv8Struct) == 5 * 8 + 6 * 4
    text = open(os.path.join(build_lib.INCLUDE, "jepa_cem.h")).read()
    assert "int32_t num_pages, page_size, kv_heads, head_dim, batch, max_pages;" in text
    assert synthetic.SMALL.head_dim == 64
