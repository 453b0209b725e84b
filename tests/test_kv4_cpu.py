"""The 4-bit cache, its eviction and the norm ahead of 8-bit products without a GPU: the oracle, and
what the entry points refuse."""
import ctypes

import numpy as np
import pytest
import torch

from cem_search_transformer_gb300 import binding, build_lib
from oracle import four_bit, quant
from test_kv8_cpu import _NoLibrary


def test_e2m1_rounding_against_all_neighbours():
    v = np.concatenate([-four_bit.E2M1[:0:-1], four_bit.E2M1])
    assert np.array_equal(four_bit.round_to_e2m1(v), v)
    for i, (a, b) in enumerate(zip(four_bit.E2M1[:-1], four_bit.E2M1[1:])):
        mid = (a + b) / 2
        even = a if i % 2 == 0 else b                      # the mantissa bit is the code's lowest
        for x, want in ((mid, even), (np.nextafter(mid, 0), a), (np.nextafter(mid, 9), b)):
            assert four_bit.round_to_e2m1(x) == want and four_bit.round_to_e2m1(-x) == -want
    assert four_bit.round_to_e2m1(1e9) == 6 and four_bit.round_to_e2m1(-7.0) == -6


def test_block_quantisation():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((50, 3, 64)) * np.exp(3 * rng.standard_normal((50, 3, 1)))).astype(np.float32)
    unit = np.array([0.25, 1.0, 8.0])[None, :, None]
    c, s = four_bit.quantise(x, unit)
    back = four_bit.values(c, s, unit)
    step = np.repeat(s * unit, 16, -1)
    # half a step: 1/4, 1/2 or 1 scale; a scale rounded down leaves up to 6 (1 + 2^-4) of itself
    big = np.abs(x) / step
    half = np.where(big < 2, 0.25, np.where(big < 4, 0.5, 1.0))
    sat = big > 6 * (1 + 2.0 ** -4 + 2.0 ** -20)          # only where the scale is at its end, or subnormal (3 bits and fewer)
    ends = np.repeat((s == quant.E4M3_MAX) | (s < 2.0 ** -6), 16, -1)
    assert sat.any() and np.all(ends[sat]) and np.all(np.abs(back[sat]) == 6 * step[sat])
    assert np.all(np.abs(back - x)[~sat] <= (step * half * (1 + 2.0 ** -20))[~sat])
    assert np.all(s >= four_bit.SCALE_MIN) and np.all(s <= quant.E4M3_MAX)
    x[0, 0, 3], x[1, 1, 20] = np.nan, np.inf
    c, s = four_bit.quantise(x, unit)
    assert np.isnan(s[0, 0, 0]) and np.isnan(s[1, 1, 1]) and np.isnan(s).sum() == 2
    c, s = four_bit.quantise(np.zeros((1, 1, 16)), 1.0)
    assert not c.any() and s[0, 0, 0] == four_bit.SCALE_MIN


def test_unpacking():
    data = np.array([[0x21, 0xf7]], np.uint8)
    assert np.array_equal(four_bit.unpack(data), [[0.5, 1.0, 6.0, -6.0]])


def test_kept_tokens():
    m = [3.0, 1.0, 3.0, np.nan, 0.0, 2.0, 9.0, 0.5]
    assert list(four_bit.kept(m, 8, 2)) == list(range(8))
    assert list(four_bit.kept(m, 4, 1)) == [0, 2, 6, 7]
    assert list(four_bit.kept(m, 2, 2)) == [6, 7]
    assert list(four_bit.kept(m, 7, 0)) == [0, 1, 2, 4, 5, 6, 7]       # NaN goes first
    assert list(four_bit.kept([1.0] * 5, 3, 1)) == [0, 1, 4]
    assert list(four_bit.kept([], 3, 1)) == []


def test_sum_and_norm():
    rng = np.random.default_rng(1)
    x, d, w = rng.standard_normal((3, 32)), rng.standard_normal((3, 32)), rng.standard_normal(32)
    s, y = four_bit.add_rmsnorm(x, d, w, 1e-6)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x + d), (32,), torch.from_numpy(w), 1e-6)
    assert np.allclose(y, want.numpy(), rtol=1e-12)


def tensors(pages=4, heads=2, page=16, dim=64, batch=2, most=3):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    return [u8(pages, heads, page, dim // 2), u8(pages, heads, page, dim // 2), u8(pages, heads, page, dim // 16),
            u8(pages, heads, page, dim // 16), torch.zeros(batch, most, dtype=torch.int32)]


@pytest.mark.parametrize("change,match", [
    (dict(), "CUDA"),                                                       # host tensors
    ({1: torch.zeros(4, 2, 16, 64, dtype=torch.uint8)}, "shape"),
    ({2: torch.zeros(4, 2, 16, 2, dtype=torch.uint8)}, "k_scale"),
    ({3: torch.zeros(4, 2)}, "v_scale"),
    ({0: torch.zeros(4, 2, 24, 32, dtype=torch.uint8)}, "page_size"),
    ({0: torch.zeros(4, 2, 16, 40, dtype=torch.uint8)}, "head_dim"),
    ({4: torch.zeros(3, dtype=torch.int32)}, "page_table"),
    ({5: torch.ones(3)}, "k_unit"),
    ({6: 4096}, "v_unit"),
    ({0: None}, "tensor"),
])
def test_cache_handle_refuses(change, match):
    t = dict(enumerate(tensors() + [None, None]))
    t.update(change)
    with pytest.raises(binding.JepaError, match=match):
        binding.KvCache4(*(t[i] for i in range(7)))


class _Cache:
    batch, kv_heads, head_dim, max_pages, page_size = 2, 2, 64, 4, 16
    ref = None

    def check(self, device):
        pass


def test_calls_refuse_before_the_library(monkeypatch):
    q = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: binding.Planner.attention_kv4(_NoLibrary(), q[0], _Cache(), n, q, 0.1, q),
                 lambda: binding.Planner.attention_kv4(_NoLibrary(), q, _Cache(), n, q, 0.1, q),
                 lambda: binding.Planner.kv4_evict(_NoLibrary(), _Cache(), None, q, 4, 1, _Cache(), n, None, q),
                 lambda: binding.Planner.kv4_read(_NoLibrary(), _Cache(), n, n, 5, q),
                 lambda: binding.Planner.add_rmsnorm_fp8(_NoLibrary(), q, None, q, q, None, None)):
        with pytest.raises(binding.JepaError):
            call()
    monkeypatch.setattr(binding, "_dev", lambda t, *a: 16)
    with pytest.raises(binding.JepaError, match="workspace.*tensor"):
        binding.Planner.attention_kv4(_NoLibrary(), q, _Cache(), n, q, 0.125, 4096)
    with pytest.raises(binding.JepaError, match="workspace.*tensor"):
        binding.Planner.kv4_evict(_NoLibrary(), _Cache(), n, q, 4, 1, _Cache(), n, None, None)


def test_caches_of_the_other_width_are_refused():
    eight, four = binding.KvCache8.__new__(binding.KvCache8), binding.KvCache4.__new__(binding.KvCache4)
    p, t = binding.Planner, torch.zeros(1)
    for call, match in ((lambda: p.rope_append_kv4(_NoLibrary(), None, t, t, None, t, t, eight, None), "KvCache8"),
                        (lambda: p.rope_append_kv8(_NoLibrary(), None, t, t, None, t, t, four, None), "KvCache4"),
                        (lambda: p.kv4_read(_NoLibrary(), eight, t, t, t, t), "KvCache8"),
                        (lambda: p.kv8_read(_NoLibrary(), four, t, t, t, t), "KvCache4"),
                        (lambda: p.attention_kv4(_NoLibrary(), t, eight, t, t, 0.1, t), "KvCache8"),
                        (lambda: p.kv4_evict(_NoLibrary(), four, t, t, 1, 0, eight, t, t, t), "KvCache8")):
        with pytest.raises(binding.JepaError, match=match):
            call()


def test_rows_refuse():
    x = torch.zeros(4, 32)
    binding._sized(x, "x")
    for t, match in ((x[0], "rows, cols"), (x.half(), "dtype"), (x.t(), "contiguous"), (x, "is on"), (7, "rows, cols")):
        with pytest.raises(binding.JepaError, match=match):
            binding._matrix(t, "x", 0)


def test_null_contexts_are_refused_by_the_library():
    build_lib.build()
    lib = binding.load()
    c, n = binding.Kv4Struct(), ctypes.c_size_t()
    r = ctypes.byref(c)
    assert lib.jepa_rope_append_kv4(None, r, *([None, 0] * 3), 1, 1, None, None, 0.0, None, 0, 0, 0,
                                    None, None, None, None, None, None) == 1
    assert lib.jepa_kv4_read(None, r, None, None, 1, None, None, None) == 1
    assert lib.jepa_attention_kv4_workspace(None, r, ctypes.byref(n)) == 1
    assert lib.jepa_attention_kv4(None, r, None, 1, 1, None, 1.0, 1, None, None, None, None, 1.0, None, 0, None) == 1
    assert lib.jepa_kv4_evict_workspace(None, r, 1, ctypes.byref(n)) == 1
    assert lib.jepa_kv4_evict(None, r, None, None, 1, 0, r, None, None, None, 0, None) == 1
    assert lib.jepa_add_rmsnorm_fp8(None, None, 0, 0, None, 0, 0, None, 0.0, 1, 16, None, 0, None, None, None, None) == 1


def test_struct_matches_the_header():
    assert ctypes.sizeof(binding.Kv4Struct) == 7 * 8 + 6 * 4
