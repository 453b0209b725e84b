"""Sizes beyond 32 bits are refused by the binding: the library takes ints, and ctypes would pass their lower bits on."""
import pytest
import torch

from cem_search_transformer_gb300 import binding
from test_kv4_cpu import _Cache
from test_kv8_cpu import _NoLibrary


@pytest.mark.parametrize("keep,recent,name", [(2 ** 32 + 5, 1, "keep"), (2 ** 31, 1, "keep"), (8, 2 ** 32, "recent"),
                                              (8, 2 ** 32 + 3, "recent"), (-2 ** 32 + 4, 0, "keep")])
def test_budgets_of_an_eviction(monkeypatch, keep, recent, name):
    monkeypatch.setattr(binding, "_dev", lambda t, *a: 16)
    t = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(binding.JepaError, match=name + " out of range"):
        binding.Planner.kv4_evict(_NoLibrary(), _Cache(), t, t, keep, recent, _Cache(), t, None, t)
    if name == "keep":
        with pytest.raises(binding.JepaError, match="keep out of range"):
            binding.Planner.kv4_evict_workspace(_NoLibrary(), _Cache(), keep)


def test_rows_of_the_norm(monkeypatch):
    x = torch.empty(2 ** 32 + 1, 16, dtype=torch.bfloat16, device="meta")
    monkeypatch.setattr(binding, "_matrix", lambda t, *a: (16, 1, 16))
    with pytest.raises(binding.JepaError, match="rows out of range"):
        binding.Planner.add_rmsnorm_fp8(_NoLibrary(), x, None, x, x, None, None)
