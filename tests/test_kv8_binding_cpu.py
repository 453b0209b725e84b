"""Arguments of the cache's and the packed attention's calls that are no tensors of the right kind are refused
with the binding's own error, before anything is looked up in them."""
import pytest
import torch

from cem_search_transformer_gb300 import binding
from test_kv8_cpu import _cache_tensors, _NoLibrary


class _Cache:
    batch, kv_heads, head_dim = 2, 2, 64
    ref = None

    def check(self, device):
        pass


@pytest.mark.parametrize("at", range(5))
@pytest.mark.parametrize("bad", [None, 4096, "k"])
def test_cache_of_no_tensors(at, bad):
    t = list(_cache_tensors())
    t[at] = bad
    with pytest.raises(binding.JepaError, match="tensor"):
        binding.KvCache8(*t)


@pytest.mark.parametrize("bad", [None, 4096, [0, 4]])
def test_offsets_workspaces_and_outputs_that_give_a_size(bad, monkeypatch):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    monkeypatch.setattr(binding, "_rows", lambda t, name, device=None: (16, 128, 4, 2, 64))
    monkeypatch.setattr(binding, "_dev", lambda t, *a: 16)
    cu = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(binding.JepaError, match="cu_q.*tensor"):
        binding.Planner.attention_packed(_NoLibrary(), x, x, x, bad, cu, x, 0.125)
    with pytest.raises(binding.JepaError, match="k_out.*tensor"):
        binding.Planner.kv8_read(_NoLibrary(), _Cache(), cu, cu, bad, x)
    q = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(binding.JepaError, match="workspace.*tensor"):
        binding.Planner.attention_kv8(_NoLibrary(), q, _Cache(), cu, q, 0.125, bad)


@pytest.mark.parametrize("table", [torch.zeros(64), torch.zeros(4, 4, 4), 4096, "table"])
def test_rotary_tables_of_no_two_dimensions(table, monkeypatch):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    monkeypatch.setattr(binding, "_rows", lambda t, name, device=None: (16, 128, 4, 2, 64))
    with pytest.raises(binding.JepaError, match="rope_table"):
        binding.Planner.rope_append_kv8(_NoLibrary(), None, x, x, table, x, x, _Cache(), None)
