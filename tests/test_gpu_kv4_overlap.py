"""Outputs of the 4-bit attention over its queries: refused where the weights, which come later, would read them."""
import numpy as np
import pytest
import torch

from test_gpu_kv4 import Pool4
from test_gpu_kv8 import bf16, i32

pytestmark = pytest.mark.gpu


def test_out_over_the_queries():
    from cem_search_transformer_gb300 import binding, synthetic
    planner = binding.Planner(synthetic.PRESETS["small"])
    lens = [300, 20]
    pool = Pool4(lens, 2, 32, 64)
    pool.fill(lens, 4)
    buf = bf16(np.random.default_rng(1).standard_normal((3, 2, 1, 4, 64))).cuda()
    q, out = buf[0], torch.empty_like(buf[0])
    lse, mass = torch.empty(2, 1, 4, device="cuda"), torch.zeros(2, 2, pool.table.shape[1] * 32, device="cuda")
    ws = torch.empty(planner.attention_kv4_workspace(pool.cache), dtype=torch.uint8, device="cuda")

    def call(out, **kw):
        planner.attention_kv4(q, pool.cache, i32(lens), out, 0.125, ws, **kw)
    flat = buf.view(-1)
    before = buf.clone()
    for over in (q, flat[q.numel() - 8:2 * q.numel() - 8].view_as(q)):
        with pytest.raises(binding.JepaError, match="overlap"):
            call(over, lse=lse, mass_out=mass)
    planner.sync_check()
    assert torch.equal(buf, before) and not mass.any()
    call(buf[1], lse=lse, mass_out=mass)                              # beside it is fine
    call(out)
    call(q)                                                          # and over it without weights
    planner.sync_check()
    assert torch.equal(buf[1], out) and torch.equal(q, out)
    assert np.allclose(mass.sum(-1).cpu().numpy(), 2, atol=1e-4)       # two heads a group, each row's weights sum to 1
    planner.close()
