"""Attention of packed prompts at the far ends of its range."""
import numpy as np
import pytest
import torch

from test_gpu_attention_packed import BF16, bf16, cu_of, f64, paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def planner():
    from cem_search_transformer_gb300 import binding, synthetic
    p = binding.Planner(synthetic.PRESETS["small"])
    yield p
    p.close()


def test_one_query_over_keys_past_4_gib(planner):
    """One item that lasts half a second, while an idle query tile and the cleaning warp wait for its
    end. All scores are 0 but those of four keys, whose weights are e^60 times the others': against
    those four alone the result is off by n e^-60 < 2^-60 besides the weights' and the output's rounding."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB")
    n, dim = 40_000_003, 64
    at = [5, 20_000_001, 34_000_000, n - 1]                # 34 000 000 rows of 128 bytes are past 4 GiB
    q = torch.zeros(1, 1, dim, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 0] = 1
    k = torch.zeros(n, 1, dim, dtype=torch.bfloat16, device="cuda")
    v = torch.full((n, 1, dim), 3.0, dtype=torch.bfloat16, device="cuda")
    scores = torch.tensor([60.0, 61.0, 60.5, 62.0])
    rng = np.random.default_rng(0)
    few = bf16(rng.standard_normal((4, dim))).cuda()
    for i, key in enumerate(at):
        k[key, 0, 0] = scores[i]
        v[key, 0] = few[i]
    out, lse = torch.zeros_like(q), torch.zeros(1, 1, device="cuda")
    planner.attention_packed(q, k, v, cu_of([1]), cu_of([n]), out, 1.0, lse=lse)
    planner.sync_check()
    p = np.exp(scores.numpy().astype(np.float64) - 62)
    total = p.sum()
    want, mag = (p @ f64(few)) / total, (p @ np.abs(f64(few))) / total
    # weights: half a bf16 step each, and the exponential's 2^-21
    assert np.all(np.abs(f64(out)[0, 0] - want) <= BF16 * np.abs(want) + (1 + BF16) * 2 * mag * (BF16 + 2.0 ** -20))
    assert abs(float(lse) - (62 + np.log(total))) <= 62 * 2.0 ** -22 + 2.0 ** -20
