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


def with_nonfinite(planner, nq, nk, q_heads, kv_heads, dim, frame, seed, count):
    """Random infinities and NaN in V: a query's columns are the sum of those it sees, and the others are
    to the bit what they are with zeros in their places."""
    rng = np.random.default_rng(seed)
    q, k, v = (bf16(rng.standard_normal((n, h, dim))).cuda() for n, h in ((sum(nq), q_heads), (sum(nk), kv_heads), (sum(nk), kv_heads)))
    odd = torch.zeros(v.shape, dtype=torch.float32)
    for value in (np.inf, -np.inf, np.nan):
        at = tuple(rng.integers(0, n, count) for n in v.shape)
        odd[at] = float(value)
    odd = odd.cuda()
    zeros, bad = torch.where(odd == 0, v, 0.0), torch.where(odd == 0, v, odd.to(torch.bfloat16))
    clean, out = torch.empty_like(q), torch.empty_like(q)
    for values, to in ((zeros, clean), (bad, out)):
        planner.attention_packed(q, k, values, cu_of(nq), cu_of(nk), to, 0.05, frame=frame)
        planner.sync_check()
    want, group, a, b = clean.float(), q_heads // kv_heads, 0, 0
    hit = 0
    for n, m in zip(nq, nk):
        lim = torch.from_numpy(paged.limits(n, m, frame)).cuda()
        sees = torch.arange(m, device="cuda")[None, :] < lim[:, None]
        x = odd[b:b + m]
        up, down, nan = ((sees.float() @ kind.float().flatten(1)).view(n, kv_heads, dim) > 0
                         for kind in (x == np.inf, x == -np.inf, torch.isnan(x)))
        total = torch.zeros(up.shape, device="cuda")
        total[up], total[down] = float("inf"), -float("inf")
        total[nan | (up & down)] = float("nan")
        total = total.repeat_interleave(group, 1)
        hit += int((total != 0).sum())
        want[a:a + n] = torch.where(total != 0, total, want[a:a + n])
        a, b = a + n, b + m
    assert hit > 0
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out.float().nan_to_num(nan=7.0), want.nan_to_num(nan=7.0))


@pytest.mark.parametrize("nq,nk,q_heads,kv_heads,dim,frame,count", [
    ([300], [300], 2, 2, 64, 1, 6),
    ([300, 150], [300, 420], 4, 2, 128, 1, 30),
    ([700], [700], 1, 1, 64, 50, 5),                       # many limits in a tile
    ([700], [900], 3, 1, 128, 258, 40),
    ([900], [700], 2, 1, 64, 1000, 3),                     # rows that see nothing beside rows that see all
    ([6, 3, 1], [500, 400, 70], 8, 8, 64, 1, 20),
    ([400], [400], 2, 1, 128, 1, 4000),
])
def test_values_that_are_not_finite_add_up(planner, nq, nk, q_heads, kv_heads, dim, frame, count):
    with_nonfinite(planner, nq, nk, q_heads, kv_heads, dim, frame, seed=sum(nq) + dim, count=count)


@pytest.mark.parametrize("dim", [64, 128])
def test_values_that_are_not_finite_add_up_in_pairs_of_heads(planner, dim):
    """Many short sequences: the last rows of two heads share an item."""
    rng = np.random.default_rng(dim)
    nq = [int(n) for n in rng.integers(0, 200, 90)]
    nk = [n + int(p) for n, p in zip(nq, rng.integers(0, 300, 90))]
    with_nonfinite(planner, nq, nk, 9, 9, dim, 1, seed=dim, count=60)


def test_infinities_a_million_keys_apart(planner):
    """The first 64 queries see nothing, the other rows of their item all keys: a read-out that looks at
    1.3 million keys again, one row's 32 columns at a time 2.3 s, more than a wait's limit."""
    nk, dim = 1_300_000, 128
    nq = nk + 64
    gen = torch.Generator(device="cuda").manual_seed(0)
    q, k, v = (torch.randn(n, 1, dim, device="cuda", generator=gen).to(torch.bfloat16) for n in (nq, nk, nk))
    outs = []
    for change in (False, True):
        if change:
            v[0, 0, 5] = v[nk - 1, 0, 5] = float("inf")
            v[nk // 2, 0, 100] = float("nan")
        out = torch.full_like(q, 9.0)
        planner.attention_packed(q, k, v, cu_of([nq]), cu_of([nk]), out, 0.01, frame=1 << 30)
        planner.sync_check()
        outs.append(out)
    clean, out = outs
    assert torch.all(out[:64] == 0) and torch.all(out[64:, 0, 5] == float("inf")) and torch.all(torch.isnan(out[64:, 0, 100]))
    rest = [c for c in range(dim) if c not in (5, 100)]
    assert torch.equal(out[..., rest], clean[..., rest])
