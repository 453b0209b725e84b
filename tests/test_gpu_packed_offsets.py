"""Packed offsets that name tokens outside their buffers, on every path that reads them: the sequence
they belong to is skipped, the others come out as without it, and the next check reports it."""
import numpy as np
import pytest
import torch

from test_gpu_kv8 import Pool, bf16, i32

pytestmark = pytest.mark.gpu

N = 200                # packed tokens
FAR = 40               # sequences of the cases whose last one is bad


@pytest.fixture(scope="module")
def planner():
    from cem_search_transformer_gb300 import binding, synthetic
    p = binding.Planner(synthetic.PRESETS["small"])
    yield p
    p.close()


# offsets, and those of the same call without the bad sequence
CASES = {
    "last bound behind the rows": ([0, 30, N + 1], [0, 30, 30]),
    "first bound ahead of the rows": ([-2, 30, N], [30, 30, N]),
    "far ahead of the rows": ([-2 ** 31, 30, N], [30, 30, N]),
    "descending": ([0, 130, 20], [0, 130, 130]),
    "nothing but bad": ([-7, N + 9], [0, 0]),
    "last of many behind the rows": ([0] + [N] * (FAR - 1) + [N + 5], [0] + [N] * FAR),
    "last of many descending": ([0] + [N] * (FAR - 1) + [N - 1], [0] + [N] * FAR),
}


def padded(cu, pad):
    """`pad` empty sequences ahead of the last one's end: the append then takes its short path."""
    return cu[:-1] + [cu[-2]] * pad + cu[-1:]


def bits(t):
    return t.view(torch.int32) if t.dtype == torch.float32 else t


@pytest.mark.parametrize("short", [True, False])
@pytest.mark.parametrize("case", list(CASES))
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 128)])
def test_append_skips_and_reports(planner, case, short, dim, page):
    from cem_search_transformer_gb300 import binding
    heads, got = 2, []
    x = bf16(np.random.default_rng(4).standard_normal((N, 3 * heads, dim))).cuda()
    rope = planner.rope_table(2 * N, dim)
    for at, cu in enumerate(CASES[case]):
        cu = padded(cu, N if short else 0)
        batch = len(cu) - 1
        assert (N <= 4 * batch) == short
        pool = Pool([N + 20] * 2, heads, page, dim, seed=1)
        table = np.full((batch, pool.table_np.shape[1]), -1)
        table[0], table[batch - 1] = pool.table_np
        cache = binding.KvCache8(pool.k, pool.v, pool.ks, pool.vs, i32(table))
        q_out = torch.full((N, heads, dim), 9.0, dtype=torch.bfloat16, device="cuda")
        k_out = q_out.clone()
        planner.rope_append_kv8(x[:, :heads], x[:, heads:2 * heads], x[:, 2 * heads:], rope, i32(cu),
                                i32([3] * batch), cache, q_out, k_out=k_out)
        if at == 0:
            with pytest.raises(binding.JepaError, match="outside its buffer"):
                planner.sync_check()
        planner.sync_check()
        got.append([q_out, k_out, pool.k, pool.v, pool.ks, pool.vs])
    for a, b in zip(*got):
        assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("case", list(CASES))
def test_read_skips_and_reports(planner, case):
    from cem_search_transformer_gb300 import binding
    heads, dim, page, got = 2, 64, 32, []
    for at, cu in enumerate(CASES[case]):
        batch = len(cu) - 1
        pool = Pool([N + 20] * 2, heads, page, dim, seed=1)
        pool.fill([N + 20] * 2, 3)
        table = np.full((batch, pool.table_np.shape[1]), -1)
        table[0], table[batch - 1] = pool.table_np
        cache = binding.KvCache8(pool.k, pool.v, pool.ks, pool.vs, i32(table))
        k = torch.full((N, heads, dim), 9.0, dtype=torch.bfloat16, device="cuda")
        v = k.clone()
        planner.kv8_read(cache, i32(cu), i32([3] * batch), k, v)
        if at == 0:
            with pytest.raises(binding.JepaError, match="outside its buffer"):
                planner.sync_check()
        planner.sync_check()
        got.append([k, v])
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("side", ["q", "k"])
@pytest.mark.parametrize("end", [5, -3])
def test_attention_of_one_query_reports_a_bad_offset_far_behind_it(planner, side, end):
    """As many places as there are items: no search goes past the last item's sequence by itself."""
    from cem_search_transformer_gb300 import binding
    x = [bf16(np.random.default_rng(i).standard_normal((1, 2, 64))).cuda() for i in range(3)]
    good = [0] + [1] * 70
    out = [torch.full_like(x[0], 9.0) for _ in range(2)]
    planner.attention_packed(*x, i32(good), i32(good), out[0], 0.125)
    planner.sync_check()
    cu = dict(q=i32(good), k=i32(good))
    cu[side] = i32(good[:-1] + [end])
    planner.attention_packed(*x, cu["q"], cu["k"], out[1], 0.125)
    with pytest.raises(binding.JepaError, match="outside its buffer"):
        planner.sync_check()
    planner.sync_check()
    assert torch.equal(*out)


@pytest.mark.parametrize("end", [2, 0])
def test_the_last_of_65535_sequences(planner, end):
    """As many sequences as a call may have and one token: every pair of offsets is looked at."""
    from cem_search_transformer_gb300 import binding
    batch, heads, dim, page = 65535, 1, 64, 16
    pool = Pool([16], heads, page, dim, seed=1)
    table = torch.full((batch, 1), -1, dtype=torch.int32, device="cuda")
    table[0] = int(pool.table_np[0, 0])
    cache = binding.KvCache8(pool.k, pool.v, pool.ks, pool.vs, table)
    x = bf16(np.random.default_rng(1).standard_normal((1, heads, dim))).cuda()
    start, k, v = torch.zeros(batch, dtype=torch.int32, device="cuda"), torch.zeros_like(x), torch.zeros_like(x)
    for last in (1, end):
        cu = torch.ones(batch + 1, dtype=torch.int32, device="cuda")
        cu[0], cu[batch] = 0, last
        for call in (lambda: planner.rope_append_kv8(None, x, x, None, cu, start, cache, None),
                     lambda: planner.kv8_read(cache, cu, start, k, v)):
            call()
            if last != 1:
                with pytest.raises(binding.JepaError, match="outside its buffer"):
                    planner.sync_check()
            planner.sync_check()
    assert torch.equal(k, v) and torch.max(torch.abs(k.float() - x.float())) <= 2.0 ** -4 * torch.max(torch.abs(x.float()))
