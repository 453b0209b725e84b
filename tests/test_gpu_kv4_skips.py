"""What an append and a read-back leave out because of bad pages, starts or offsets, and nothing else: every byte of
the cache and every row of the outputs."""
import numpy as np
import pytest
import torch

from test_gpu_kv4 import Pool4
from test_gpu_kv8 import bf16, cu_of, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def planner():
    from cem_search_transformer_gb300 import binding, synthetic
    p = binding.Planner(synthetic.PRESETS["small"])
    yield p
    p.close()


N = 20                                                       # tokens of each of four sequences, pages of 16


def change_of(kind):
    """(packed offsets, starts, entry of sequence 1's table (or None), {token: (sequence, place)} that are appended)."""
    cu, start, entry = [0, 20, 40, 60, 80], [0] * 4, None
    fine = {t: (t // N, t % N) for t in range(80) if t // N != 1}
    if kind == "page":                                       # the first page of sequence 1: its second is there
        entry = 0
        fine.update({t: (1, t - 20) for t in range(36, 40)})
    elif kind == "later page":
        entry = 1
        fine.update({t: (1, t - 20) for t in range(20, 36)})
    elif kind == "start":                                    # a negative start is bad as a whole
        start = [0, -3, 0, 0]
    elif kind == "far start":                                # behind what the table names
        start = [0, 10 ** 9, 0, 0]
    elif kind == "end of the table":                         # tokens 12 .. of the table's 32 places
        start = [0, 20, 0, 0]
        fine.update({t: (1, t) for t in range(20, 32)})
    elif kind == "behind":                                   # 1 and on leave the rows
        cu = [0, 20, 81, 90, 100]
        fine = {t: (0, t) for t in range(20)}
    return cu, start, entry, fine


@pytest.mark.parametrize("kind", ["page", "later page", "start", "far start", "end of the table", "behind"])
@pytest.mark.parametrize("dim,heads", [(64, 2), (128, 9)])
def test_only_what_is_bad_is_left_out(planner, kind, dim, heads):
    from cem_search_transformer_gb300 import binding
    cu, start, entry, fine = change_of(kind)
    x = bf16(np.random.default_rng(6).standard_normal((80, heads, dim))).cuda()
    y = bf16(np.random.default_rng(7).standard_normal((80, heads, dim))).cuda()
    good = Pool4([N] * 4, heads, 16, dim, seed=2, room=12)   # tables of two pages
    planner.rope_append_kv4(None, x, y, None, cu_of([N] * 4), i32([0] * 4), good.cache, None)
    planner.sync_check()
    pool = Pool4([N] * 4, heads, 16, dim, seed=2, room=12)
    assert pool.table.shape[1] == 2
    if entry is not None:
        pool.table[1, entry] = pool.pages
    names = ("k", "v", "ks", "vs")
    want = {n: getattr(pool, n).clone() for n in names}
    for t, (s, place) in fine.items():
        page, slot = int(pool.table_np[s, place // 16]), place % 16
        first = t % N                                        # where the good pool has this row
        for n in names:
            from_page = int(good.table_np[t // N, first // 16])
            want[n][page, :, slot] = getattr(good, n)[from_page, :, first % 16]
    q_out, k_out = torch.full_like(x, 5.0), torch.full_like(x, 5.0)
    planner.rope_append_kv4(x, x, y, None, i32(cu), i32(start), pool.cache, q_out, k_out=k_out)
    with pytest.raises(binding.JepaError, match="outside"):
        planner.sync_check()
    planner.sync_check()                                     # reported once
    for n in names:
        assert torch.equal(getattr(pool, n), want[n]), n
    there = torch.zeros(80, dtype=torch.bool, device="cuda")
    there[list(fine)] = True
    assert torch.equal(k_out[there], x[there]) and torch.all(k_out[~there] == 5.0)
    # queries need no pages: left out only where their place is
    q_there = there.clone()
    if "page" in kind:
        q_there[20:40] = True
    assert torch.equal(q_out[q_there], x[q_there]) and torch.all(q_out[~q_there] == 5.0)
    k_read, v_read = torch.full_like(x, 5.0), torch.full_like(x, 5.0)
    planner.kv4_read(pool.cache, i32(cu), i32(start), k_read, v_read)
    with pytest.raises(binding.JepaError, match="outside"):
        planner.sync_check()
    k_want, v_want = torch.empty_like(x), torch.empty_like(x)
    planner.kv4_read(good.cache, cu_of([N] * 4), i32([0] * 4), k_want, v_want)
    planner.sync_check()
    for got, ref in ((k_read, k_want), (v_read, v_want)):
        assert torch.equal(got[there], ref[there]) and torch.all(got[~there] == 5.0)


def test_offsets_out_of_order(planner):
    """A sequence that ends before it begins, and an empty one, write nothing; the first is reported."""
    from cem_search_transformer_gb300 import binding
    cu, start = [0, 20, 70, 60, 60], [0] * 4
    x = bf16(np.random.default_rng(6).standard_normal((80, 2, 64))).cuda()
    pool = Pool4([N] * 4, 2, 16, 64, seed=2, room=12)
    before = pool.k.clone()
    planner.rope_append_kv4(None, x, x, None, i32(cu), i32(start), pool.cache, None)
    with pytest.raises(binding.JepaError, match="outside"):
        planner.sync_check()
    for s in (2, 3):
        assert torch.equal(pool.k[pool.table_np[s]], before[pool.table_np[s]])
    k, v = torch.full_like(x, 5.0), torch.full_like(x, 5.0)
    planner.kv4_read(pool.cache, i32([0, 20, 20, 20, 20]), i32(start), k, v)
    planner.sync_check()
    assert not torch.any(k[:20] == 5.0) and torch.all(k[20:] == 5.0)
