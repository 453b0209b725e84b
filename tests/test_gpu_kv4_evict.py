"""Eviction from the 4-bit cache: which tokens stay is compared for equality, and so is what is moved
(codes and scales are copied); then the norm, the 8-bit product, the cache, the attention and the eviction as a
decoder layer uses them."""
import numpy as np
import pytest
import torch

from gpu_helpers import cuda  # noqa: F401 (the suite's helpers are importable)
from oracle import four_bit
from test_gpu_kv4 import Pool4, check_attention
from test_gpu_kv8 import bf16, cu_of, f64, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def planner():
    from cem_search_transformer_gb300 import binding, synthetic
    p = binding.Planner(synthetic.PRESETS["small"])
    yield p
    p.close()


class Target:
    """Fresh pages for `keep` tokens of each sequence in the pool's own buffers, or in others."""

    def __init__(self, pool, batch, keep, page=None, seed=1):
        from cem_search_transformer_gb300 import binding
        self.page = page or pool.page
        per = -(-keep // self.page)
        rng = np.random.default_rng(seed)
        pages = batch * per + 1
        u8 = lambda n: torch.full((pages, pool.heads, self.page, n), 0xee, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.k, self.v, self.ks, self.vs = u8(pool.dim // 2), u8(pool.dim // 2), u8(pool.dim // 16), u8(pool.dim // 16)
        self.table_np = rng.permutation(pages)[:batch * per].reshape(batch, per)
        self.table = i32(self.table_np)
        self.heads, self.dim, self.pages, self.unit_np = pool.heads, pool.dim, pages, pool.unit_np
        self.cache = binding.KvCache4(self.k, self.v, self.ks, self.vs, self.table, *pool.units)

    held = Pool4.held


def masses(rng, batch, heads, reach, kind):
    m = np.exp(2 * rng.standard_normal((batch, heads, reach))).astype(np.float32)
    if kind == "ties":
        m = np.floor(2 * m).astype(np.float32) / 4
    if kind == "one":
        m[:] = 0.5
    if kind == "odd":
        m *= np.sign(rng.standard_normal(m.shape)).astype(np.float32)
        m[rng.random(m.shape) < 0.1] = np.nan
        m[rng.random(m.shape) < 0.1] = np.inf
        m[rng.random(m.shape) < 0.1] = -0.0
        m[rng.random(m.shape) < 0.1] = 0.0
    return m


@pytest.mark.parametrize("lens,heads,dim,page,to_page,keep,recent,kind", [
    ([1], 1, 64, 16, 16, 1, 0, "plain"),
    ([0, 2, 1], 2, 128, 16, 32, 1, 1, "plain"),
    ([40, 0, 7, 33], 3, 64, 16, 16, 20, 5, "plain"),
    ([517, 300], 4, 128, 64, 64, 129, 0, "ties"),
    ([517, 300], 2, 64, 32, 16, 129, 129, "plain"),             # the latest only
    ([900, 20], 2, 128, 128, 128, 899, 1, "one"),               # all alike
    ([3000, 2049, 700], 2, 64, 16, 128, 700, 33, "odd"),
    ([20000], 1, 128, 64, 64, 5000, 100, "ties"),               # a cluster of eight
    ([20000, 19000], 2, 64, 128, 64, 1, 0, "plain"),            # one token
    ([70] * 200, 2, 64, 16, 16, 33, 4, "plain"),
    ([100000], 1, 64, 128, 128, 3000, 50, "ties"),              # pieces beyond what shared memory holds
    ([100000], 1, 64, 128, 128, 50000, 0, "odd"),
])
def test_matches_oracle(planner, lens, heads, dim, page, to_page, keep, recent, kind):
    rng = np.random.default_rng(keep)
    pool = Pool4(lens, heads, page, dim, seed=2, room=3)
    pool.fill(lens, 3)
    held = [pool.held(s, n) for s, n in enumerate(lens)]
    to = Target(pool, len(lens), keep, to_page)
    reach = pool.table.shape[1] * page
    m = masses(rng, len(lens), heads, reach, kind)
    mass = torch.from_numpy(m).cuda()
    len_out = i32([-5] * len(lens))
    mass_out = torch.full((len(lens), heads, to.table.shape[1] * to_page), 9.0, device="cuda")
    ws = torch.empty(planner.kv4_evict_workspace(pool.cache, keep), dtype=torch.uint8, device="cuda")
    planner.kv4_evict(pool.cache, i32(lens), mass, keep, recent, to.cache, len_out, mass_out, ws)
    planner.sync_check()
    assert len_out.tolist() == [min(n, keep) for n in lens]
    got_mass = mass_out.cpu().numpy()
    for s, n in enumerate(lens):
        got = to.held(s, min(n, keep))
        for h in range(heads):
            at = four_bit.kept(m[s, h, :n], keep, recent)
            for g, w in zip(got, held[s]):
                assert np.array_equal(g[:, h], w[at, h], equal_nan=True), (s, h)
            assert np.array_equal(got_mass[s, h, :len(at)], m[s, h, at], equal_nan=True)
            assert not got_mass[s, h, len(at):].any()
    # tokens behind the kept ones are left as they were
    for s, n in enumerate(lens):
        k = min(n, keep)
        if k % to_page:
            assert torch.all(to.k[int(to.table_np[s, k // to_page]), :, k % to_page:] == 0xee)


def test_same_buffers_and_sequences_that_stay(planner):
    """The target's table names other pages of the same buffers; a sequence within the budget names its own."""
    from cem_search_transformer_gb300 import binding
    lens, page, dim, keep = [100, 20], 16, 64, 32
    pool = Pool4(lens, 2, page, dim, spare=4)
    pool.fill(lens, 5)
    before = [pool.held(s, n) for s, n in enumerate(lens)]
    all_before = [t.clone() for t in (pool.k, pool.v, pool.ks, pool.vs)]
    table = np.stack([pool.spare[:2], pool.table_np[1, :2]])
    cache = binding.KvCache4(pool.k, pool.v, pool.ks, pool.vs, i32(table), *pool.units)
    m = np.random.default_rng(1).random((2, 2, pool.table.shape[1] * page)).astype(np.float32)
    ws = torch.empty(planner.kv4_evict_workspace(pool.cache, keep), dtype=torch.uint8, device="cuda")
    len_out = i32([0, 0])
    planner.kv4_evict(pool.cache, i32(lens), torch.from_numpy(m).cuda(), keep, 8, cache, len_out, None, ws)
    planner.sync_check()
    pool.table_np = table
    for h in range(2):
        at = four_bit.kept(m[0, h, :100], keep, 8)
        for g, w in zip(pool.held(0, 32), before[0]):
            assert np.array_equal(g[:, h], w[at, h])
    others = np.setdiff1d(np.arange(pool.pages), pool.spare[:2])
    for t, b in zip((pool.k, pool.v, pool.ks, pool.vs), all_before):
        assert torch.equal(t[others], b[others])


def test_shared_pages_stay_as_they_are(planner):
    """Three sequences that name the same pages choose for themselves; the pages themselves are not written."""
    from cem_search_transformer_gb300 import binding
    n, heads, page, dim, keep = 150, 2, 32, 128, 40
    pool = Pool4([n], heads, page, dim, seed=2, spare=7)
    pool.fill([n], 3)
    held = pool.held(0, n)
    before = [t.clone() for t in (pool.k, pool.v, pool.ks, pool.vs)]
    shared = binding.KvCache4(pool.k, pool.v, pool.ks, pool.vs, i32(np.repeat(pool.table_np, 3, 0)), *pool.units)
    table = pool.spare[:6].reshape(3, 2)
    to = binding.KvCache4(pool.k, pool.v, pool.ks, pool.vs, i32(table), *pool.units)
    m = masses(np.random.default_rng(3), 3, heads, shared.max_pages * page, "ties")
    ws = torch.empty(planner.kv4_evict_workspace(shared, keep), dtype=torch.uint8, device="cuda")
    len_out = i32([0] * 3)
    planner.kv4_evict(shared, i32([n, n, 90]), torch.from_numpy(m).cuda(), keep, 9, to, len_out, None, ws)
    planner.sync_check()
    pages = pool.table_np[0]
    for t, b in zip((pool.k, pool.v, pool.ks, pool.vs), before):
        assert torch.equal(t[pages], b[pages])
    pool.table_np = table
    for s, length in enumerate((n, n, 90)):
        got = pool.held(s, keep)
        for h in range(heads):
            at = four_bit.kept(m[s, h, :length], keep, 9)
            for g, w in zip(got, held):
                assert np.array_equal(g[:, h], w[at, h])


def test_budgets_beyond_the_targets_room(planner):
    """keep above what the target's table names counts as that; above a sequence's length all stay."""
    lens, heads, page, dim = [300, 40], 2, 16, 64
    pool = Pool4(lens, heads, page, dim, seed=2)
    pool.fill(lens, 3)
    m = masses(np.random.default_rng(8), 2, heads, pool.table.shape[1] * page, "plain")
    for keep, recent in ((48, 48), (1000, 7), (1000, 999)):
        to = Target(pool, 2, 48)
        mass_out, len_out = torch.empty(2, heads, 48, device="cuda"), i32([0, 0])
        ws = torch.empty(planner.kv4_evict_workspace(pool.cache, keep), dtype=torch.uint8, device="cuda")
        planner.kv4_evict(pool.cache, i32(lens), torch.from_numpy(m).cuda(), keep, recent, to.cache, len_out, mass_out, ws)
        planner.sync_check()
        assert len_out.tolist() == [48, 40]
        for s, n in enumerate(lens):
            for h in range(heads):
                at = four_bit.kept(m[s, h, :n], 48, min(recent, 48))
                assert np.array_equal(mass_out[s, h, :len(at)].cpu().numpy(), m[s, h, at]) and not mass_out[s, h, len(at):].any()


def test_captured_and_on_two_streams(planner):
    lens, keep, recent = [5000, 300], 512, 64
    pool = Pool4(lens, 2, 64, 64)
    pool.fill(lens, 5)
    reach = pool.table.shape[1] * 64
    kv_len, mass = i32(lens), torch.zeros(2, 2, reach, device="cuda")
    calls = []
    for i in range(2):
        to = Target(pool, 2, keep, seed=i)
        len_out, mass_out = i32([0, 0]), torch.empty(2, 2, keep, device="cuda")
        ws = torch.empty(planner.kv4_evict_workspace(pool.cache, keep), dtype=torch.uint8, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            planner.kv4_evict(pool.cache, kv_len, mass, keep, recent, to.cache, len_out, mass_out, ws,
                              stream=torch.cuda.current_stream())
        calls.append((graph, side, to, len_out, mass_out, ws))
    for n, seed in (([5000, 300], 1), ([4000, 0], 2), ([513, 300], 3)):
        m = np.random.default_rng(seed).random((2, 2, reach)).astype(np.float32)
        mass.copy_(torch.from_numpy(m))
        kv_len.copy_(i32(n))
        torch.cuda.synchronize()
        for graph, side, *_ in calls:
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for _, _, to, len_out, mass_out, _ in calls:
            assert len_out.tolist() == [min(x, keep) for x in n]
            for s in range(2):
                for h in range(2):
                    at = four_bit.kept(m[s, h, :n[s]], keep, recent)
                    assert np.array_equal(mass_out[s, h, :len(at)].cpu().numpy(), m[s, h, at])
    planner.sync_check()


def test_bad_lengths_and_pages_are_reported(planner):
    from cem_search_transformer_gb300 import binding
    pool = Pool4([64, 64], 1, 16, 64)
    pool.fill([64, 64], 1)
    to = Target(pool, 2, 16)
    mass = torch.rand(2, 1, 64, device="cuda")
    ws = torch.empty(planner.kv4_evict_workspace(pool.cache, 16), dtype=torch.uint8, device="cuda")
    len_out = i32([0, 0])
    call = lambda n: planner.kv4_evict(pool.cache, i32(n), mass, 16, 4, to.cache, len_out, None, ws)  # noqa: E731
    for n, got in (([65, -2], [16, 0]), ([2 ** 31 - 1, 64], [16, 16])):
        call(n)
        with pytest.raises(binding.JepaError, match="outside"):
            planner.sync_check()
        assert len_out.tolist() == got
    good = to.k.clone()
    for t in (pool.table, to.table):
        keep = t.clone()
        t[1] = 10 ** 6
        call([64, 64])
        with pytest.raises(binding.JepaError, match="outside"):
            planner.sync_check()
        assert torch.equal(to.k[to.table_np[0]], good[to.table_np[0]])
        t.copy_(keep)


def test_refusals(planner):
    from cem_search_transformer_gb300 import binding
    pool = Pool4([64], 2, 16, 64)
    to = Target(pool, 1, 32)
    n = planner.kv4_evict_workspace(pool.cache, 32)
    assert n == 4 * 2 * 32
    ws, mass = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.zeros(1, 2, 64, device="cuda")
    kv_len, len_out = i32([64]), i32([0])
    ok = dict(cache=pool.cache, kv_len=kv_len, mass=mass, keep=32, recent=4, to=to.cache, len_out=len_out,
              mass_out=torch.empty(1, 2, 32, device="cuda"), workspace=ws)
    planner.kv4_evict(**ok)
    other = Pool4([64], 2, 16, 64)                           # units of its own
    wide = Pool4([64], 2, 16, 128)
    for change, match in ((dict(recent=33), "bad argument"), (dict(recent=-1), "bad argument"), (dict(keep=0), "bad argument"),
                          (dict(workspace=ws[:n - 4]), "small"), (dict(len_out=kv_len), "bad argument"),
                          (dict(to=other.cache, mass_out=None), "units"), (dict(to=wide.cache, mass_out=None), "differ"), (dict(mass=mass[:, :, :63].contiguous()), "elements"),
                          (dict(mass=None), "required"), (dict(mass_out=mass[:, :1, :16].contiguous()), "elements")):
        with pytest.raises(binding.JepaError, match=match):
            planner.kv4_evict(**{**ok, **change})
    with pytest.raises(binding.JepaError, match="range"):
        planner.kv4_evict_workspace(pool.cache, 0)
    planner.sync_check()


def test_a_decoder_layer_step_by_step(planner):
    """Norm, 8-bit projection, append, attention with weights, and an eviction half way; then on from the
    evicted cache. Every step against what the cache holds."""
    rng = np.random.default_rng(12)
    batch, width, q_heads, heads, dim, page, keep = 3, 256, 4, 2, 64, 16, 40
    n_out = (q_heads + 2 * heads) * dim
    old = [70, 39, 55]
    pool = Pool4(old, heads, page, dim, seed=3, room=8)
    pool.fill(old, 4)
    to = Target(pool, batch, keep + page)
    wq, sq = torch.empty(n_out, width, dtype=torch.uint8, device="cuda"), torch.empty(n_out, device="cuda")
    weight = torch.from_numpy(rng.standard_normal((n_out, width)).astype(np.float32)).cuda() * width ** -0.5
    planner.quantize_rows_fp8(weight, n_out, width, wq, sq)
    gain = torch.rand(width, device="cuda") + 0.5
    rope = planner.rope_table(256, dim)
    x = torch.from_numpy(rng.standard_normal((batch, width)).astype(np.float32)).cuda()
    codes, scales = torch.empty(batch, width, dtype=torch.uint8, device="cuda"), torch.empty(batch, device="cuda")
    proj = torch.empty(batch, n_out, device="cuda")
    ws = torch.empty(planner.attention_kv4_workspace(pool.cache), dtype=torch.uint8, device="cuda")
    now, lens, seen = pool, list(old), list(old)             # cached tokens, and positions
    mass = torch.zeros(batch, heads, pool.table.shape[1] * page, device="cuda")
    for step in range(8):
        if step == 4:
            work = torch.empty(planner.kv4_evict_workspace(pool.cache, keep), dtype=torch.uint8, device="cuda")
            len_out, mass_out = i32([0] * batch), torch.empty(batch, heads, to.table.shape[1] * page, device="cuda")
            planner.kv4_evict(pool.cache, i32(lens), mass, keep, 8, to.cache, len_out, mass_out, work)
            now, lens, mass = to, len_out.tolist(), mass_out
            assert lens == [min(n + 4, keep) for n in old]
        delta = bf16(rng.standard_normal((batch, width)) * 0.5).cuda()
        planner.add_rmsnorm_fp8(x, delta, gain, x, codes, scales)
        planner.linear_fp8(codes, scales, wq, sq, None, batch, n_out, width, 0, proj)
        qkv = proj.to(torch.bfloat16).view(batch, -1, dim)
        q_out = torch.empty(batch, q_heads, dim, dtype=torch.bfloat16, device="cuda")
        # stored behind the cached tokens, rotated for its position: after an eviction these differ
        k_out = torch.empty(batch, heads, dim, dtype=torch.bfloat16, device="cuda")
        planner.rope_append_kv4(qkv[:, :q_heads], qkv[:, q_heads:q_heads + heads], qkv[:, q_heads + heads:], rope, cu_of([1] * batch),
                                i32(lens), now.cache, q_out, k_out=k_out, rope_start=i32(seen) if step >= 4 else None)
        want = four_bit.norm_rotate(f64(qkv[:, q_heads:q_heads + heads]), None, rope.cpu().numpy(), np.array(seen), False)
        assert np.all(np.abs(f64(k_out) - want) <= 2.0 ** -8 * np.abs(want))
        lens, seen = [n + 1 for n in lens], [p + 1 for p in seen]
        before = mass.clone()
        out, lse = torch.empty(batch, 1, q_heads, dim, dtype=torch.bfloat16, device="cuda"), torch.empty(batch, 1, q_heads, device="cuda")
        planner.attention_kv4(q_out.unsqueeze(1), now.cache, i32(lens), out, dim ** -0.5, ws, lse=lse, mass=mass, mass_out=mass)
        planner.sync_check()
        held = [now.held(s, n) for s, n in enumerate(lens)]
        ref = [(four_bit.values(h[0], h[1], pool.unit_np[0][None, :, None]), four_bit.values(h[2], h[3], pool.unit_np[1][None, :, None]))
               for h in held]
        again, _, _ = check_attention(planner, now, ref, lens, 1, q_heads, True, seed=0, q=q_out.unsqueeze(1))
        assert torch.equal(again, out)
        for s, n in enumerate(lens):
            got = f64(mass[s, :, :n] - before[s, :, :n]).sum()
            assert abs(got - q_heads) <= 1e-4 * q_heads          # each row's weights sum to 1
            # the newest token is there with the values of its projection
            k, v = ref[s]
            c, sc = four_bit.quantise(f64(qkv[s, q_heads + heads:]), pool.unit_np[1][:, None])
            assert np.array_equal(v[-1], four_bit.values(c, sc, pool.unit_np[1][:, None]))
