"""Calls that follow one another without a gap: each may begin while the one before it ends, and reads what that one
wrote. Captured in one graph and replayed, against the same calls with a synchronisation behind each, bit for bit."""
import numpy as np
import pytest
import torch

from test_gpu_kv4 import Pool4
from test_gpu_kv4_evict import Target
from test_gpu_kv8 import bf16, cu_of, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def planner():
    from cem_search_transformer_gb300 import binding, synthetic
    p = binding.Planner(synthetic.PRESETS["small"])
    yield p
    p.close()


@pytest.mark.parametrize("dim,lens", [(64, [300, 45, 700]), (128, [5000, 130, 1031]), (64, [30000])])
def test_steps_and_evictions_back_to_back(planner, dim, lens):
    """Per round: norm in place, append behind the cached tokens, attention that adds up the weights, eviction by them,
    and on from the evicted cache: lengths, weights and places go from call to call on the device."""
    heads, q_heads, page, keep, recent, rounds = 2, 8, 16, 40, 7, 3
    batch, width = len(lens), (q_heads + 2 * heads) * dim
    rng = np.random.default_rng(dim)
    rope = planner.rope_table(64, dim)
    gain = torch.rand(width, device="cuda") + 0.5
    pools = [Pool4([n + 1 for n in lens], heads, page, dim, seed=4) for _ in range(2)]
    for p in pools:
        p.fill(lens, 9)
    rows = bf16(rng.standard_normal((batch, width))).cuda()
    deltas = [bf16(rng.standard_normal((batch, width))).cuda() for _ in range(rounds)]

    def buffers(pool):
        b = dict(x=rows.clone(), y=torch.empty_like(rows), q=torch.empty(batch, q_heads, dim, dtype=torch.bfloat16, device="cuda"),
                 out=[], lse=[], mass=[torch.zeros(batch, heads, pool.table.shape[1] * page, device="cuda")], lens=[i32(lens)],
                 caches=[pool], now=[], len=torch.empty(batch, dtype=torch.int32, device="cuda"))
        for i in range(rounds):
            b["out"].append(torch.empty(batch, 1, q_heads, dim, dtype=torch.bfloat16, device="cuda"))
            b["lse"].append(torch.empty(batch, 1, q_heads, device="cuda"))
            to = Target(pool, batch, keep + 1, seed=i)
            b["caches"].append(to)
            b["mass"].append(torch.empty(batch, heads, to.table.shape[1] * page, device="cuda"))
            b["lens"].append(torch.empty(batch, dtype=torch.int32, device="cuda"))
        b["ws"] = torch.empty(planner.attention_kv4_workspace(pool.cache), dtype=torch.uint8, device="cuda")
        b["work"] = torch.empty(planner.kv4_evict_workspace(pool.cache, keep), dtype=torch.uint8, device="cuda")
        return b

    def run(b, behind):
        stream = torch.cuda.current_stream()
        for i in range(rounds):
            cache, to = b["caches"][i].cache, b["caches"][i + 1].cache
            planner.add_rmsnorm_fp8(b["x"], deltas[i], gain, b["x"], None, None, y=b["y"], stream=stream)
            behind()
            qkv = b["y"].view(batch, -1, dim)
            planner.rope_append_kv4(qkv[:, :q_heads], qkv[:, q_heads:q_heads + heads], qkv[:, q_heads + heads:], rope,
                                    cu_fixed, b["lens"][i], cache, b["q"], stream=stream, rope_start=at[i])
            behind()
            torch.add(b["lens"][i], 1, out=b["len"])
            behind()
            planner.attention_kv4(b["q"].unsqueeze(1), cache, b["len"], b["out"][i], 0.2, b["ws"], lse=b["lse"][i],
                                  mass=b["mass"][i], mass_out=b["mass"][i], decay=0.9, stream=stream)
            behind()
            planner.kv4_evict(cache, b["len"], b["mass"][i], keep, recent, to, b["lens"][i + 1], b["mass"][i + 1], b["work"], stream=stream)
            behind()
    cu_fixed, at = cu_of([1] * batch), [i32([i + 5] * batch) for i in range(rounds)]
    apart, chain = buffers(pools[0]), buffers(pools[1])
    run(apart, torch.cuda.synchronize)
    planner.sync_check()
    first = [chain["x"].clone(), chain["mass"][0].clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run(chain, lambda: None)
    for _ in range(20):
        chain["x"].copy_(first[0])
        chain["mass"][0].copy_(first[1])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        for name in ("x", "y", "q"):
            assert torch.equal(chain[name], apart[name])
        for name in ("out", "lse", "mass", "lens"):
            for a, b in zip(chain[name], apart[name]):
                assert torch.equal(a, b), name
        for a, b in zip(chain["caches"], apart["caches"]):
            for t in ("k", "v", "ks", "vs"):
                assert torch.equal(getattr(a, t), getattr(b, t)), t
    planner.sync_check()


@pytest.mark.parametrize("cols,pitch", [(16, 24), (48, 56), (272, 280), (1024, 1032)])
def test_norm_in_place_on_rows_that_share_sectors(planner, cols, pitch):
    """Rows of 16 bytes more than a multiple of 32: a row's writes and its neighbour's reads lie in one sector."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    wide = torch.randn(3000, pitch, device="cuda", generator=g).to(torch.bfloat16)
    delta, w = torch.randn(3000, cols, device="cuda", generator=g).to(torch.bfloat16), torch.rand(cols, device="cuda", generator=g) + 0.5
    x, y = torch.empty(3000, cols, dtype=torch.bfloat16, device="cuda"), [torch.empty(3000, cols, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    behind = wide[:, cols:].clone()
    for _ in range(5):                                               # again and again on what the last one left
        planner.add_rmsnorm_fp8(wide[:, :cols], delta, w, x, None, None, y=y[0])
        planner.add_rmsnorm_fp8(wide[:, :cols], delta, w, wide[:, :cols], None, None, y=y[1])
        assert torch.equal(y[0], y[1]) and torch.equal(wide[:, :cols], x) and torch.equal(wide[:, cols:], behind)
    planner.sync_check()


def test_weights_units_and_tables_written_by_the_kernel_before(planner):
    """A copy into the weights, units, offsets or tables directly ahead of the call that goes by them."""
    heads, dim, page, n, times = 4, 64, 16, 50, 6
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.rand(*s, device="cuda", generator=g) + 0.5  # noqa: E731
    rows = (torch.randn(700, 256, device="cuda", generator=g)).to(torch.bfloat16)
    gains, norms, ropes = [rand(256) for _ in range(times)], [rand(dim) for _ in range(times)], [rand(64, dim) for _ in range(times)]
    units = [2.0 ** torch.randint(-3, 3, (heads,), device="cuda", generator=g).float() for _ in range(times)]
    k = torch.randn(n, heads, dim, device="cuda", generator=g).to(torch.bfloat16)
    orders = [torch.randperm(4, device="cuda", generator=g).to(torch.int32)[None] for _ in range(times)]
    firsts = [i32([i]) for i in range(times)]

    def state():
        pool = Pool4([64], heads, page, dim, spare=0)
        s = dict(pool=pool, gain=torch.empty(256, device="cuda"), norm=torch.empty(dim, device="cuda"), rope=torch.empty(64, dim, device="cuda"),
                 first=i32([0]), q=torch.empty_like(k), out=[])
        for _ in range(times):
            s["out"].append([torch.empty_like(rows), torch.empty_like(k), torch.empty_like(k), torch.empty_like(k),
                             torch.empty(1, n, heads, dim, dtype=torch.bfloat16, device="cuda")])
        s["ws"] = torch.empty(planner.attention_kv4_workspace(pool.cache), dtype=torch.uint8, device="cuda")
        return s
    cu = cu_of([n])

    def run(s, behind):
        stream, pool = torch.cuda.current_stream(), s["pool"]
        for i in range(times):
            y, q, kr, vr, att = s["out"][i]
            s["gain"].copy_(gains[i])
            behind()
            planner.add_rmsnorm_fp8(rows, None, s["gain"], None, None, None, y=y, stream=stream)
            behind()
            for a, b in ((s["rope"], ropes[i]), (s["first"], firsts[i]), (pool.table, orders[i]), (pool.units[0], units[i]), (pool.units[1], units[i])):
                a.copy_(b)
            s["norm"].copy_(norms[i])
            behind()
            planner.rope_append_kv4(k, k, k, s["rope"], cu, s["first"], pool.cache, q, q_norm=s["norm"], k_norm=s["norm"], stream=stream)
            behind()
            pool.units[1].copy_(units[i - 1])
            behind()
            planner.kv4_read(pool.cache, cu, s["first"], kr, vr, stream=stream)
            behind()
            s["first"].add_(n)
            behind()
            planner.attention_kv4(q.unsqueeze(0), pool.cache, s["first"], att, 0.125, s["ws"], stream=stream)
            behind()
    apart, chain = state(), state()
    run(apart, torch.cuda.synchronize)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run(chain, lambda: None)
    for _ in range(20):
        # (slots ahead of a round's first token may hold what the last replay left: both start from the same bytes)
        for t in ("k", "v", "ks", "vs"):
            getattr(chain["pool"], t).zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
    for t in ("k", "v", "ks", "vs"):
        getattr(apart["pool"], t).zero_()
    run(apart, torch.cuda.synchronize)
    planner.sync_check()
    for a, b in zip(chain["out"], apart["out"]):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
