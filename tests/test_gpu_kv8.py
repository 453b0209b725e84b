"""The 8-bit paged cache on the GPU: append (norm, rotation, quantisation), read-back and
attention over it, against the oracle in 64 bits.

Tolerances, derived before the first run. Half a step is 2^-8 (bf16), 2^-11 (f16), 2^-4 (e4m3)
relative, 2^-10 of the scale for subnormal e4m3.
  * A rotated, normed element a c - b s in fp32: three roundings and the table's two, the norm's
    chain (mean, root, reciprocal, two products) under eight more: 16 * 2^-24 (|a| + |b|).
  * Values copied without arithmetic (v; k without norm and rotation) are quantised exactly.
  * Attention, row r: every weight is off by 2^-11 (f16) and by the error of its exponent: the
    score's D products in fp32 (a truncating adder: 2 * 2^-24 a step) give D 2^-22 s_abs with
    s_abs = scale sum |q k|; the base-2 exponential 2^-21; the running sum n 2^-23; f16's smallest
    step 2^-25 for weights scaled by 2^7 at least gives n 2^-32 max|v|. Weights and their sum are
    both off: factor 2. Output: half a bf16 step of the result."""
import numpy as np
import pytest
import torch

from gpu_helpers import cuda, host, make_planner
from oracle import paged, quant

pytestmark = pytest.mark.gpu

BF16, F16 = 2.0 ** -8, 2.0 ** -11


@pytest.fixture(scope="module")
def planner():
    from cem_search_transformer_gb300 import binding, synthetic
    p = binding.Planner(synthetic.PRESETS["small"])
    yield p
    p.close()


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def codes_f64(c):
    return c.view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def cu_of(lens):
    return i32(np.concatenate([[0], np.cumsum(lens)]))


class Pool:
    """A cache whose pages hold NaN codes and absurd scales until something is written."""

    def __init__(self, lens, heads, page, dim, spare=2, seed=0):
        from cem_search_transformer_gb300 import binding
        rng = np.random.default_rng(seed)
        need = [-(-int(n) // page) for n in lens]
        self.pages, self.page = sum(need) + spare, page
        order = rng.permutation(self.pages)
        self.table_np = np.full((len(lens), max(1, max(need))), -1, np.int64)
        at = 0
        for s, n in enumerate(need):
            self.table_np[s, :n] = order[at:at + n]
            at += n
        shape = (self.pages, heads, page, dim)
        self.k = torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda")
        self.v = torch.full(shape, 0xff, dtype=torch.uint8, device="cuda")
        self.ks = torch.full((self.pages, heads), float("nan"), device="cuda")
        self.vs = torch.full((self.pages, heads), 1e30, device="cuda")
        self.table = i32(self.table_np)
        self.cache = binding.KvCache8(self.k, self.v, self.ks, self.vs, self.table)

    def fill(self, lens, seed, spread=2):
        """Random codes and scales for the first lens[s] tokens of each sequence; the rest of
        their last pages keeps NaN codes."""
        rng = np.random.default_rng(seed)
        heads, dim = self.k.shape[1], self.k.shape[3]
        out = []
        k, v = self.k.cpu(), self.v.cpu()
        ks, vs = self.ks.cpu(), self.vs.cpu()
        for s, n in enumerate(lens):
            kk, vv = np.zeros((n, heads, dim)), np.zeros((n, heads, dim))
            for i in range(-(-int(n) // self.page)):
                pg, m = int(self.table_np[s, i]), min(self.page, n - i * self.page)
                for codes, scales, vals, low in ((k, ks, kk, -8), (v, vs, vv, -7)):
                    x = torch.from_numpy(rng.standard_normal((heads, m, dim)) * 100).float()
                    c = x.clamp(-448, 448).to(torch.float8_e4m3fn)
                    sc = np.exp2(rng.integers(low - spread, low + 1, heads)).astype(np.float32)
                    codes[pg, :, :m] = c.view(torch.uint8)
                    scales[pg] = torch.from_numpy(sc)
                    vals[i * self.page:i * self.page + m] = (c.float().numpy() * sc[:, None, None]).transpose(1, 0, 2)
            out.append((kk, vv))
        for dst, src in ((self.k, k), (self.v, v), (self.ks, ks), (self.vs, vs)):
            dst.copy_(src)
        return out

    def values(self, s, n):
        kk, vv = [], []
        for i in range(-(-n // self.page)):
            pg = int(self.table_np[s, i])
            for codes, scales, to in ((self.k, self.ks, kk), (self.v, self.vs, vv)):
                to.append((codes_f64(codes[pg]) * f64(scales[pg])[:, None, None]).transpose(1, 0, 2))
        return np.concatenate(kk)[:n], np.concatenate(vv)[:n]


# ---- rotary table ----

@pytest.mark.parametrize("positions,rot,base,factor", [(1, 16, 10000.0, 1.0), (1000, 64, 10000.0, 1.0),
                                                       (131077, 128, 500000.0, 8.0)])
def test_rope_table(planner, positions, rot, base, factor):
    t = planner.rope_table(positions, rot, base, factor)
    planner.sync_check()
    # correctly rounded but for the angle's own error: position * 2^-50 rad at most
    assert np.max(np.abs(f64(t) - paged.rope_table(positions, rot, base, factor))) <= 2.0 ** -24 + positions * 2.0 ** -50


# ---- append and read ----

def check_append(planner, new, old, q_heads, kv_heads, dim, page, rot, interleaved, norm, seed, chunks=(None,)):
    """Append `old` then `new` tokens per sequence; compare the pages with the oracle's."""
    rng = np.random.default_rng(seed)
    lens = [a + b for a, b in zip(new, old)]
    pool = Pool(lens, kv_heads, page, dim, seed=seed)
    table = planner.rope_table(max(lens) + 1, rot) if rot else None
    t64 = paged.rope_table(max(lens) + 1, rot) if rot else None
    wq = rng.uniform(0.5, 1.5, dim).astype(np.float32) if norm else None
    wk = rng.uniform(0.5, 1.5, dim).astype(np.float32) if norm else None
    ref = [[None, None] for _ in lens]
    for start, count, size in ((np.zeros(len(lens), int), old, 1.0), (np.array(old), new, 4.0)):
        n = int(sum(count))
        if n == 0:
            continue
        qkv = bf16(rng.standard_normal((n + 3, q_heads + 2 * kv_heads, dim)) * size).cuda()
        q, k, v = qkv[:, :q_heads], qkv[:, q_heads:q_heads + kv_heads], qkv[:, q_heads + kv_heads:]
        q_out = torch.full((n + 3, q_heads, dim), 77.0, dtype=torch.bfloat16, device="cuda")
        k_out = torch.full((n + 3, kv_heads, dim), 77.0, dtype=torch.bfloat16, device="cuda")
        planner.rope_append_kv8(q, k, v, table, cu_of(count), i32(start), pool.cache, q_out,
                                q_norm=None if wq is None else cuda(wq), k_norm=None if wk is None else cuda(wk),
                                interleaved=interleaved, k_out=k_out)
        planner.sync_check()
        assert torch.all(q_out[n:] == 77) and torch.all(k_out[n:] == 77)   # behind the last sequence
        at = 0
        for s, c in enumerate(count):
            rows, pos = slice(at, at + c), start[s] + np.arange(c)
            at += c
            for got, x, w in ((q_out, q, wq), (k_out, k, wk)):
                want = paged.norm_rotate(f64(x[rows]), w, t64, pos, interleaved)
                both = np.abs(paged.norm_rotate(f64(x[rows]), w, None, pos, interleaved)).max(-1, keepdims=True) * 2 if c else 0
                assert np.all(np.abs(f64(got[rows]) - want) <= BF16 * np.abs(want) + 16 * 2.0 ** -24 * both)
            kk = paged.norm_rotate(f64(k[rows]), wk, t64, pos, interleaved)
            ref[s] = [kk if ref[s][0] is None else np.concatenate([ref[s][0], kk]),
                      f64(v[rows]) if ref[s][1] is None else np.concatenate([ref[s][1], f64(v[rows])])]
    exact_k = not rot and not norm
    for s, n in enumerate(lens):
        if n == 0:
            continue
        got = pool.values(s, n)
        for which, scales in ((0, pool.ks), (1, pool.vs)):
            x = ref[s][which]
            for i in range(-(-n // page)):
                lo, hi = i * page, min(n, i * page + page)
                o = min(max(old[s] - lo, 0), hi - lo)          # earlier tokens in this page
                sc = f64(scales[int(pool.table_np[s, i])])
                for h in range(kv_heads):
                    a, b = x[lo:lo + o, h], x[lo + o:hi, h]
                    e0 = 2.0 ** paged.block_exponent(np.abs(a).max()) if o else 0.0
                    held = quant.round_to_e4m3(a / e0) if o else np.zeros((0, dim))
                    if len(b):
                        codes, want = paged.append_block(held, e0, b)
                    else:
                        codes, want = held, e0
                    if which == 1 or exact_k:
                        assert sc[h] == want
                        assert np.array_equal(got[which][lo:hi, h], codes * want)
                    else:
                        # fp32 against 64 bits: the maximum may fall on the other side of a border
                        near = np.abs(x[lo:hi, h]).max()
                        assert sc[h] == want or abs(near / (448 * min(sc[h], want)) - 1) < 2.0 ** -20
                        tol = np.maximum(np.abs(x[lo:hi, h]) * 2.0 ** -4, sc[h] * 2.0 ** -10)
                        tol[:o] *= 2                             # rounded twice where the scale grew
                        tol += 16 * 2.0 ** -24 * 2 * np.abs(x[lo:hi, h]).max()
                        assert np.all(np.abs(got[which][lo:hi, h] - x[lo:hi, h]) <= tol)
    return pool, lens


@pytest.mark.parametrize("new,old,q_heads,kv_heads,dim,page,rot,interleaved,norm", [
    ([1], [0], 1, 1, 64, 16, 64, False, False),
    ([1], [300], 16, 16, 64, 16, 32, True, False),
    ([1, 1, 1, 1], [15, 16, 17, 0], 8, 2, 128, 16, 128, False, True),
    ([3, 0, 1, 2], [14, 5, 63, 31], 6, 2, 64, 32, 16, True, True),
    ([5], [126], 4, 1, 128, 128, 0, False, False),
    ([130, 0, 7, 65], [3, 70, 0, 64], 4, 2, 128, 64, 128, False, True),
    ([258, 33], [258, 1], 16, 16, 64, 32, 64, False, False),
    ([200, 1], [60, 127], 3, 3, 128, 128, 96, True, True),
    ([40], [0], 7, 1, 64, 128, 48, False, True),
    ([17, 90], [9, 0], 2, 2, 64, 16, 0, False, False),
])
def test_append_matches_oracle(planner, new, old, q_heads, kv_heads, dim, page, rot, interleaved, norm):
    check_append(planner, new, old, q_heads, kv_heads, dim, page, rot, interleaved, norm, seed=len(new) + dim + page)


@pytest.mark.parametrize("dim,page,n", [(64, 16, 50), (128, 128, 200), (128, 64, 100)])
def test_both_launch_shapes_give_the_same_bits(planner, dim, page, n):
    """A batch padded with empty sequences is appended by warps, a single one by CTAs."""
    rng = np.random.default_rng(n)
    x = [bf16(rng.standard_normal((n, h, dim))).cuda() for h in (4, 2, 2)]
    table = planner.rope_table(n + 8, dim // 2)
    got = []
    for batch in (1, n):
        pool = Pool([n + 5] + [0] * (batch - 1), 2, page, dim)
        q_out, k_out = torch.empty_like(x[0]), torch.empty_like(x[1])
        planner.rope_append_kv8(*x, table, cu_of([n] + [0] * (batch - 1)), i32([5] + [0] * (batch - 1)), pool.cache,
                                q_out, k_out=k_out)
        planner.sync_check()
        pages = [int(p) for p in pool.table_np[0]]
        got.append([q_out, k_out, pool.k[pages], pool.v[pages], pool.ks[pages], pool.vs[pages]])
    # the first page's five earlier slots hold NaN codes on an absurd scale, moved alike
    for a, b in zip(*got):
        assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))


def test_append_again_changes_nothing_and_in_place(planner):
    rng = np.random.default_rng(3)
    n, heads, dim, page = 37, 2, 128, 32
    pool = Pool([n + 11], heads, page, dim)
    pool.fill([11], 1)
    q = bf16(rng.standard_normal((n, heads, dim))).cuda()
    k, v = bf16(rng.standard_normal((n, heads, dim)) * 9).cuda(), bf16(rng.standard_normal((n, heads, dim)) * 9).cuda()
    table = planner.rope_table(64, dim)
    out = torch.empty_like(q)
    for _ in range(2):
        planner.rope_append_kv8(q, k, v, table, cu_of([n]), i32([11]), pool.cache, out)
        planner.sync_check()
        state = [t.clone() for t in (pool.k, pool.v, pool.ks, pool.vs)]
        if _ == 0:
            first = state
    assert all(torch.equal(a, b) for a, b in zip(first[:2], state[:2]))
    assert all(torch.equal(a.nan_to_num(), b.nan_to_num()) for a, b in zip(first[2:], state[2:]))
    q2, k2 = q.clone(), k.clone()
    planner.rope_append_kv8(q2, k2, v, table, cu_of([n]), i32([11]), pool.cache, q2, k_out=k2)
    planner.sync_check()
    assert torch.equal(q2, out) and not torch.equal(k2, k)
    with pytest.raises(Exception, match="dense"):
        wide = torch.zeros(n, 2 * heads, dim, dtype=torch.bfloat16, device="cuda")
        from cem_search_transformer_gb300 import binding
        s = pool.cache.struct
        planner._check(planner.lib.jepa_rope_append_kv8(
            planner.h, pool.cache.ref, wide.data_ptr(), 2 * heads * dim, k.data_ptr(), heads * dim, v.data_ptr(),
            heads * dim, n, heads, None, None, 0.0, table.data_ptr(), 64, dim, 0, cu_of([n]).data_ptr(),
            i32([11]).data_ptr(), wide.data_ptr(), None, None), "rope_append_kv8")


def test_append_of_infinities_and_nan(planner):
    n, heads, dim, page = 20, 1, 64, 16
    x = np.random.default_rng(0).standard_normal((n, heads, dim))
    x[3, 0, 5], x[3, 0, 6], x[18, 0, 0] = np.inf, -np.inf, np.nan
    pool = Pool([n], heads, page, dim)
    k = bf16(x).cuda()
    planner.rope_append_kv8(None, k, k, None, cu_of([n]), i32([0]), pool.cache, None)
    planner.sync_check()
    ref = f64(k)
    got, _ = pool.values(0, n)
    for lo, hi in ((0, 16), (16, 20)):
        codes, scale = paged.append_block(np.zeros((0, dim)), 1.0, ref[lo:hi, 0])
        assert np.array_equal(got[lo:hi, 0], codes * scale, equal_nan=True)
    assert got[3, 0, 5] == 448 * 2.0 ** 40 and np.isnan(got[18, 0, 0])


@pytest.mark.parametrize("by_warp", [True, False])
def test_bad_pages_and_positions_are_skipped_and_reported(planner, by_warp):
    from cem_search_transformer_gb300 import binding
    n, heads, dim, page = 40, 2, 64, 16
    pool = Pool([n, n], heads, page, dim, spare=0)
    table = planner.rope_table(n, dim)
    x = bf16(np.random.default_rng(1).standard_normal((2 * n, heads, dim))).cuda()
    pad = [0] * (2 * n if by_warp else 0)
    t = np.full((2 + len(pad), pool.table_np.shape[1]), -1)
    t[:2] = pool.table_np
    keep = int(t[0, 2])
    t[0, 1], t[1, 0] = 10 ** 6, -5
    cache = binding.KvCache8(pool.k, pool.v, pool.ks, pool.vs, i32(t))
    before = pool.k.clone()
    out = torch.zeros(2 * n, heads, dim, dtype=torch.bfloat16, device="cuda")
    planner.rope_append_kv8(x, x, x, table, cu_of([n, n] + pad), i32([0, 0] + pad), cache, out)
    with pytest.raises(binding.JepaError, match="outside its buffer") as e:
        planner.sync_check()
    assert e.value.status == 1
    planner.sync_check()                                   # reported once
    touched = {int(t[0, 0]), keep, int(t[1, 1]), int(t[1, 2])}
    for pg in range(pool.pages):
        assert torch.equal(pool.k[pg], before[pg]) == (pg not in touched)
    # positions past the rotary table and the page table, and a negative start
    for start in (30, 10 ** 9, -1, 2 ** 31 - 2):
        planner.rope_append_kv8(x[:n], x[:n], x[:n], table, cu_of([n, 0] + pad), i32([start, 0] + pad), cache, out[:n])
        with pytest.raises(binding.JepaError, match="outside its buffer"):
            planner.sync_check()


def test_read_windows(planner):
    lens, heads, dim, page = [100, 0, 33, 1], 3, 128, 32
    pool = Pool(lens, heads, page, dim)
    ref = pool.fill(lens, 5)
    first = [17, 0, 32, 0]
    count = [n - f for n, f in zip(lens, first)]
    total = sum(count)
    k = torch.full((total + 2, heads, dim), 55.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    planner.kv8_read(pool.cache, cu_of(count), i32(first), k, v)
    planner.sync_check()
    assert torch.all(k[total:] == 55) and torch.all(v[total:] == 55)
    assert np.array_equal(f64(k[:total]), np.concatenate([r[0][f:] for r, f in zip(ref, first)]))
    assert np.array_equal(f64(v[:total]), np.concatenate([r[1][f:] for r, f in zip(ref, first)]))


# ---- attention over the cache ----

def attention_tolerance(want, a, s_abs, n, dim, vmax):
    delta = dim * 2.0 ** -22 * s_abs[..., None] + 2.0 ** -21 + n * 2.0 ** -23
    return BF16 * np.abs(want) + (1 + BF16) * (2 * a * (F16 + delta) + n * 2.0 ** -32 * vmax)


def lse_tolerance(s_abs, n, dim, lse):
    return dim * 2.0 ** -22 * s_abs + 2.0 ** -20 + n * 2.0 ** -23 + 4 * 2.0 ** -24 * np.abs(np.where(np.isfinite(lse), lse, 0))


def check_attention(planner, pool, ref, lens, q_tokens, q_heads, causal, seed, scale=None, q=None, workspace=None):
    rng = np.random.default_rng(seed)
    dim = pool.k.shape[3]
    scale = dim ** -0.5 if scale is None else scale
    if q is None:
        q = bf16(rng.standard_normal((len(lens), q_tokens, q_heads, dim))).cuda()
    out = torch.full_like(q, 9.0)
    lse = torch.full(q.shape[:3], 9.0, device="cuda")
    if workspace is None:
        workspace = torch.empty(planner.attention_kv8_workspace(pool.cache), dtype=torch.uint8, device="cuda")
    planner.attention_kv8(q, pool.cache, i32(lens), out, scale, workspace, causal=causal, lse=lse)
    planner.sync_check()
    for s, n in enumerate(lens):
        k, v = ref[s]
        lim = [max(0, n - q_tokens + t + 1) if causal else n for t in range(q_tokens)]
        want, want_lse, a, s_abs = paged.softmax_rows(f64(q[s]), k[:n], v[:n], lim, scale)
        got, got_lse = f64(out[s]), f64(lse[s])
        assert np.all(np.isfinite(got)), s
        assert np.all(np.abs(got - want) <= attention_tolerance(want, a, s_abs, n, dim, np.abs(v[:n]).max() if n else 0)), \
            (s, np.abs(got - want).max())
        empty = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(got_lse), empty)
        err = np.abs(got_lse[~empty] - want_lse[~empty])
        assert np.all(err <= lse_tolerance(s_abs, n, dim, want_lse)[~empty]), (s, err.max())
    return out, lse


@pytest.mark.parametrize("lens,q_tokens,q_heads,kv_heads,dim,page,causal", [
    ([1], 1, 1, 1, 64, 16, True),
    ([0], 1, 2, 1, 128, 16, True),                        # nothing cached
    ([5, 0, 1, 64], 1, 4, 2, 128, 32, True),
    ([63, 64, 65, 128], 1, 8, 1, 128, 64, True),          # around a unit of 64 keys
    ([127, 128, 129, 257], 1, 3, 3, 64, 16, True),        # around a unit of 128 keys
    ([517], 1, 16, 16, 64, 32, True),
    ([2, 1, 0, 40], 4, 6, 2, 128, 16, True),              # rows that see nothing
    ([300, 17], 8, 14, 2, 64, 128, True),                 # 56 rows: four tiles
    ([70, 33], 3, 5, 1, 128, 32, False),
    ([776, 776, 12], 2, 4, 4, 64, 16, False),
    ([6000, 11, 2049], 1, 8, 2, 128, 128, True),          # split over many CTAs
    ([20011], 2, 7, 1, 64, 64, True),
    ([40] * 70, 1, 4, 4, 128, 16, True),                  # more sequences than a warp's scan
])
def test_attention_matches_oracle(planner, lens, q_tokens, q_heads, kv_heads, dim, page, causal):
    pool = Pool(lens, kv_heads, page, dim, seed=len(lens))
    ref = pool.fill(lens, 7)
    check_attention(planner, pool, ref, lens, q_tokens, q_heads, causal, seed=q_heads)


@pytest.mark.parametrize("dim", [64, 128])
def test_scales_far_apart(planner, dim):
    """Pages whose scales differ by up to 2^30, in either order, and large scores."""
    lens = [700, 700]
    pool = Pool(lens, 2, 16, dim)
    ref = pool.fill(lens, 3)
    rng = np.random.default_rng(0)
    for s in range(2):
        for i in range(pool.table_np.shape[1]):
            pg = int(pool.table_np[s, i])
            e = rng.integers(-15, 16) if s == 0 else 15 - i
            old = f64(pool.vs[pg])
            pool.vs[pg] = 2.0 ** float(e)
            rows = slice(16 * i, min(700, 16 * i + 16))
            ref[s][1][rows] *= (2.0 ** float(e) / old)[None, :, None]
    check_attention(planner, pool, ref, lens, 1, 4, True, seed=1)
    check_attention(planner, pool, ref, lens, 1, 4, True, seed=2, scale=1.0)


def test_magnitudes_of_queries(planner):
    """Query rows from 2^-60 to 2^60 (the softmax then picks one key), and a row of zeros."""
    lens, dim = [200], 128
    pool = Pool(lens, 1, 64, dim)
    ref = pool.fill(lens, 9, spread=0)
    q = np.random.default_rng(4).standard_normal((1, 1, 6, dim))
    q *= np.array([2.0 ** -60, 2.0 ** -20, 1, 2.0 ** 20, 2.0 ** 60, 0])[:, None]
    # with scores this large the exponent's error decides nothing but near ties: compare the
    # rows whose scores fp32 resolves
    qt = bf16(q).cuda()
    keep = qt.clone()
    keep[:, :, 3:5] = 0
    check_attention(planner, pool, ref, lens, 1, 6, True, seed=0, q=keep)
    out = torch.empty_like(qt)
    ws = torch.empty(planner.attention_kv8_workspace(pool.cache), dtype=torch.uint8, device="cuda")
    planner.attention_kv8(qt, pool.cache, i32(lens), out, dim ** -0.5, ws)
    planner.sync_check()
    for h in (3, 4):
        best = np.argmax(f64(qt[0, 0, h]) @ ref[0][0][:, 0].T)
        assert np.max(np.abs(f64(out[0, 0, h]) - ref[0][1][best, 0])) <= BF16 * np.abs(ref[0][1][best, 0]).max()


@pytest.mark.parametrize("dim", [64, 128])
def test_unseen_keys_do_not_reach_a_query(planner, dim):
    """NaN in the keys and values of the newest tokens: queries before them are untouched, those
    that see them become NaN (values) in just those elements."""
    lens, tq, page = [75, 40], 4, 16
    pool = Pool(lens, 1, page, dim)
    ref = pool.fill(lens, 2)
    clean, _ = check_attention(planner, pool, ref, lens, tq, 2, True, seed=5)
    n = lens[0]
    pg, off = int(pool.table_np[0, (n - 2) // page]), (n - 2) % page
    pool.v[pg, 0, off, 3] = 0x7f
    pool.v[pg, 0, off, dim - 1] = 0xff
    q = bf16(np.random.default_rng(5).standard_normal((2, tq, 2, dim))).cuda()
    out = torch.empty_like(q)
    ws = torch.empty(planner.attention_kv8_workspace(pool.cache), dtype=torch.uint8, device="cuda")
    planner.attention_kv8(q, pool.cache, i32(lens), out, dim ** -0.5, ws)
    planner.sync_check()
    assert torch.equal(out[0, :2], clean[0, :2]) and torch.equal(out[1], clean[1])
    bad = torch.zeros(dim, dtype=torch.bool, device="cuda")
    bad[3] = bad[dim - 1] = True
    assert torch.all(torch.isnan(out[0, 2:][..., bad]))
    assert torch.equal(out[0, 2:][..., ~bad], clean[0, 2:][..., ~bad])
    pg, off = int(pool.table_np[0, (n - 1) // page]), (n - 1) % page
    pool.k[pg, 0, off, 0] = 0x7f                             # the newest key: only the last query sees it
    planner.attention_kv8(q, pool.cache, i32(lens), out, dim ** -0.5, ws)
    planner.sync_check()
    assert torch.equal(out[0, :2], clean[0, :2]) and torch.all(torch.isnan(out[0, 3]))


def test_nan_queries_stay_in_their_row(planner):
    lens = [90]
    pool = Pool(lens, 1, 32, 128)
    ref = pool.fill(lens, 2)
    clean, _ = check_attention(planner, pool, ref, lens, 1, 4, True, seed=5)
    q = bf16(np.random.default_rng(5).standard_normal((1, 1, 4, 128))).cuda()
    q[0, 0, 1, 7] = float("nan")
    out, lse = torch.empty_like(q), torch.zeros(1, 1, 4, device="cuda")
    ws = torch.empty(planner.attention_kv8_workspace(pool.cache), dtype=torch.uint8, device="cuda")
    planner.attention_kv8(q, pool.cache, i32(lens), out, 128 ** -0.5, ws, lse=lse)
    planner.sync_check()
    assert torch.all(torch.isnan(out[0, 0, 1])) and torch.isnan(lse[0, 0, 1])
    keep = [0, 2, 3]
    assert torch.equal(out[0, 0, keep], clean[0, 0, keep])


def test_shared_pages_and_bad_lengths(planner):
    """Two sequences with a common prefix name the same pages; lengths out of range are clamped
    and reported."""
    from cem_search_transformer_gb300 import binding
    lens, page, dim = [64, 64], 32, 64
    pool = Pool(lens, 2, page, dim)
    ref = pool.fill(lens, 4)
    t = pool.table_np.copy()
    t[1, 0] = t[0, 0]
    ref[1][0][:page], ref[1][1][:page] = ref[0][0][:page], ref[0][1][:page]
    pool.table.copy_(i32(t))
    check_attention(planner, pool, ref, lens, 1, 4, True, seed=1)
    q = torch.zeros(2, 1, 4, dim, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(planner.attention_kv8_workspace(pool.cache), dtype=torch.uint8, device="cuda")
    for bad in ([65, 64], [-1, 3]):
        planner.attention_kv8(q, pool.cache, i32(bad), torch.empty_like(q), 0.1, ws)
        with pytest.raises(binding.JepaError, match="outside its buffer"):
            planner.sync_check()
    t[0, 1] = pool.pages
    pool.table.copy_(i32(t))
    planner.attention_kv8(q, pool.cache, i32(lens), torch.empty_like(q), 0.1, ws)
    with pytest.raises(binding.JepaError, match="outside its buffer"):
        planner.sync_check()


def test_refusals_of_the_library(planner):
    from cem_search_transformer_gb300 import binding
    pool = Pool([32], 2, 16, 64)
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    n = planner.attention_kv8_workspace(pool.cache)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    ok = dict(q=q, cache=pool.cache, kv_len=i32([3]), out=torch.empty_like(q), scale=0.1, workspace=ws)
    for change, match in ((dict(scale=0.0), "bad argument"), (dict(scale=float("nan")), "bad argument"),
                          (dict(workspace=ws[:n - 1]), "too small"), (dict(workspace=ws[1:]), "bad argument"),
                          (dict(q=q[:, :, :3].contiguous()), "bad argument"),       # 3 heads over 2
                          (dict(out=q[:, :, :2].contiguous()), "elements")):
        with pytest.raises(binding.JepaError, match=match):
            planner.attention_kv8(**{**ok, **change})
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    for table, match in ((torch.zeros(8, 24, device="cuda"), "rotary"), (torch.zeros(8, 80, device="cuda"), "rotary")):
        with pytest.raises(binding.JepaError, match=match):
            planner.rope_append_kv8(None, x, x, table, cu_of([3]), i32([0]), pool.cache, None)
    with pytest.raises(binding.JepaError, match="together"):
        planner.rope_append_kv8(x, x, x, None, cu_of([3]), i32([0]), pool.cache, None)
    from cem_search_transformer_gb300 import synthetic
    fp32 = binding.Planner(synthetic.PRESETS["tiny"])
    with pytest.raises(binding.JepaError, match="bf16 context"):
        fp32.attention_kv8(**ok)
    fp32.close()


def test_graph_replay_reads_lengths_anew_and_streams_run_apart(planner):
    lens, page, dim = [3000, 50], 64, 128
    pool = Pool(lens, 2, page, dim)
    ref = pool.fill(lens, 8)
    q = bf16(np.random.default_rng(11).standard_normal((2, 1, 8, dim))).cuda()
    need = planner.attention_kv8_workspace(pool.cache)
    kv_len = i32(lens)

    def direct(n):
        out = torch.empty_like(q)
        planner.attention_kv8(q, pool.cache, i32(n), out, 0.09, torch.empty(need, dtype=torch.uint8, device="cuda"))
        planner.sync_check()
        return out
    want = {n: direct(list(n)) for n in ((3000, 50), (64, 0), (2999, 1))}
    calls = []
    for _ in range(2):
        out, ws = torch.empty_like(q), torch.empty(need, dtype=torch.uint8, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            planner.attention_kv8(q, pool.cache, kv_len, out, 0.09, ws, stream=torch.cuda.current_stream())
        calls.append((graph, out, side))
    for n, w in want.items():
        kv_len.copy_(i32(list(n)))
        torch.cuda.synchronize()
        for graph, out, side in calls:
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for _, out, _ in calls:
            assert torch.equal(out, w)
    # the same bits again: no order of CTAs enters the result
    for _ in range(3):
        assert torch.equal(direct([3000, 50]), want[(3000, 50)])
    del calls


@pytest.mark.parametrize("by_warp", [True, False])
def test_tokens_ahead_of_the_first_sequence_are_left(planner, by_warp):
    """Offsets that begin behind packed token 0: the rows ahead belong to nobody."""
    n, ahead, heads, dim, page = 70, 37, 2, 64, 32
    pool = Pool([n], heads, page, dim)
    pad = n if by_warp else 0
    x = bf16(np.random.default_rng(3).standard_normal((n + ahead, heads, dim))).cuda()
    from cem_search_transformer_gb300 import binding
    t = np.full((1 + pad, pool.table_np.shape[1]), -1)
    t[0] = pool.table_np[0]
    cache = binding.KvCache8(pool.k, pool.v, pool.ks, pool.vs, i32(t))
    cu = i32([ahead] + [ahead + n] * (1 + pad))
    q_out = torch.full_like(x, 5.0)
    planner.rope_append_kv8(x, x, x, None, cu, i32([0] * (1 + pad)), cache, q_out)
    k, v = torch.full_like(x, 5.0), torch.full_like(x, 5.0)
    planner.kv8_read(cache, cu, i32([0] * (1 + pad)), k, v)
    planner.sync_check()
    for got in (q_out, k, v):
        assert torch.all(got[:ahead] == 5)
    assert torch.equal(q_out[ahead:], x[ahead:])
    ref = f64(x)[ahead:]
    for lo in range(0, n, page):
        for h in range(heads):
            codes, scale = paged.append_block(np.zeros((0, dim)), 1.0, ref[lo:lo + page, h])
            assert np.array_equal(f64(k[ahead:])[lo:lo + page, h], codes * scale)
            assert np.array_equal(f64(v[ahead:])[lo:lo + page, h], codes * scale)


def test_thousands_of_sequences(planner):
    """More sequences than two levels of the search hold, most of them with one token or none."""
    rng = np.random.default_rng(8)
    batch, heads, dim, page = 2500, 1, 64, 16
    new = rng.integers(0, 3, batch)
    old = rng.integers(0, 20, batch)
    n = int(new.sum())
    most = -(-int((new + old).max()) // page)
    table = np.arange(batch * most).reshape(batch, most)
    from cem_search_transformer_gb300 import binding
    shape = (batch * most, heads, page, dim)
    k, v = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full(shape[:2], 2.0 ** -8, device="cuda") for _ in range(2))
    cache = binding.KvCache8(k, v, ks, vs, i32(table))
    x = bf16(rng.standard_normal((n, heads, dim))).cuda()
    planner.rope_append_kv8(None, x, x, None, cu_of(new), i32(old), cache, None)
    got, got_v = torch.empty_like(x), torch.empty_like(x)
    planner.kv8_read(cache, cu_of(new), i32(old), got, got_v)
    planner.sync_check()
    err = np.abs(f64(got) - f64(x))
    top = np.abs(f64(x)).max((1, 2), keepdims=True)
    # half an e4m3 step; the block's scale is set by at most its two new tokens (and 2^-8 before)
    assert np.all(err <= np.maximum(np.abs(f64(x)) * 2.0 ** -4, 2 * 4 * top.max() / 448 * 2.0 ** -10))
    assert torch.equal(got, got_v)
    q = bf16(rng.standard_normal((batch, 1, 2, dim))).cuda()
    lens = new + old
    out = torch.full_like(q, 3.0)
    ws = torch.empty(planner.attention_kv8_workspace(cache), dtype=torch.uint8, device="cuda")
    planner.attention_kv8(q, cache, i32(lens), out, 0.125, ws)
    planner.sync_check()
    assert torch.all(out[torch.from_numpy(lens == 0).cuda()] == 0)
    for s in rng.integers(0, batch, 20):
        m = int(lens[s])
        if m:
            pages = [int(p) for p in table[s][:-(-m // page)]]
            kk, vv = (np.concatenate([(codes_f64(c[p]) * f64(sc[p])[:, None, None]).transpose(1, 0, 2) for p in pages])[:m]
                      for c, sc in ((k, ks), (v, vs)))
            want, _, a, s_abs = paged.softmax_rows(f64(q[s]), kk, vv, [m], 0.125)
            assert np.all(np.abs(f64(out[s]) - want) <= attention_tolerance(want, a, s_abs, m, dim, np.abs(vv).max()))


def test_offsets_past_32_bits(planner):
    """Pages behind the first 4 GiB of a pool: appended, read back and attended to."""
    from cem_search_transformer_gb300 import binding
    heads, page, dim = 8, 64, 128
    pages = (5 << 30) // (heads * page * dim)
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GiB")
    k, v = (torch.empty(pages, heads, page, dim, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(pages, heads, device="cuda") for _ in range(2))
    lens = [150, 90]
    table = np.array([[pages - 1, 3, pages - 7], [pages - 2, pages - 3, 0]])
    cache = binding.KvCache8(k, v, ks, vs, i32(table))
    x = bf16(np.random.default_rng(2).standard_normal((sum(lens), heads, dim))).cuda()
    y = bf16(np.random.default_rng(3).standard_normal((sum(lens), heads, dim))).cuda()
    planner.rope_append_kv8(None, x, y, None, cu_of(lens), i32([0, 0]), cache, None)
    rk, rv = torch.empty_like(x), torch.empty_like(x)
    planner.kv8_read(cache, cu_of(lens), i32([0, 0]), rk, rv)
    planner.sync_check()
    for got, want in ((rk, x), (rv, y)):
        assert np.all(np.abs(f64(got) - f64(want)) <= np.maximum(np.abs(f64(want)) * 2.0 ** -4, 2 * 6.0 / 448 * 2.0 ** -10))
    q = bf16(np.random.default_rng(4).standard_normal((2, 1, 16, dim))).cuda()
    out = torch.empty_like(q)
    ws = torch.empty(planner.attention_kv8_workspace(cache), dtype=torch.uint8, device="cuda")
    planner.attention_kv8(q, cache, i32(lens), out, dim ** -0.5, ws)
    planner.sync_check()
    at = 0
    for s, n in enumerate(lens):
        kk, vv = f64(rk[at:at + n]), f64(rv[at:at + n])
        at += n
        want, _, a, s_abs = paged.softmax_rows(f64(q[s]), kk, vv, [n], dim ** -0.5)
        assert np.all(np.abs(f64(out[s]) - want) <= attention_tolerance(want, a, s_abs, n, dim, np.abs(vv).max()))


@pytest.mark.parametrize("dim", [64, 128])
def test_scales_that_are_no_powers_of_two(planner, dim):
    """A cache written by others: any scale in the range stands for code * scale."""
    lens = [400, 37]
    pool = Pool(lens, 2, 32, dim)
    ref = pool.fill(lens, 3)
    rng = np.random.default_rng(1)
    for s in range(2):
        for i in range(-(-lens[s] // 32)):
            pg, rows = int(pool.table_np[s, i]), slice(32 * i, min(lens[s], 32 * i + 32))
            for scales, which in ((pool.ks, 0), (pool.vs, 1)):
                f = rng.uniform(0.6, 1.7, 2).astype(np.float32)
                old = f64(scales[pg])
                scales[pg] = cuda(f) * scales[pg]
                ref[s][which][rows] *= (f64(scales[pg]) / old)[None, :, None]
    check_attention(planner, pool, ref, lens, 1, 4, True, seed=1)


@pytest.mark.parametrize("n_new", [[1, 1, 1], [70, 3, 129]])
def test_captured_append_attention_and_read(planner, n_new):
    """Copies, fills, torch's kernels and a joined stream ahead of the calls of one graph."""
    page, dim, heads, q_heads = 32, 64, 2, 4
    old = [40, 0, 95]
    total, cu = sum(n_new), cu_of(n_new)
    lens = [a + b for a, b in zip(old, n_new)]
    start, kv_len = i32(old), i32(lens)
    rng = np.random.default_rng(21)
    rounds = [[bf16(rng.standard_normal((total, h, dim))).cuda() for h in (q_heads, heads, heads)] for _ in range(4)]
    rope = planner.rope_table(256, dim)
    past = [bf16(rng.standard_normal((sum(old), heads, dim))).cuda() for _ in range(2)]

    def fresh():
        pool = Pool(lens, heads, page, dim, seed=5)
        planner.rope_append_kv8(None, *past, rope, cu_of(old), i32([0] * 3), pool.cache, None)
        return pool

    def steps(pool, x, q_out, k, v, att, ws):
        planner.rope_append_kv8(*x, rope, cu, start, pool.cache, q_out, stream=torch.cuda.current_stream())
        planner.attention_kv8(q_out[-3:].unsqueeze(1), pool.cache, kv_len, att, 0.125, ws,
                              stream=torch.cuda.current_stream())
        planner.kv8_read(pool.cache, cu, start, k, v, stream=torch.cuda.current_stream())

    def buffers():
        return [torch.empty(total, h, dim, dtype=torch.bfloat16, device="cuda") for h in (q_heads, heads, heads)] + \
            [torch.empty(3, 1, q_heads, dim, dtype=torch.bfloat16, device="cuda")]

    pool, x, given = fresh(), [torch.empty_like(t) for t in rounds[0]], [torch.empty_like(t) for t in rounds[0]]
    ws = torch.empty(planner.attention_kv8_workspace(pool.cache), dtype=torch.uint8, device="cuda")
    got = buffers()
    codes = [t.clone() for t in (pool.k, pool.v, pool.ks, pool.vs)]
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for t, s in zip((pool.k, pool.v, pool.ks, pool.vs), codes):
            t.copy_(s)                                   # every replay begins with the same cache
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            x[0].copy_(given[0])
        for a, b in zip(x[1:], given[1:]):
            a.zero_()
            a.add_(b)
        torch.cuda.current_stream().wait_stream(other)
        steps(pool, x, *got, ws)
        for t in x:
            t.zero_()                                    # the calls are done with their inputs
    for values in rounds:
        for a, b in zip(given, values):
            a.copy_(b)
        for t in got:
            t.fill_(7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
            graph.replay()
        torch.cuda.synchronize()
        want, again = buffers(), fresh()
        steps(again, values, *want, ws)
        planner.sync_check()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("longest,page", [(2000, 64), (100, 16)])
def test_attention_of_a_mostly_empty_batch(planner, longest, page):
    lens = [0] * 300
    for at, n in ((3, 1), (60, longest), (61, 17), (299, longest // 2)):
        lens[at] = n
    pool = Pool(lens, 2, page, 128)
    ref = pool.fill(lens, 5)
    check_attention(planner, pool, ref, lens, 1, 4, True, seed=4)
    check_attention(planner, pool, ref, lens, 2, 16, False, seed=5)
    check_attention(planner, pool, ref, [0] * 300, 1, 4, True, seed=6)


def test_misaligned_offsets_are_refused(planner):
    pool, lib, h = Pool([32], 2, 16, 64), planner.lib, planner.h
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    n = torch.zeros(8, dtype=torch.int32, device="cuda")
    ws = torch.empty(planner.attention_kv8_workspace(pool.cache), dtype=torch.uint8, device="cuda")
    p, good, odd, ref = x.data_ptr(), n.data_ptr(), n.data_ptr() + 2, pool.cache.ref
    for a, b in ((odd, good), (good, odd)):
        assert lib.jepa_kv8_read(h, ref, a, b, 4, y.data_ptr(), z.data_ptr(), None) == 1
        assert lib.jepa_rope_append_kv8(h, ref, None, 0, p, 128, p, 128, 4, 0, None, None, 0.0, None, 0, 0, 0, a, b,
                                        None, None, None) == 1
        assert lib.jepa_attention_packed(h, p, 128, p, 128, p, 128, 4, 4, 1, 2, 2, 64, a, b, 0.1, 1, y.data_ptr(),
                                         None, None) == 1
    assert lib.jepa_attention_kv8(h, ref, p, 1, 2, odd, 0.1, 1, y.data_ptr(), None, ws.data_ptr(), ws.numel(),
                                  None) == 1
    planner.sync_check()
