"""The 4-bit paged cache on the GPU: append (norm, rotation, quantisation), read-back, attention over it
and the weights that its tokens receive, against the oracle.

Tolerances, derived before the first run.
  * What decides a code is defined in fp32 operation by operation, and every code and scale
    is compared for equality. Two places allow otherwise: the norm's factor is rounded from 64 bits
    by the oracle and from two floats by the kernel (they differ where 64 bits lie within 2^-40 of a tie, about once in
    10^5 rows), so rows with a norm may differ by a code in one row of a test.
  * k_out: bf16 of those fp32 values: half a step. q_out: as the 8-bit cache's queries, 16 * 2^-24 (|a| + |b|)
    beside that, where |a| + |b| <= 2 sqrt(2) times the row's largest rotated element: 48 * 2^-24 of it.
  * Attention and lse: as derived in test_gpu_kv8.py (the same products, probabilities and sums; 4-bit codes
    times their scale are exact in f16).
  * A weight exp(s - lse): the score's and lse's errors and the exponential's, relative. The sum of R of
    them adds R 2^-23, the decayed part 2 * 2^-24."""
import numpy as np
import pytest
import torch

from oracle import four_bit, paged
from test_gpu_kv8 import BF16, attention_tolerance, bf16, cu_of, f64, i32, lse_tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def planner():
    from cem_search_transformer_gb300 import binding, synthetic
    p = binding.Planner(synthetic.PRESETS["small"])
    yield p
    p.close()


class Pool4:
    """A cache whose pages hold NaN scales until something is written."""

    def __init__(self, lens, heads, page, dim, spare=2, seed=0, units=True, room=0):
        from cem_search_transformer_gb300 import binding
        rng = np.random.default_rng(seed)
        need = [-(-int(n + room) // page) for n in lens]
        self.pages, self.page, self.heads, self.dim = sum(need) + spare, page, heads, dim
        order = rng.permutation(self.pages)
        self.table_np = np.full((len(lens), max(1, max(need))), -1, np.int64)
        at = 0
        for s, n in enumerate(need):
            self.table_np[s, :n] = order[at:at + n]
            at += n
        self.spare = order[at:]
        u8 = lambda n, fill: torch.full((self.pages, heads, page, n), fill, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.k, self.v, self.ks, self.vs = u8(dim // 2, 0x77), u8(dim // 2, 0xff), u8(dim // 16, 0x7f), u8(dim // 16, 0xff)
        self.table = i32(self.table_np)
        self.unit_np = [2.0 ** rng.integers(-4, 3, heads) if units else np.ones(heads) for _ in range(2)]
        self.units = [torch.tensor(u, dtype=torch.float32, device="cuda") if units else None for u in self.unit_np]
        self.cache = binding.KvCache4(self.k, self.v, self.ks, self.vs, self.table, *self.units)

    def fill(self, lens, seed, spread=1):
        """Random codes and scales for the first lens[s] tokens of each sequence; returns their
        values [n, heads, dim] (k, v) by sequence."""
        rng = np.random.default_rng(seed)
        host = [t.cpu().numpy() for t in (self.k, self.v, self.ks, self.vs)]
        out = []
        for s, n in enumerate(lens):
            vals = []
            for kind in (0, 1):
                x = rng.standard_normal((n, self.heads, self.dim)) * np.exp(spread * rng.standard_normal((n, self.heads, 1)))
                c, sc = four_bit.quantise(x.astype(np.float32), self.unit_np[kind][None, :, None])
                vals.append(four_bit.values(c, sc, self.unit_np[kind][None, :, None]))
                code = np.abs(c[..., None] - np.concatenate([four_bit.E2M1, -four_bit.E2M1])).argmin(-1)
                code = code.astype(np.uint8)
                sbytes = torch.from_numpy(sc.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
                for i in range(-(-n // self.page)):
                    rows = slice(i * self.page, min(n, (i + 1) * self.page))
                    m, pg = rows.stop - rows.start, int(self.table_np[s, i])
                    part = code[rows].transpose(1, 0, 2)
                    host[kind][pg, :, :m] = part[..., 0::2] | part[..., 1::2] << 4
                    host[2 + kind][pg, :, :m] = sbytes[rows].transpose(1, 0, 2)
            out.append(tuple(vals))
        for dst, src in zip((self.k, self.v, self.ks, self.vs), host):
            dst.copy_(torch.from_numpy(src))
        return out

    def held(self, s, n):
        """(code values, scales) of k and of v of sequence s's first n tokens."""
        got = []
        for codes, scales in ((self.k, self.ks), (self.v, self.vs)):
            pgs = self.table_np[s, :-(-n // self.page)]
            c = four_bit.unpack(codes[pgs].cpu().numpy()).transpose(0, 2, 1, 3).reshape(len(pgs) * self.page, self.heads, self.dim)[:n]
            sc = scales[pgs].view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64)
            got += [c, sc.transpose(0, 2, 1, 3).reshape(len(pgs) * self.page, self.heads, self.dim // 16)[:n]]
        return got


# ---- append and read ----

def same_codes(got, want, rows_that_may_differ):
    off = (got != want) & ~(np.isnan(got) & np.isnan(want))
    rows = off.reshape(-1, off.shape[-1]).any(-1).sum()
    assert rows <= rows_that_may_differ, (rows, np.argwhere(off)[:4])


def check_append(planner, new, old, q_heads, kv_heads, dim, page, rot, interleaved, norm, seed, units=True):
    rng = np.random.default_rng(seed)
    lens = [a + b for a, b in zip(new, old)]
    pool = Pool4(lens, kv_heads, page, dim, seed=seed, units=units)
    before = pool.fill(old, seed + 1)
    kept = [pool.held(s, n) for s, n in enumerate(old)]
    total = sum(new)
    qkv = bf16(rng.standard_normal((total, q_heads + 2 * kv_heads, dim)) * np.exp(rng.standard_normal((total, q_heads + 2 * kv_heads, 1)))).cuda()
    q, k, v = qkv[:, :q_heads], qkv[:, q_heads:q_heads + kv_heads], qkv[:, q_heads + kv_heads:]
    wq, wk = ((torch.rand(dim, device="cuda") + 0.5) for _ in range(2)) if norm else (None, None)
    table = planner.rope_table(max(lens) + 1, rot) if rot else None
    q_out = torch.full((total, q_heads, dim), 9.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((total, kv_heads, dim), 9.0, dtype=torch.bfloat16, device="cuda")
    planner.rope_append_kv4(q, k, v, table, cu_of(new), i32(old), pool.cache, q_out, q_norm=wq, k_norm=wk,
                            interleaved=interleaved, k_out=k_out)
    k_read = torch.full((sum(lens), kv_heads, dim), 9.0, dtype=torch.bfloat16, device="cuda")
    v_read = torch.full_like(k_read, 9.0)
    planner.kv4_read(pool.cache, cu_of(lens), i32([0] * len(lens)), k_read, v_read)
    planner.sync_check()
    pos = np.concatenate([np.arange(o, o + n) for n, o in zip(new, old)]).astype(np.int64)
    tab = None if table is None else table.cpu().numpy()
    w = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    slack = 1 if norm else 0
    want_q = four_bit.norm_rotate(f64(q), w(wq), tab, pos, interleaved)
    want_k = four_bit.norm_rotate(f64(k), w(wk), tab, pos, interleaved)
    assert np.all(np.abs(f64(k_out) - want_k) <= (BF16 + slack * 2.0 ** -23) * np.abs(want_k) + slack * 2.0 ** -22)
    most = np.abs(want_q).max(-1, keepdims=True)
    assert np.all(np.abs(f64(q_out) - want_q) <= BF16 * np.abs(want_q) + 48 * 2.0 ** -24 * most)
    at = read = 0
    for s, (n, o) in enumerate(zip(new, old)):
        ck, sk, cv, sv = pool.held(s, n + o)
        for (codes, scales), first in (((ck, sk), 0), ((cv, sv), 2)):
            assert np.array_equal(codes[:o], kept[s][first]) and np.array_equal(scales[:o], kept[s][first + 1])
        for codes, scales, x, unit, may in ((ck, sk, want_k[at:at + n], pool.unit_np[0], slack),
                                            (cv, sv, f64(v)[at:at + n], pool.unit_np[1], 0)):
            c, sc = four_bit.quantise(x, unit[None, :, None])
            same_codes(scales[o:], sc, may)
            same_codes(codes[o:] * 1.0, c, may)
        for codes, scales, unit, out in ((ck, sk, pool.unit_np[0], k_read), (cv, sv, pool.unit_np[1], v_read)):
            assert np.array_equal(f64(out)[read:read + n + o], four_bit.values(codes, scales, unit[None, :, None]))
        at += n
        read += n + o
    del before


@pytest.mark.parametrize("new,old,q_heads,kv_heads,dim,page,rot,interleaved,norm", [
    ([1], [0], 1, 1, 64, 16, 16, False, False),
    ([1], [300], 16, 16, 64, 16, 32, True, False),
    ([1, 1, 1], [15, 16, 0], 9, 9, 128, 16, 128, False, True),     # more heads than a warp takes
    ([3, 0, 5], [7, 0, 130], 6, 2, 128, 64, 48, False, True),      # an odd number of rotating lanes
    ([40, 1, 70], [0, 63, 64], 4, 1, 64, 32, 48, False, False),
    ([258, 17], [258, 0], 10, 10, 64, 128, 64, True, True),
    ([130, 33], [3, 9], 3, 3, 128, 128, 112, True, True),
    ([65], [0], 8, 8, 128, 64, 80, False, False),
    ([5, 9], [2, 0], 2, 2, 64, 16, 0, False, True),                # no rotation
])
@pytest.mark.parametrize("units", [True, False])
def test_append_matches_oracle(planner, new, old, q_heads, kv_heads, dim, page, rot, interleaved, norm, units):
    check_append(planner, new, old, q_heads, kv_heads, dim, page, rot, interleaved, norm, seed=sum(new) + dim, units=units)


def test_blocks_that_are_not_finite_zeros_and_ends_of_the_scale(planner):
    pool = Pool4([9], 2, 16, 64)
    rng = np.random.default_rng(3)
    x = rng.standard_normal((9, 2, 64))
    x[0, 0, 5], x[1, 1, 40], x[2, 0, 63] = np.nan, np.inf, -np.inf
    x[3] = 0
    x[4], x[5], x[6] = x[4] * 1e-8, x[5] * 2.0 ** 14, 2.0 ** 60
    x[7] = 3 * 2.0 ** -10 * pool.unit_np[1][:, None]               # the least scale: 1.5 codes
    x[8, :, ::16] = 5.0
    x[8, :, 1::16] = 2.5                                            # ties of 6 at half the block's scale
    t = bf16(x).cuda()
    k_read, v_read = torch.empty_like(t), torch.empty_like(t)
    planner.rope_append_kv4(None, t, t, None, cu_of([9]), i32([0]), pool.cache, None)
    planner.kv4_read(pool.cache, cu_of([9]), i32([0]), k_read, v_read)
    planner.sync_check()
    ck, sk, cv, sv = pool.held(0, 9)
    for codes, scales, unit, out in ((ck, sk, pool.unit_np[0], k_read), (cv, sv, pool.unit_np[1], v_read)):
        c, sc = four_bit.quantise(f64(t), unit[None, :, None])
        same_codes(scales, sc, 0)
        same_codes(codes, c, 0)
        assert np.array_equal(f64(out), four_bit.values(c, sc, unit[None, :, None]), equal_nan=True)


def test_in_place_and_again(planner):
    rng = np.random.default_rng(5)
    n, page, dim = [70, 3], 32, 128
    rows = [bf16(rng.standard_normal((73, h, dim))).cuda() for h in (4, 2, 2)]
    table = planner.rope_table(100, dim)
    pools = [Pool4(n, 2, page, dim, seed=1) for _ in range(2)]
    q_out, k_out = torch.empty_like(rows[0]), torch.empty_like(rows[1])
    for _ in range(2):
        planner.rope_append_kv4(*rows, table, cu_of(n), i32([0, 0]), pools[0].cache, q_out, k_out=k_out)
    q, k = rows[0].clone(), rows[1].clone()
    planner.rope_append_kv4(q, k, rows[2], table, cu_of(n), i32([0, 0]), pools[1].cache, q, k_out=k)
    planner.sync_check()
    assert torch.equal(q, q_out) and torch.equal(k, k_out)
    for a, b in ((pools[0].k, pools[1].k), (pools[0].ks, pools[1].ks), (pools[0].v, pools[1].v), (pools[0].vs, pools[1].vs)):
        assert torch.equal(a, b)


def test_positions_apart_from_places(planner):
    """rope_start: tokens are rotated for other positions than their places, which may lie behind the table's end."""
    from cem_search_transformer_gb300 import binding
    n, old, at, page, dim = [3, 0, 70], [60, 5, 0], [900, 7, 130], 32, 128
    lens = [a + b for a, b in zip(n, old)]
    rng = np.random.default_rng(4)
    rows = [bf16(rng.standard_normal((73, h, dim))).cuda() for h in (4, 2, 2)]
    table = planner.rope_table(1000, 64)
    got = []
    for first, apart in ((old, at), (at, None)):
        pool = Pool4([a + b for a, b in zip(n, first)], 2, page, dim, seed=1)
        q_out, k_out = torch.empty_like(rows[0]), torch.empty_like(rows[1])
        planner.rope_append_kv4(*rows, table, cu_of(n), i32(first), pool.cache, q_out, k_out=k_out, interleaved=True,
                                rope_start=None if apart is None else i32(apart))
        k_read, v_read = torch.empty_like(rows[1]), torch.empty_like(rows[2])
        planner.kv4_read(pool.cache, cu_of(n), i32(first), k_read, v_read)
        planner.sync_check()
        got.append((q_out, k_out, k_read, v_read))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    pool = Pool4(lens, 2, page, dim, seed=1)
    short = planner.rope_table(40, 64)                                # places may pass the table's end, positions may not
    q_out = torch.full_like(rows[0], 5.0)
    planner.rope_append_kv4(*rows, short, cu_of(n), i32(old), pool.cache, q_out, rope_start=i32([37, 0, 38]))
    with pytest.raises(binding.JepaError, match="outside"):
        planner.sync_check()
    assert not torch.any(torch.all(q_out[:5].reshape(5, -1) == 5.0, 1)) and torch.all(q_out[5:] == 5.0)
    planner.rope_append_kv4(*rows, short, cu_of(n), i32(old), pool.cache, q_out, rope_start=i32([-1, 0, 2 ** 31 - 3]))
    with pytest.raises(binding.JepaError, match="outside"):
        planner.sync_check()
    with pytest.raises(binding.JepaError, match="elements"):
        planner.rope_append_kv4(*rows, short, cu_of(n), i32(old), pool.cache, q_out, rope_start=i32([0, 0]))
    u8 = torch.zeros(8, 2, 32, 128, dtype=torch.uint8, device="cuda")
    ones = torch.ones(8, 2, device="cuda")
    eight = binding.KvCache8(u8, u8.clone(), ones, ones.clone(), i32(np.arange(9).reshape(3, 3) % 8))
    with pytest.raises(binding.JepaError, match="rope_start"):
        planner.rope_append_kv8(*rows, short, cu_of(n), i32(old), eight, q_out, rope_start=i32(old))


def test_bad_pages_positions_and_offsets_are_skipped_and_reported(planner):
    from cem_search_transformer_gb300 import binding
    n, page, dim = [20, 20, 20, 20], 16, 64
    x = bf16(np.random.default_rng(6).standard_normal((80, 2, dim))).cuda()
    good = Pool4(n, 2, page, dim, seed=2)
    planner.rope_append_kv4(None, x, x, None, cu_of(n), i32([0] * 4), good.cache, None)
    planner.sync_check()
    for change in ("page", "start", "table", "cu", "behind"):
        pool = Pool4(n, 2, page, dim, seed=2)
        start, cu, table, rows = i32([0] * 4), cu_of(n), None, x
        if change == "page":
            pool.table[1] = pool.pages
        elif change == "start":
            start[1] = -3
        elif change == "table":                                      # positions past the rotary table
            table, start = planner.rope_table(20, 16), i32([0, 10 ** 9, 0, 0])
        elif change == "cu":                                         # sequences 1 and 2 share tokens, 3 owns none
            cu = i32([0, 20, 70, 60, 60])
        else:
            cu = i32([0, 20, 81, 90, 100])
        before = [t.clone() for t in (pool.k, pool.ks)]
        q_out = torch.full_like(rows, 5.0)
        planner.rope_append_kv4(rows if change == "table" else None, rows, rows, table, cu, start, pool.cache,
                                q_out if change == "table" else None)
        with pytest.raises(binding.JepaError, match="outside"):
            planner.sync_check()
        planner.sync_check()
        pg = pool.table_np[0]
        if change != "table":
            assert torch.equal(pool.k[pg, :, :4], good.k[pg, :, :4])             # the sequence ahead is there
        if change == "table":
            assert torch.all(q_out[20:40] == 5.0) and not torch.any(q_out[:20] == 5.0)
        if change == "behind":
            pgs = np.concatenate([pool.table_np[s] for s in (1, 2, 3)])
            for t, b in zip((pool.k, pool.ks), before):
                assert torch.equal(t[pgs], b[pgs])
        out = torch.full((80, 2, dim), 5.0, dtype=torch.bfloat16, device="cuda")
        planner.kv4_read(pool.cache, cu, start, out, out.clone())
        if change in ("page", "start", "table", "cu", "behind"):
            with pytest.raises(binding.JepaError, match="outside"):
                planner.sync_check()


def test_rows_ahead_of_the_first_sequence_and_behind_the_last_are_left(planner):
    cu, old = [7, 7, 30, 64], [3, 0, 40]
    n = np.diff(cu)
    pool = Pool4([a + b for a, b in zip(n, old)], 3, 32, 64, seed=1)
    rng = np.random.default_rng(1)
    q, k, v = (bf16(rng.standard_normal((80, h, 64))).cuda() for h in (6, 3, 3))
    q_out, k_out, k_read, v_read = (torch.full_like(t, 5.0) for t in (q, k, k, v))
    planner.rope_append_kv4(q, k, v, None, i32(cu), i32(old), pool.cache, q_out, k_out=k_out)
    planner.kv4_read(pool.cache, i32(cu), i32(old), k_read, v_read)
    planner.sync_check()
    for t in (q_out, k_out, k_read, v_read):
        assert torch.all(t[:7] == 5.0) and torch.all(t[64:] == 5.0)
    assert torch.equal(q_out[7:64], q[7:64]) and torch.equal(k_out[7:64], k[7:64])
    for got, rows, unit in ((k_read, k, pool.unit_np[0]), (v_read, v, pool.unit_np[1])):
        want = four_bit.values(*four_bit.quantise(f64(rows), unit[None, :, None]), unit[None, :, None])
        assert np.array_equal(f64(got)[7:64], want[7:64])


# ---- attention and weights ----

def weights_of(q, k, lim, scale):
    """[q_heads' rows summed per key / value head][n] and the same sum of weight * |score|'s bound."""
    n, hq, d = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    out = np.zeros((hkv, k.shape[0]))
    for h in range(hq):
        s = q[:, h] @ k[:, h // g].T * scale
        for i in range(n):
            m = int(lim[i])
            if m > 0:
                p = np.exp(s[i, :m] - s[i, :m].max())
                out[h // g, :m] += p / p.sum()
    return out


def check_attention(planner, pool, ref, lens, q_tokens, q_heads, causal, seed, scale=None, weights=True, q=None):
    rng = np.random.default_rng(seed)
    dim, heads = pool.dim, pool.heads
    scale = dim ** -0.5 if scale is None else scale
    if q is None:
        q = bf16(rng.standard_normal((len(lens), q_tokens, q_heads, dim))).cuda()
    out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:3], 9.0, device="cuda")
    ws = torch.empty(planner.attention_kv4_workspace(pool.cache), dtype=torch.uint8, device="cuda")
    reach = pool.table.shape[1] * pool.page
    mass = torch.rand(len(lens), heads, reach, device="cuda") if weights else None
    mass_out = torch.full((len(lens), heads, reach), 9.0, device="cuda") if weights else None
    planner.attention_kv4(q, pool.cache, i32(lens), out, scale, ws, causal=causal, lse=lse, mass=mass,
                          mass_out=mass_out, decay=0.75)
    planner.sync_check()
    for s, n in enumerate(lens):
        k, v = (x[:n] for x in ref[s])
        lim = [max(0, n - q_tokens + t + 1) if causal else n for t in range(q_tokens)]
        want, want_lse, a, s_abs = paged.softmax_rows(f64(q[s]), k, v, lim, scale)
        got, got_lse = f64(out[s]), f64(lse[s])
        assert np.all(np.isfinite(got)), s
        assert np.all(np.abs(got - want) <= attention_tolerance(want, a, s_abs, n, dim, np.abs(v).max() if n else 0)), \
            (s, np.abs(got - want).max())
        empty = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(got_lse), empty)
        tol = lse_tolerance(s_abs, n, dim, want_lse)
        assert np.all(np.abs(got_lse[~empty] - want_lse[~empty]) <= tol[~empty])
        if weights:
            m = f64(mass_out[s])
            w = weights_of(f64(q[s]), k, lim, scale)
            rows = q_tokens * q_heads // heads
            rel = 2 * (dim * 2.0 ** -22 * s_abs.max() + tol[~empty].max() if n and (~empty).any() else 0) + 2.0 ** -20 + rows * 2.0 ** -23
            old = 0.75 * f64(mass[s])[:, :n]
            assert np.all(np.abs(m[:, :n] - old - w) <= rel * w + 2.0 ** -23 * (old + w)), (s, np.abs(m[:, :n] - old - w).max())
            assert np.all(m[:, n:] == 9.0)
    return out, lse, mass_out


@pytest.mark.parametrize("lens,q_tokens,q_heads,kv_heads,dim,page,causal", [
    ([1], 1, 1, 1, 64, 16, True),
    ([0], 1, 2, 1, 128, 16, True),                        # nothing cached
    ([5, 0, 1, 64], 1, 4, 2, 128, 32, True),
    ([31, 32, 33, 127, 128, 129], 1, 8, 1, 128, 64, True),  # around a step and a unit
    ([127, 128, 129, 257], 1, 3, 3, 64, 16, True),
    ([517], 1, 16, 16, 64, 32, True),
    ([2, 1, 0, 40], 4, 6, 2, 128, 16, True),              # rows that see nothing
    ([300, 17], 8, 14, 2, 64, 128, True),                 # 56 rows: four tiles
    ([70, 33], 3, 5, 1, 128, 32, False),
    ([300, 9], 2, 8, 1, 128, 64, True),                   # 16 rows
    ([776, 776, 12], 2, 4, 4, 64, 16, False),
    ([6000, 11, 2049], 1, 8, 2, 128, 128, True),          # split over many CTAs
    ([20011], 2, 7, 1, 64, 64, True),
    ([40] * 70, 1, 4, 4, 128, 16, True),                  # more sequences than a warp's scan
])
def test_attention_matches_oracle(planner, lens, q_tokens, q_heads, kv_heads, dim, page, causal):
    pool = Pool4(lens, kv_heads, page, dim, seed=len(lens))
    ref = pool.fill(lens, 7)
    check_attention(planner, pool, ref, lens, q_tokens, q_heads, causal, seed=q_heads)


def test_attention_without_units_lse_or_weights(planner):
    pool = Pool4([90], 2, 32, 64, units=False)
    ref = pool.fill([90], 3)
    out, lse, _ = check_attention(planner, pool, ref, [90], 1, 4, True, seed=2, weights=False)
    q = bf16(np.random.default_rng(2).standard_normal((1, 1, 4, 64))).cuda()
    again = torch.empty_like(q)
    ws = torch.empty(planner.attention_kv4_workspace(pool.cache), dtype=torch.uint8, device="cuda")
    planner.attention_kv4(q, pool.cache, i32([90]), again, 64 ** -0.5, ws)
    planner.sync_check()
    assert torch.equal(again, out)


@pytest.mark.parametrize("dim", [64, 128])
def test_magnitudes_far_apart(planner, dim):
    """Tokens whose scales differ by up to 2^17, units from 2^-40 to 2^40, and large scores."""
    lens = [700, 400]
    pool = Pool4(lens, 2, 16, dim)
    ref = pool.fill(lens, 3, spread=3)
    check_attention(planner, pool, ref, lens, 1, 4, True, seed=1, scale=0.01)
    for unit in (2.0 ** -40, 2.0 ** 40):
        pool.units[1].fill_(unit)
        far = [(k, v / pool.unit_np[1][None, :, None] * unit) for k, v in ref]
        check_attention(planner, pool, far, lens, 2, 4, True, seed=2, scale=0.001)


def test_weights_in_place_and_from_nothing(planner):
    lens = [100, 333]
    pool = Pool4(lens, 2, 64, 128)
    ref = pool.fill(lens, 4)
    q = bf16(np.random.default_rng(9).standard_normal((2, 1, 4, 128))).cuda()
    out, lse, mass_out = check_attention(planner, pool, ref, lens, 1, 4, True, seed=0, q=q)
    ws = torch.empty(planner.attention_kv4_workspace(pool.cache), dtype=torch.uint8, device="cuda")
    call = lambda **kw: planner.attention_kv4(q, pool.cache, i32(lens), out, 128 ** -0.5, ws, lse=lse, **kw)  # noqa: E731
    fresh, sums = torch.full_like(mass_out, 7.0), torch.zeros_like(mass_out)
    call(mass_out=fresh)
    for _ in range(3):
        call(mass=sums, mass_out=sums)
    planner.sync_check()
    for s, n in enumerate(lens):
        w = f64(fresh[s, :, :n])
        assert np.all(fresh[s, :, n:].cpu().numpy() == 7.0) and not sums[s, :, n:].any()
        assert np.all(np.abs(f64(sums[s, :, :n]) - 3 * w) <= 4 * 2.0 ** -24 * 3 * w)
        assert abs(w.sum() - 4) <= 4 * n * 2.0 ** -20                # two heads a group: each row sums to 1


@pytest.mark.parametrize("dim", [64, 128])
def test_unseen_keys_do_not_reach_a_query(planner, dim):
    """NaN scales in the newest tokens: queries before them are untouched, those that see them become NaN
    (values) in just those blocks; their weights stay numbers."""
    lens, tq, page = [75, 40], 4, 16
    pool = Pool4(lens, 1, page, dim)
    ref = pool.fill(lens, 2)
    q = bf16(np.random.default_rng(5).standard_normal((2, tq, 2, dim))).cuda()
    clean, _, clean_mass = check_attention(planner, pool, ref, lens, tq, 2, True, seed=5, q=q)
    n = lens[0]
    pg, off = int(pool.table_np[0, (n - 2) // page]), (n - 2) % page
    pool.vs[pg, 0, off, 1], pool.vs[pg, 0, off, dim // 16 - 1] = 0x7f, 0xff
    out, lse = torch.empty_like(q), torch.empty(2, tq, 2, device="cuda")
    mass = torch.zeros_like(clean_mass)
    ws = torch.empty(planner.attention_kv4_workspace(pool.cache), dtype=torch.uint8, device="cuda")
    call = lambda: planner.attention_kv4(q, pool.cache, i32(lens), out, dim ** -0.5, ws, lse=lse, mass_out=mass)  # noqa: E731
    call()
    planner.sync_check()
    assert torch.equal(out[0, :2], clean[0, :2]) and torch.equal(out[1], clean[1])
    bad = torch.zeros(dim, dtype=torch.bool, device="cuda")
    bad[16:32] = bad[dim - 16:] = True
    assert torch.all(torch.isnan(out[0, 2:][..., bad]))
    assert torch.equal(out[0, 2:][..., ~bad], clean[0, 2:][..., ~bad])
    assert torch.isfinite(mass[0, 0, :n]).all()
    pg, off = int(pool.table_np[0, (n - 1) // page]), (n - 1) % page
    pool.ks[pg, 0, off, 0] = 0x7f                            # the newest key: only the last query sees it
    call()
    planner.sync_check()
    assert torch.equal(out[0, :2], clean[0, :2]) and torch.all(torch.isnan(out[0, 3]))
    assert torch.equal(out[1], clean[1]) and torch.isfinite(mass[1, 0, :40]).all()


def test_nan_queries_stay_in_their_row(planner):
    pool = Pool4([90], 1, 32, 128)
    ref = pool.fill([90], 2)
    clean, _, _ = check_attention(planner, pool, ref, [90], 1, 4, True, seed=5)
    q = bf16(np.random.default_rng(5).standard_normal((1, 1, 4, 128))).cuda()
    q[0, 0, 1, 7] = float("nan")
    out, lse = torch.empty_like(q), torch.zeros(1, 1, 4, device="cuda")
    ws = torch.empty(planner.attention_kv4_workspace(pool.cache), dtype=torch.uint8, device="cuda")
    planner.attention_kv4(q, pool.cache, i32([90]), out, 128 ** -0.5, ws, lse=lse)
    planner.sync_check()
    assert torch.all(torch.isnan(out[0, 0, 1])) and torch.isnan(lse[0, 0, 1])
    assert torch.equal(out[0, 0, [0, 2, 3]], clean[0, 0, [0, 2, 3]])


def test_bad_lengths_and_pages_are_reported(planner):
    from cem_search_transformer_gb300 import binding
    pool = Pool4([64, 64], 2, 32, 64)
    ref = pool.fill([64, 64], 4)
    want, _, mass = check_attention(planner, pool, ref, [64, 64], 1, 4, True, seed=1)
    q = bf16(np.random.default_rng(1).standard_normal((2, 1, 4, 64))).cuda()
    ws = torch.empty(planner.attention_kv4_workspace(pool.cache), dtype=torch.uint8, device="cuda")
    for lens, same in (([65, 64], [0, 1]), ([64, -1], [0])):        # clamped to what the table names, or to 0
        out, lse = torch.empty_like(q), torch.empty(2, 1, 4, device="cuda")
        planner.attention_kv4(q, pool.cache, i32(lens), out, 0.125, ws, lse=lse, mass_out=torch.empty_like(mass))
        with pytest.raises(binding.JepaError, match="outside"):
            planner.sync_check()
        assert all(torch.equal(out[s], want[s]) for s in same)
    pool.table[1, 1] = pool.pages + 7
    out = torch.empty_like(q)
    planner.attention_kv4(q, pool.cache, i32([64, 64]), out, 0.125, ws)
    with pytest.raises(binding.JepaError, match="outside"):
        planner.sync_check()
    assert torch.equal(out[0], want[0]) and torch.isfinite(out[1]).all()


def test_graph_replay_reads_lengths_anew_and_streams_run_apart(planner):
    lens, page, dim = [3000, 50], 64, 128
    pool = Pool4(lens, 2, page, dim)
    pool.fill(lens, 8)
    q = bf16(np.random.default_rng(11).standard_normal((2, 1, 8, dim))).cuda()
    need = planner.attention_kv4_workspace(pool.cache)
    kv_len, reach = i32(lens), pool.table.shape[1] * page

    def buffers():
        return (torch.empty_like(q), torch.empty(2, 1, 8, device="cuda"), torch.zeros(2, 2, reach, device="cuda"),
                torch.empty(need, dtype=torch.uint8, device="cuda"))

    def call(n, out, lse, mass, ws, stream=None):
        planner.attention_kv4(q, pool.cache, n, out, 0.09, ws, lse=lse, mass_out=mass, stream=stream)

    def direct(n):
        got = buffers()
        call(i32(n), *got)
        planner.sync_check()
        return got[:3]
    cases = [[3000, 50], [64, 0], [2999, 1]]
    want = [direct(n) for n in cases]
    calls = []
    for _ in range(2):
        got = buffers()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got[2].zero_()
            call(kv_len, *got, stream=torch.cuda.current_stream())
        calls.append((graph, got, side))
    for n, w in zip(cases, want):
        kv_len.copy_(i32(n))
        torch.cuda.synchronize()
        for graph, _, side in calls:
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for _, got, _ in calls:
            for a, b in zip(got[:3], w):
                assert torch.equal(a, b)
    for _ in range(3):                                       # no order of CTAs enters the result
        for a, b in zip(direct(cases[0]), want[0]):
            assert torch.equal(a, b)
    planner.sync_check()
    calls.clear()


def test_refusals(planner):
    from cem_search_transformer_gb300 import binding, synthetic
    pool = Pool4([32], 2, 16, 64)
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    n = planner.attention_kv4_workspace(pool.cache)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    lse, mass = torch.empty(1, 1, 4, device="cuda"), torch.zeros(1, 2, 32, device="cuda")
    ok = dict(q=q, cache=pool.cache, kv_len=i32([3]), out=torch.empty_like(q), scale=0.1, workspace=ws)
    for change, match in ((dict(scale=0.0), "bad argument"), (dict(scale=float("nan")), "bad argument"),
                          (dict(workspace=ws[:n - 1]), "too small"), (dict(workspace=ws[1:]), "bad argument"),
                          (dict(q=q[:, :, :3].contiguous()), "bad argument"),       # 3 heads over 2
                          (dict(out=q[:, :, :2].contiguous()), "elements"),
                          (dict(mass_out=mass), "lse"), (dict(mass=mass, lse=lse), "mass_out"),
                          (dict(mass_out=mass, lse=lse, decay=float("inf")), "decay"),
                          (dict(mass_out=mass[:, :, :31].contiguous(), lse=lse), "elements")):
        with pytest.raises(binding.JepaError, match=match):
            planner.attention_kv4(**{**ok, **change})
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    for table in (torch.zeros(8, 24, device="cuda"), torch.zeros(8, 80, device="cuda")):
        with pytest.raises(binding.JepaError, match="rotary"):
            planner.rope_append_kv4(None, x, x, table, cu_of([3]), i32([0]), pool.cache, None)
    with pytest.raises(binding.JepaError, match="together"):
        planner.rope_append_kv4(x, x, x, None, cu_of([3]), i32([0]), pool.cache, None)
    with pytest.raises(binding.JepaError, match="fit"):
        planner.rope_append_kv4(None, x[:, :1], x[:, :1], None, cu_of([3]), i32([0]), pool.cache, None)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    odd = u8(2 * 2 * 16 * 4 + 4)[4:].view(2, 2, 16, 4)              # scales 4 bytes off
    c = binding.KvCache4(u8(2, 2, 16, 32), u8(2, 2, 16, 32), odd, u8(2, 2, 16, 4), i32([[0, 1]]))
    with pytest.raises(binding.JepaError, match="misaligned"):
        planner.attention_kv4_workspace(c)
    fp32 = binding.Planner(synthetic.PRESETS["tiny"])
    with pytest.raises(binding.JepaError, match="bf16 context"):
        fp32.attention_kv4(**ok)
    fp32.close()
    planner.sync_check()


@pytest.mark.parametrize("dim,q_tokens,group,heads", [(128, 1, 4, 8), (64, 2, 1, 16), (128, 2, 8, 4), (64, 3, 5, 6)])
def test_short_sequences_a_warp_each(planner, dim, q_tokens, group, heads):
    """As many (sequence, head) items of at most a few hundred tokens as the machine has warps: 3 or 4 CTAs a SM with four
    warps, one fewer where a head has more than 8 query rows."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    slots = sms * 4 * ((4 if dim == 64 else 3) - (q_tokens * group > 8))
    tiles = -(-q_tokens * group // (16 if q_tokens * group > 8 else 8))
    batch = slots // (heads * tiles)
    rng = np.random.default_rng(dim)
    lens = [int(n) for n in rng.integers(0, 40, batch)]
    lens[0], lens[1], lens[2] = 300, 0, 257
    pool = Pool4(lens, heads, 16, dim)
    ref = pool.fill(lens, 3)
    check_attention(planner, pool, ref, lens, q_tokens, heads * group, q_tokens != 2, seed=1)


def test_thousands_of_sequences_most_of_them_empty(planner):
    lens = [0] * 3000
    for s, n in ((0, 3), (17, 2500), (1031, 70), (2999, 129)):
        lens[s] = n
    pool = Pool4(lens, 2, 64, 64)
    ref = pool.fill(lens, 6)
    check_attention(planner, pool, ref, lens, 1, 8, True, seed=3)


def test_offsets_past_32_bits(planner):
    """Pools of more than 2^32 bytes of codes: the same tokens at the first and at the last pages."""
    from cem_search_transformer_gb300 import binding
    heads, page, dim, n = 8, 128, 128, 300
    pages = 2 ** 32 // (heads * page * dim // 2) + 9
    u8 = lambda k: torch.empty(pages, heads, page, k, dtype=torch.uint8, device="cuda")  # noqa: E731
    pools = u8(dim // 2), u8(dim // 2), u8(dim // 16), u8(dim // 16)
    rows = bf16(np.random.default_rng(2).standard_normal((n, heads, dim))).cuda()
    q = bf16(np.random.default_rng(3).standard_normal((1, 1, 16, dim))).cuda()
    got = []
    for first in (0, pages - 3):
        table = i32([[first, first + 1, first + 2]])
        cache = binding.KvCache4(*pools, table)
        planner.rope_append_kv4(None, rows, rows, None, cu_of([n]), i32([0]), cache, None)
        k, v = torch.empty_like(rows), torch.empty_like(rows)
        planner.kv4_read(cache, cu_of([n]), i32([0]), k, v)
        out, lse, mass = torch.empty_like(q), torch.empty(1, 1, 16, device="cuda"), torch.zeros(1, heads, 3 * page, device="cuda")
        ws = torch.empty(planner.attention_kv4_workspace(cache), dtype=torch.uint8, device="cuda")
        planner.attention_kv4(q, cache, i32([n]), out, 0.1, ws, lse=lse, mass_out=mass)
        to = binding.KvCache4(*pools, i32([[pages - 5 if first else 4]]))
        keep, new_len = torch.empty(1, heads, page, device="cuda"), i32([0])
        work = torch.empty(planner.kv4_evict_workspace(cache, 100), dtype=torch.uint8, device="cuda")
        planner.kv4_evict(cache, i32([n]), mass, 100, 10, to, new_len, keep, work)
        kept = torch.empty(100, heads, dim, dtype=torch.bfloat16, device="cuda")
        planner.kv4_read(to, cu_of([100]), i32([0]), kept, torch.empty_like(kept))
        planner.sync_check()
        got.append((k, v, out, lse, mass, keep, kept))
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n_new", [[1, 1, 1], [700, 3, 1500]])
def test_captured_append_attention_and_read(planner, n_new):
    """One graph with torch's kernels, copies and the calls, replayed with other inputs and lengths; both shapes of the append."""
    page, dim, heads, q_heads = 32, 64, 8, 16
    old = [40, 0, 95]
    total, cu = sum(n_new), cu_of(n_new)
    lens = [a + b for a, b in zip(old, n_new)]
    rng = np.random.default_rng(21)
    rope = planner.rope_table(2048, dim)
    past = [bf16(rng.standard_normal((sum(old), heads, dim))).cuda() for _ in range(2)]
    pool = Pool4(lens, heads, page, dim, seed=5)
    planner.rope_append_kv4(None, *past, rope, cu_of(old), i32([0] * 3), pool.cache, None)
    reach = pool.table.shape[1] * page
    given = [torch.empty(total, h, dim, dtype=torch.bfloat16, device="cuda") for h in (q_heads, heads, heads)]
    start, kv_len = i32(old), i32(lens)

    def buffers():
        return [torch.empty(total, h, dim, dtype=torch.bfloat16, device="cuda") for h in (q_heads, heads, heads)] + \
            [torch.empty(3, 1, q_heads, dim, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 1, q_heads, device="cuda"),
             torch.zeros(3, heads, reach, device="cuda")]

    def steps(x, q_out, k, v, att, lse, mass, ws, stream=None):
        planner.rope_append_kv4(*x, rope, cu, start, pool.cache, q_out, stream=stream)
        planner.attention_kv4(q_out[-3:].unsqueeze(1), pool.cache, kv_len, att, 0.125, ws, lse=lse, mass=mass, mass_out=mass,
                              decay=0.5, stream=stream)
        planner.kv4_read(pool.cache, cu, start, k, v, stream=stream)
    ws = torch.empty(planner.attention_kv4_workspace(pool.cache), dtype=torch.uint8, device="cuda")
    x, got = [torch.empty_like(t) for t in given], buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for a, b in zip(x, given):
            a.zero_()
            a.add_(b)
        got[-1].zero_()
        steps(x, *got, ws, stream=torch.cuda.current_stream())
        steps(x, *got, ws, stream=torch.cuda.current_stream())        # the same tokens again: only the weights move on
        for t in x:
            t.zero_()                                                 # the calls are done with their inputs
    for seed in range(3):
        values = [bf16(np.random.default_rng(seed).standard_normal(t.shape)).cuda() for t in given]
        for a, b in zip(given, values):
            a.copy_(b)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        want = buffers()
        steps(values, *want, ws)
        steps(values, *want, ws)
        planner.sync_check()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
