"""The append to the 4-bit cache at the ends of the number range, against the oracle.

What decides a code is defined in fp32 operation by operation, so codes and scales are compared for equality
(test_gpu_kv4.py)."""
import numpy as np
import pytest
import torch

from oracle import four_bit, paged
from test_gpu_kv4 import Pool4, same_codes
from test_gpu_kv8 import bf16, cu_of, f64, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def planner():
    from cem_search_transformer_gb300 import binding, synthetic
    p = binding.Planner(synthetic.PRESETS["small"])
    yield p
    p.close()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("unit", [2.0 ** -40, 2.0 ** -12, 2.0 ** 40])
def test_elements_beyond_the_largest_scale_keep_their_sign(planner, dim, unit):
    """|x| / (scale unit) past fp32: codes saturate at 6 with the element's sign."""
    rng = np.random.default_rng(dim)
    x = rng.standard_normal((12, 2, dim))
    x[0], x[1], x[2] = 3e38 * np.sign(x[0]), 1e30 * x[1], -3e38
    x[3, :, ::16] = -1e38                                          # one to a block, among ordinary ones
    x[4, :, 5::16] = 3e38
    x[5] *= 448 * 6 * unit                                         # about the largest scale
    x[6] *= 448 * 8 * unit
    x[7:10] = np.clip(x[7:10] * unit * 2.0 ** np.array([40, 88, 120])[:, None, None], -3e38, 3e38)
    pool = Pool4([12], 2, 16, dim)
    for u, t in zip(pool.unit_np, pool.units):
        u[:] = unit
        t.fill_(unit)
    t = bf16(x).cuda()
    k_read, v_read = torch.empty_like(t), torch.empty_like(t)
    for interleaved in (False, True):
        planner.rope_append_kv4(None, t, t, None, cu_of([12]), i32([0]), pool.cache, None, interleaved=interleaved)
        planner.kv4_read(pool.cache, cu_of([12]), i32([0]), k_read, v_read)
        planner.sync_check()
        ck, sk, cv, sv = pool.held(0, 12)
        with np.errstate(over="ignore"):
            c, sc = four_bit.quantise(f64(t), np.float32(unit))
        for codes, scales, out in ((ck, sk, k_read), (cv, sv, v_read)):
            same_codes(scales, sc, 0)
            same_codes(codes, c, 0)
            assert np.array_equal(f64(out), four_bit.values(c, sc, unit))


def far_heads(rng, n, heads, dim):
    """Finite head rows whose squares, or their sum, leave fp32: above, and (with no epsilon) below."""
    x = rng.standard_normal((n, heads, dim))
    x /= np.abs(x).max(-1, keepdims=True)
    size = np.array([2.0 ** 64, 1.8e19, 1e19, 3e19, 1e25, 1e38, 3.3e38, 1.0])
    x = x * np.resize(size, n)[:, None, None]
    x[5, 0, 1:] = 1.0                                              # one far element among ordinary ones
    x[6, -1, :] = 3.3e38 * (-1.0) ** np.arange(dim)                # the factor is subnormal
    return np.clip(x, -3.38e38, 3.38e38)


@pytest.mark.parametrize("dim,heads,rot,interleaved", [(64, 2, 64, False), (128, 3, 48, False), (64, 5, 32, True), (128, 8, 128, True)])
@pytest.mark.parametrize("size,eps", [(1.0, 1e-6), (2.0 ** -140, 0.0), (2.0 ** -100, 0.0)])
def test_norm_of_keys_whose_squares_leave_fp32(planner, dim, heads, rot, interleaved, size, eps):
    """The norm's factor is that of the definition: only rows of zeros without an epsilon are 0 / 0, codes and scales
    are equal but for a code in one row, and k_out is half a bf16 step off (test_gpu_kv4.py)."""
    rng = np.random.default_rng(dim + heads)
    n = 24
    x = far_heads(rng, n, heads, dim) * size
    pool = Pool4([n], heads, 16, dim)
    k, v = bf16(x).cuda(), bf16(rng.standard_normal((n, heads, dim))).cuda()
    w = torch.rand(dim, device="cuda") + 0.5
    table = planner.rope_table(n, rot)
    k_out = torch.empty_like(k)
    planner.rope_append_kv4(None, k, v, table, cu_of([n]), i32([0]), pool.cache, None, k_norm=w, norm_eps=eps,
                            interleaved=interleaved, k_out=k_out)
    planner.sync_check()
    with np.errstate(divide="ignore", invalid="ignore"):
        want = four_bit.norm_rotate(f64(k), w.cpu().numpy(), table.cpu().numpy(), np.arange(n), interleaved, eps)
    some = (f64(k) != 0).any(-1)                                     # bf16 ends at 2^-133
    assert np.array_equal(np.isfinite(want).all(-1), some) and some.mean() > 0.8
    got = f64(k_out)
    assert np.isnan(got[~some]).all()
    assert np.all(np.abs(got - want)[some] <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want[some]) + 2.0 ** -22)
    codes, scales, _, _ = pool.held(0, n)
    c, sc = four_bit.quantise(want, pool.unit_np[0][None, :, None])
    same_codes(scales, sc, 1)
    same_codes(codes, c, 1)


def test_infinities_and_nan_under_the_norm_stay_in_their_head(planner):
    """inf / inf is NaN in its block and x / inf zero in the others; a NaN is all of its head; heads beside them, in
    the same warp, are as without them."""
    rng = np.random.default_rng(8)
    x = rng.standard_normal((6, 4, 64))
    w = torch.rand(64, device="cuda") + 0.5
    v = bf16(rng.standard_normal((6, 4, 64))).cuda()
    got = []
    for bad in (False, True):
        if bad:
            x[1, 2, 20], x[4, 0, 63], x[2, 3, 5], x[5, 1, 0] = np.inf, -np.inf, np.nan, 2e38
        k = bf16(x).cuda()
        pool = Pool4([6], 4, 16, 64)
        planner.rope_append_kv4(None, k, v, None, cu_of([6]), i32([0]), pool.cache, None, k_norm=w)
        planner.sync_check()
        got.append(pool.held(0, 6))
        with np.errstate(invalid="ignore"):
            c, sc = four_bit.quantise(four_bit.norm_rotate(f64(k), w.cpu().numpy(), None, None, False), pool.unit_np[0][None, :, None])
        same_codes(got[-1][1], sc, 1)
        same_codes(got[-1][0], c, 1)
    touched = np.zeros((6, 4), bool)
    touched[[1, 4, 2, 5], [2, 0, 3, 1]] = True
    for a, b in zip(*got):
        assert np.array_equal(a[~touched], b[~touched])
    assert np.isnan(got[1][1][2, 3]).all() and np.isnan(got[1][1][1, 2]).sum() == 1 and not got[1][0][1, 2].any()


@pytest.mark.parametrize("dim,heads,rot,interleaved", [(64, 2, 64, False), (128, 3, 48, False), (64, 5, 32, True), (128, 8, 128, True)])
@pytest.mark.parametrize("size,eps", [(1.0, 1e-6), (1.0, 1e25), (2.0 ** -140, 0.0), (2.0 ** -100, 0.0), (2.0 ** -100, 1e-35)])
@pytest.mark.parametrize("batch", [1, 12])
def test_norm_of_queries_and_of_the_8_bit_caches_keys_whose_squares_leave_fp32(planner, dim, heads, rot, interleaved, size, eps, batch):
    """Both appends' queries and the 8-bit one's keys, in both its launch shapes, against 64 bits: half a bf16 step, and
    16 * 2^-24 (|a| + |b|) for the rotated fp32 values (test_gpu_kv8.py)."""
    from cem_search_transformer_gb300 import binding
    rng = np.random.default_rng(dim + heads)
    n = 24
    x = far_heads(rng, n, heads, dim) * size
    new = [n] + [0] * (batch - 1)
    pool = Pool4([n] * batch, heads, 16, dim)
    q, v = bf16(x).cuda(), bf16(rng.standard_normal((n, heads, dim))).cuda()
    w = torch.rand(dim, device="cuda") + 0.5
    table = planner.rope_table(n, rot)
    u8 = torch.zeros(2 * batch, heads, 16, dim, dtype=torch.uint8, device="cuda")
    scale = torch.ones(2 * batch, heads, device="cuda")
    eight = binding.KvCache8(u8, u8.clone(), scale, scale.clone(), i32(np.arange(2 * batch).reshape(batch, 2)))
    got = [torch.empty_like(q) for _ in range(3)]
    args = dict(q_norm=w, k_norm=w, norm_eps=eps, interleaved=interleaved)
    planner.rope_append_kv4(q, v, v, table, cu_of(new), i32([0] * batch), pool.cache, got[0], **args)
    planner.rope_append_kv8(q, q, v, table, cu_of(new), i32([0] * batch), eight, got[1], k_out=got[2], **args)
    planner.sync_check()
    e32 = float(np.float32(eps))
    some = (f64(q) != 0).any(-1) | (e32 > 0)
    for t in got:
        for i in range(n):
            for h in range(heads):
                if not some[i, h]:
                    assert torch.isnan(t[i, h]).all()
                    continue
                a = f64(q)[i:i + 1, h:h + 1]
                want = paged.norm_rotate(a, w.cpu().numpy(), table.cpu().numpy(), np.array([i]), interleaved, e32)
                both = 2 * np.abs(paged.norm_rotate(a, w.cpu().numpy(), None, None, interleaved, e32)).max()
                assert np.all(np.abs(f64(t)[i, h] - want[0, 0]) <= 2.0 ** -8 * np.abs(want[0, 0]) + 16 * 2.0 ** -24 * both + 2.0 ** -133), (i, h)


@pytest.mark.parametrize("given,read", [(0.3, 0.25), (3.99, 2.0), (float("nan"), 2.0 ** -40), (0.0, 2.0 ** -40), (-2.0, 2.0 ** -40),
                                        (2.0 ** 50, 2.0 ** 40), (float("inf"), 2.0 ** 40), (2.0 ** -60, 2.0 ** -40)])
@pytest.mark.parametrize("dim", [64, 128])
def test_units_that_are_no_powers_of_two_or_beyond_their_ends(planner, given, read, dim):
    """Read as the power of two at or below or the nearer end, NaN as the least, by the append, the read-back and the
    attention alike: the same bytes and outputs as with that unit."""
    rng = np.random.default_rng(dim)
    x = bf16(rng.standard_normal((40, 2, dim)) * read).cuda()
    q = bf16(rng.standard_normal((1, 1, 4, dim)) * max(2.0 ** -20, min(1.0, 1 / read))).cuda()
    got = []
    for unit in (given, read):
        pool = Pool4([40], 2, 16, dim)
        for t in pool.units:
            t.fill_(unit)
        planner.rope_append_kv4(None, x, x, None, cu_of([40]), i32([0]), pool.cache, None)
        k_read, v_read, out, lse = torch.empty_like(x), torch.empty_like(x), torch.empty_like(q), torch.empty(1, 1, 4, device="cuda")
        planner.kv4_read(pool.cache, cu_of([40]), i32([0]), k_read, v_read)
        ws = torch.empty(planner.attention_kv4_workspace(pool.cache), dtype=torch.uint8, device="cuda")
        mass = torch.zeros(1, 2, pool.table.shape[1] * 16, device="cuda")
        planner.attention_kv4(q, pool.cache, i32([40]), out, 0.125, ws, lse=lse, mass_out=mass)
        planner.sync_check()
        pgs = pool.table_np[0]
        got.append([t[pgs].cpu() for t in (pool.k, pool.v, pool.ks, pool.vs)] + [k_read, v_read, out, lse, mass])
    # (slots behind the 40 tokens keep the pool's filling in both)
    for a, b in zip(*got):
        assert torch.equal(a, b)
    c, sc = four_bit.quantise(f64(x), np.float32(read))
    assert np.array_equal(f64(got[0][5]), four_bit.values(c, sc, read))
