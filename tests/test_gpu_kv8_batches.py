"""The 8-bit cache and the packed attention in batches that mix what the single tests keep apart."""
import numpy as np
import pytest
import torch

from oracle import paged
from test_gpu_attention_packed import call, check, tolerance
from test_gpu_kv8 import BF16, Pool, bf16, check_append, cu_of, f64, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def planner():
    from cem_search_transformer_gb300 import binding, synthetic
    p = binding.Planner(synthetic.PRESETS["small"])
    yield p
    p.close()


@pytest.mark.parametrize("dim,page,rot,interleaved,norm", [
    (64, 128, 64, False, True), (128, 128, 128, True, False), (128, 64, 32, False, True), (64, 64, 0, False, False),
    (64, 16, 48, True, True), (128, 32, 128, False, True)])
def test_many_short_sequences_in_one_chunk(planner, dim, page, rot, interleaved, norm):
    """Five to nine new tokens a sequence, some with none: the whole-page path, where a team of warps
    goes through a score of sequences one after the other, most of them from the middle of a page."""
    rng = np.random.default_rng(page + dim)
    new = [int(n) for n in rng.integers(5, 10, 60)]
    for at in (0, 7, 8, 31, 59):
        new[at] = 0
    old = [int(n) for n in rng.integers(0, 2 * page, 60)]
    assert sum(new) > 4 * 60
    check_append(planner, new, old, 4, 2, dim, page, rot, interleaved, norm, seed=page)


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 32)])
def test_pieces_of_a_page_beside_single_tokens(planner, dim, page):
    """The short path with pieces that it takes a row at a time."""
    new = [1] * 60 + [40, 3, 0, 17]
    old = [int(n) for n in np.random.default_rng(1).integers(0, 50, len(new))]
    assert sum(new) <= 4 * len(new)
    check_append(planner, new, old, 2, 2, dim, page, dim, False, True, seed=dim)


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dim,heads", [(64, 5), (128, 3)])
def test_short_append_in_place(planner, dim, heads, norm):
    """q_out over q and k_out over k, one to three tokens a sequence: a row is written by the lanes that
    read it, after its last use."""
    rng = np.random.default_rng(dim)
    new, page = [1, 3, 2, 0, 3, 1, 2, 2], 16
    old = [15, 14, 0, 3, 30, 7, 16, 31]
    n, batch = sum(new), len(new)
    assert n <= 4 * batch
    rope = planner.rope_table(64, dim)
    weight = torch.from_numpy(rng.uniform(0.5, 1.5, dim).astype(np.float32)).cuda() if norm else None
    x = [bf16(rng.standard_normal((n, heads, dim))).cuda() for _ in range(3)]
    states = []
    for in_place in (False, True):
        pool = Pool([a + b for a, b in zip(new, old)], heads, page, dim, seed=4)
        pool.fill(old, 6)
        q, k, v = (t.clone() for t in x)
        q_out, k_out = (q, k) if in_place else (torch.empty_like(q), torch.empty_like(k))
        planner.rope_append_kv8(q, k, v, rope, cu_of(new), i32(old), pool.cache, q_out, q_norm=weight, k_norm=weight,
                                k_out=k_out)
        planner.sync_check()
        states.append([q_out, k_out, pool.k, pool.v, pool.ks.view(torch.int32), pool.vs.view(torch.int32)])
    for a, b in zip(*states):
        assert torch.equal(a, b)
    assert not torch.equal(states[0][1], x[1])


@pytest.mark.parametrize("heads,group,dim,frame", [(7, 1, 64, 1), (9, 2, 128, 1), (5, 3, 64, 40)])
def test_odd_heads_over_cached_beginnings(planner, heads, group, dim, frame):
    """Enough items that the last rows of two heads share one, with a head left over and more keys than
    queries."""
    rng = np.random.default_rng(heads * group)
    nq = [int(n) for n in rng.integers(0, 300 // group, 120)]
    nk = [n + int(p) for n, p in zip(nq, rng.integers(0, 250, 120))]
    check(planner, nq, nk, heads * group, heads, dim, frame, seed=5, behind=2)


@pytest.mark.parametrize("dim,page,norm", [(128, 32, True), (64, 16, False)])
def test_what_is_read_back_is_what_was_appended(planner, dim, page, norm):
    """Prompts, then a second chunk; every sequence's cached keys and values, element by element, against
    the rotated keys that the calls gave out and the values that they were given."""
    rng = np.random.default_rng(2)
    heads, counts = 2, ([70, 1, 131], [20, 33, 1])
    lens = [a + b for a, b in zip(*counts)]
    pool = Pool(lens, heads, page, dim)
    rope = planner.rope_table(max(lens), dim)
    weight = torch.rand(dim, device="cuda") + 0.5 if norm else None
    keys, values = [[] for _ in lens], [[] for _ in lens]
    for count, start in ((counts[0], [0] * 3), (counts[1], counts[0])):
        n = sum(count)
        k, v = (bf16(rng.standard_normal((n, heads, dim))).cuda() for _ in range(2))
        k_out = torch.empty_like(k)
        planner.rope_append_kv8(None, k, v, rope, cu_of(count), i32(start), pool.cache, None, k_norm=weight, k_out=k_out)
        table, pos = paged.rope_table(max(lens), dim), np.concatenate([s + np.arange(c) for s, c in zip(start, count)])
        want = paged.norm_rotate(f64(k), None if weight is None else f64(weight), table, pos, False)
        both = np.abs(paged.norm_rotate(f64(k), None if weight is None else f64(weight), None, pos, False)).max(-1, keepdims=True) * 2
        assert np.all(np.abs(f64(k_out) - want) <= BF16 * np.abs(want) + 16 * 2.0 ** -24 * both)
        at = 0
        for s, c in enumerate(count):
            keys[s].append(f64(k_out[at:at + c]))
            values[s].append(f64(v[at:at + c]))
            at += c
    got = [torch.empty(sum(lens), heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    planner.kv8_read(pool.cache, cu_of(lens), i32([0] * 3), *got)
    planner.sync_check()
    at = 0
    for s, n in enumerate(lens):
        pages = [int(pool.table_np[s, i // page]) for i in range(n)]
        for out, given, scales, rounded in ((got[0], keys, pool.ks, BF16), (got[1], values, pool.vs, 0.0)):
            x = np.concatenate(given[s])
            scale = f64(scales)[pages][:, :, None]
            # half an e4m3 step; twice for tokens of the first call, whose page's scale may have grown
            # under the second; the keys given out are themselves half a bf16 step off
            step = np.maximum(np.abs(x) * (1 + rounded) * 2.0 ** -4, scale * 2.0 ** -10)
            step[:counts[0][s]] *= 2
            err = np.abs(f64(out[at:at + n]) - x)
            assert np.all(err <= step * (1 + 2.0 ** -4) + rounded * np.abs(x)), err.max()
        at += n


def test_frames_of_packed_and_the_predictors_attention_against_the_oracle(planner):
    """Both within the tolerance of bf16 weights, element by element."""
    T, frames, heads, dim, ncand = 130, 3, 2, 64, 2
    d = heads * dim
    qkv = bf16(np.random.default_rng(9).standard_normal((ncand, frames * T, 3 * d)) * 0.7).cuda()
    flat = qkv.view(ncand * frames * T, 3 * heads, dim)
    lens = [frames * T] * ncand
    out, _ = call(planner, flat[:, :heads], flat[:, heads:2 * heads], flat[:, 2 * heads:], lens, lens, frame=T)
    kv = qkv[:, :, d:].contiguous()
    dense = torch.zeros(frames, ncand * T, d, dtype=torch.bfloat16, device="cuda")
    for f in range(frames):
        planner.attention_bf16(qkv[:, f * T:(f + 1) * T, :d].contiguous().view(torch.int16), kv.view(torch.int16),
                               dense[f].view(torch.int16), ncand, T, (f + 1) * T, frames * T, heads, d)
    planner.sync_check()
    dense = dense.view(frames, ncand, T, heads, dim).permute(1, 0, 2, 3, 4).reshape(ncand, frames * T, heads, dim)
    for c in range(ncand):
        rows = slice(c * frames * T, (c + 1) * frames * T)
        q, k, v = (f64(flat[rows, i * heads:(i + 1) * heads]) for i in range(3))
        want, _, mag, s_abs = paged.softmax_rows(q, k, v, paged.limits(frames * T, frames * T, T), dim ** -0.5)
        for got in (out[rows], dense[c]):
            assert np.all(np.abs(f64(got) - want) <= tolerance(want, mag, s_abs, frames * T, dim))
