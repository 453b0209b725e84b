"""Attention of packed prompts on the GPU against the oracle in 64 bits, and the packed prompt, the
8-bit cache and the attention over it used together.

Tolerances as in the cached attention's tests, with bf16 weights (half a step 2^-8; bf16 has fp32's
range, so no smallest-step term); a weight's reference may trail the maximum, which changes no
relative error."""
import numpy as np
import pytest
import torch

from oracle import paged
from test_gpu_kv8 import BF16, Pool, bf16, check_attention, cu_of, f64, i32, lse_tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def planner():
    from cem_search_transformer_gb300 import binding, synthetic
    p = binding.Planner(synthetic.PRESETS["small"])
    yield p
    p.close()


def tolerance(want, a, s_abs, n, dim):
    delta = dim * 2.0 ** -22 * s_abs[..., None] + 2.0 ** -21 + n * 2.0 ** -23
    return BF16 * np.abs(want) + (1 + BF16) * 2 * a * (BF16 + delta)


def call(planner, q, k, v, nq, nk, frame=1, scale=None, extra=0):
    out = torch.full((q.shape[0], q.shape[1], q.shape[2]), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 9.0, device="cuda")
    planner.attention_packed(q, k, v, cu_of(nq), cu_of(nk), out, q.shape[2] ** -0.5 if scale is None else scale,
                             frame=frame, lse=lse)
    planner.sync_check()
    return out, lse


def check(planner, nq, nk, q_heads, kv_heads, dim, frame=1, seed=0, behind=0, scale=None):
    rng = np.random.default_rng(seed)
    tq, tk = sum(nq) + behind, sum(nk) + behind
    qkv = bf16(rng.standard_normal((max(tq, tk), q_heads + 2 * kv_heads, dim))).cuda()
    q, k, v = qkv[:tq, :q_heads], qkv[:tk, q_heads:q_heads + kv_heads], qkv[:tk, q_heads + kv_heads:]
    out, lse = call(planner, q, k, v, nq, nk, frame, scale)
    scale = dim ** -0.5 if scale is None else scale
    a_q = a_k = 0
    for a, b in zip(nq, nk):
        want, want_lse, mag, s_abs = paged.softmax_rows(f64(q[a_q:a_q + a]), f64(k[a_k:a_k + b]), f64(v[a_k:a_k + b]),
                                                        paged.limits(a, b, frame), scale)
        got, got_lse = f64(out[a_q:a_q + a]), f64(lse[a_q:a_q + a])
        assert np.all(np.isfinite(got))
        assert np.all(np.abs(got - want) <= tolerance(want, mag, s_abs, b, dim)), np.abs(got - want).max()
        empty = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(got_lse), empty)
        assert np.all(np.abs(got_lse[~empty] - want_lse[~empty]) <= lse_tolerance(s_abs, b, dim, want_lse)[~empty])
        a_q, a_k = a_q + a, a_k + b
    assert torch.all(out[a_q:] == 9) and torch.all(lse[a_q:] == 9)
    return q, k, v, out


@pytest.mark.parametrize("nq,nk,q_heads,kv_heads,dim,frame", [
    ([1], [1], 1, 1, 64, 1),
    ([1], [1], 1, 1, 128, 1),
    ([128], [128], 1, 1, 128, 1),
    ([129], [129], 2, 2, 64, 1),
    ([256], [256], 1, 1, 128, 1),
    ([257], [257], 1, 1, 64, 1),
    ([700], [700], 2, 1, 128, 1),
    ([200], [200], 4, 4, 64, 1),
    ([33, 1, 150, 64], [33, 1, 150, 64], 8, 2, 128, 1),
    ([5, 0, 77], [5, 0, 77], 6, 2, 64, 1),                 # a group of three: 126 of 128 rows
    ([90], [90], 7, 1, 128, 1),
    ([40, 9], [40, 9], 16, 1, 64, 1),
    ([3], [130], 128, 1, 64, 1),                           # one token a tile
    ([4], [4], 100, 1, 128, 1),
    ([10, 200], [300, 200], 4, 1, 128, 1),                 # a cached beginning
    ([50, 20], [20, 0], 4, 2, 64, 1),                      # rows that see nothing; no keys at all
    ([300], [40], 1, 1, 128, 1),                           # tiles that see nothing
    ([130], [130], 2, 2, 64, 66),
    ([774], [774], 2, 2, 64, 258),
    ([258, 516], [774, 516], 2, 1, 128, 258),
    ([100], [333], 2, 1, 64, 1000),                        # no mask
    ([1100], [1100], 1, 1, 64, 1),                         # the ring's second lap
    ([1500], [1500], 1, 1, 128, 3),
])
def test_packed_matches_oracle(planner, nq, nk, q_heads, kv_heads, dim, frame):
    check(planner, nq, nk, q_heads, kv_heads, dim, frame, seed=sum(nq) + dim, behind=3)


def test_many_sequences(planner):
    rng = np.random.default_rng(1)
    nq = [int(x) for x in rng.integers(0, 40, 100)]
    check(planner, nq, [n + int(x) for n, x in zip(nq, rng.integers(0, 60, 100))], 4, 2, 64, seed=2)


@pytest.mark.parametrize("scale", [1e-4, 1.0])
def test_scales(planner, scale):
    check(planner, [200, 60], [200, 90], 2, 1, 128, seed=3, scale=scale)


@pytest.mark.parametrize("dim,frame", [(64, 1), (128, 1), (128, 66)])
def test_unseen_values_do_not_reach_a_query(planner, dim, frame):
    """Infinities and NaN in the other sequences and in later tokens: a query that does not see
    them is untouched to the bit; one that does shows them."""
    nq = [150, 200, 70]
    q, k, v, clean = check(planner, nq, nq, 2, 1, dim, frame, seed=6)
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    at = 150 + 137                                          # token 137 of the second sequence
    k2, v2 = k.clone(), v.clone()
    k2[:150], v2[:150] = float("nan"), float("inf")         # the neighbours
    k2[350:], v2[350:] = float("inf"), float("nan")
    v2[at, 0, 5], v2[at, 0, dim - 1] = float("inf"), float("nan")
    out, _ = call(planner, q, k2, v2, nq, nq, frame)
    first = 137 // frame * frame                            # the first query that sees token 137
    mine = slice(150, 150 + first)
    assert torch.equal(out[mine], clean[mine])
    seen = out[150 + first:350]
    assert torch.all(seen[..., 5] == float("inf")) and torch.all(torch.isnan(seen[..., dim - 1]))
    rest = torch.ones(dim, dtype=torch.bool, device="cuda")
    rest[5] = rest[dim - 1] = False
    assert torch.equal(seen[..., rest], clean[150 + first:350][..., rest])
    k2 = k.clone()
    k2[at] = float("nan")
    out, _ = call(planner, q, k2, v, nq, nq, frame)
    assert torch.equal(out[mine], clean[mine]) and torch.all(torch.isnan(out[150 + first:350]))


@pytest.mark.parametrize("nq,nk,q_heads,kv_heads,dim,frame", [
    ([1], [1000], 2, 1, 64, 1),
    ([100], [1000], 1, 1, 128, 1),
    ([5], [193], 16, 1, 128, 1),                           # four tiles of keys, one in the last
    ([5], [192], 16, 1, 64, 1),
    ([60, 300, 2, 7], [500, 300, 3, 700], 4, 2, 64, 50),
    ([1, 17, 130, 40], [900, 640, 450, 321], 2, 2, 128, 1),
])
def test_few_queries_over_many_keys(planner, nq, nk, q_heads, kv_heads, dim, frame):
    check(planner, nq, nk, q_heads, kv_heads, dim, frame, seed=nk[0])


@pytest.mark.parametrize("dim", [64, 128])
def test_few_queries_and_values_that_are_not_finite(planner, dim):
    nq, nk = [6, 3], [500, 400]
    q, k, v, clean = check(planner, nq, nk, 2, 1, dim, seed=2)
    k, v = k.contiguous(), v.contiguous()
    v2, k2 = v.clone(), k.clone()
    v2[497, 0, 5] = float("inf")                           # the first two queries do not see key 497 ..
    v2[40, 0, 7] = -float("inf")                           # all of the sequence see key 40
    k2[498] = float("nan")                                 # nor the first four key 498
    out, lse = call(planner, q, k2, v2, nq, nk)
    assert torch.all(out[:6, :, 7][:4] == -float("inf"))
    rest = torch.ones(dim, dtype=torch.bool, device="cuda")
    rest[5] = rest[7] = False
    assert torch.equal(out[:4][..., rest], clean[:4][..., rest])
    assert torch.equal(out[:3, :, 5], clean[:3, :, 5]) and torch.all(out[3, :, 5] == float("inf"))
    assert torch.all(torch.isnan(out[4:6])) and torch.all(torch.isnan(lse[4:6]))
    assert torch.equal(out[6:], clean[6:])


@pytest.mark.parametrize("heads,group,dim,frame,prefix", [(7, 1, 64, 1, 0), (8, 2, 128, 1, 200), (8, 1, 64, 50, 90),
                                                          (9, 3, 128, 7, 0)])
def test_many_short_sequences(planner, heads, group, dim, frame, prefix):
    """Enough items that one query tile's worth of rows is taken for two heads at a time."""
    rng = np.random.default_rng(heads)
    nq = [int(n) for n in rng.integers(0, 300 // group, 100)]
    nk = [n + int(p) for n, p in zip(nq, rng.integers(0, prefix + 1, 100))]
    q, k, v, clean = check(planner, nq, nk, heads * group, heads, dim, frame, seed=3, behind=2)
    s = max(range(100), key=lambda i: (0 < nq[i] <= 128 // group) * nk[i])   # one tile of queries
    q0, k0 = sum(nq[:s]), sum(nk[:s])
    k, v = k.contiguous(), v.contiguous()
    last = k0 + nk[s] - 1                                  # seen by its last queries alone, if causal
    v[last, 1, 3] = float("nan")
    v[last, 0, 4] = float("inf")
    out, _ = call(planner, q, k, v, nq, nk, frame)
    sees = np.array(paged.limits(nq[s], nk[s], frame)) == nk[s]
    hit = torch.zeros_like(out, dtype=torch.bool)
    rows = torch.from_numpy(np.flatnonzero(sees)).cuda() + q0
    for at, column in ((1, 3), (0, 4)):
        hit[rows, at * group:(at + 1) * group, column] = True
    assert torch.equal(out[~hit], clean[~hit])
    assert torch.all(torch.isnan(out[rows, group:2 * group, 3])) and torch.all(out[rows, :group, 4] == float("inf"))


def test_mostly_empty_batch(planner):
    """A batch padded with empty sequences, ahead, between and behind those with tokens: far more
    places than there are items."""
    n = [0] * 900
    for at, tokens in ((40, 300), (41, 1), (600, 150), (899, 20)):
        n[at] = tokens
    check(planner, n, n, 4, 4, 64, seed=9, behind=700)
    check(planner, [0] * 50 + [5], [7] * 50 + [5], 2, 1, 128, seed=10, behind=5)


def test_bad_offsets_are_skipped_and_reported(planner):
    from cem_search_transformer_gb300 import binding
    x = bf16(np.random.default_rng(0).standard_normal((64, 2, 64))).cuda()
    for cq, ck in (([0, 32, 65], [0, 32, 64]), ([0, 32, 64], [0, 40, 30]), ([-1, 32, 64], [0, 32, 64])):
        out = torch.full_like(x, 9.0)
        planner.attention_packed(x, x, x, i32(cq), i32(ck), out, 0.1)
        with pytest.raises(binding.JepaError, match="outside its buffer"):
            planner.sync_check()
    for change, match in ((dict(scale=-1.0), "bad argument"), (dict(frame=0), "bad argument"),
                          (dict(q=x[:, :1]), None), (dict(k=x[..., :32]), "contiguous")):
        args = {**dict(q=x, k=x, v=x, cu_q=i32([0, 64]), cu_k=i32([0, 64]), out=torch.empty_like(x), scale=0.1, frame=1),
                **change}
        with pytest.raises(binding.JepaError, match=match):
            planner.attention_packed(**args)
    planner.sync_check()


def test_nan_queries_stay_in_their_row(planner):
    q, k, v, clean = check(planner, [140], [140], 2, 1, 128, seed=4)
    q = q.contiguous()
    q[50, 1, 3] = float("nan")
    q[100, 0, 5] = float("inf")
    out, lse = call(planner, q, k, v, [140], [140])
    bad = torch.zeros(140, 2, dtype=torch.bool, device="cuda")
    bad[50, 1] = bad[100, 0] = True
    assert torch.all(torch.isnan(out[bad])) and torch.all(torch.isnan(lse[bad]))
    assert torch.equal(out[~bad], clean[~bad])


def test_offsets_that_begin_behind_token_0(planner):
    x = [bf16(np.random.default_rng(i).standard_normal((200, h, 64))).cuda() for i, h in enumerate((4, 2, 2))]
    want, _ = call(planner, x[0][30:], x[1][50:], x[2][50:], [100], [150])
    out = torch.full_like(x[0], 9.0)
    planner.attention_packed(*x, i32([30, 130]), i32([50, 200]), out, 0.125)
    planner.sync_check()
    assert torch.equal(out[30:130], want[:100]) and torch.all(out[:30] == 9) and torch.all(out[130:] == 9)


def test_graph_replay(planner):
    rng = np.random.default_rng(5)
    x = [bf16(rng.standard_normal((300, h, 128))).cuda() for h in (4, 2, 2)]
    cu = cu_of([100, 200])
    out = torch.zeros_like(x[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        planner.attention_packed(*x, cu, cu, out, 0.1)
    for lens in ([100, 200], [300, 0], [1, 2]):
        cu.copy_(cu_of(lens))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = torch.zeros_like(out)
        planner.attention_packed(*x, cu_of(lens), cu_of(lens), want, 0.1)
        planner.sync_check()
        assert torch.equal(out, want)


def test_frames_agree_with_the_predictors_attention(planner):
    """Block-causal attention over three frames of T tokens in one call, against the predictor's
    frame-by-frame attention over its dense cache (both within the tolerance of bf16 weights)."""
    T, frames, heads, dim, ncand = 130, 3, 2, 64, 2
    d = heads * dim
    rng = np.random.default_rng(9)
    qkv = bf16(rng.standard_normal((ncand, frames * T, 3 * d)) * 0.7).cuda()
    flat = qkv.view(ncand * frames * T, 3 * heads, dim)
    lens = [frames * T] * ncand
    out, _ = call(planner, flat[:, :heads], flat[:, heads:2 * heads], flat[:, 2 * heads:], lens, lens, frame=T)
    kv = qkv[:, :, d:].contiguous()
    for f in range(frames):
        qf = qkv[:, f * T:(f + 1) * T, :d].contiguous()
        o = torch.zeros(ncand * T, d, dtype=torch.bfloat16, device="cuda")
        planner.attention_bf16(qf.view(torch.int16), kv.view(torch.int16), o.view(torch.int16), ncand, T, (f + 1) * T,
                               frames * T, heads, d)
        planner.sync_check()
        got = out.view(ncand, frames, T, d)[:, f].reshape(ncand * T, d)
        # both are within 2^-8 sum p |v| (weights) and half a bf16 step of the exact result
        assert torch.max(torch.abs(got.float() - o.float())) <= 2 * (2 * BF16 * 0.7 * 5)
        assert torch.mean(torch.abs(got.float() - o.float())) < 2e-3


@pytest.mark.parametrize("dim,page,norm", [(128, 32, True), (64, 16, False)])
def test_prompt_then_chunk_then_single_tokens(planner, dim, page, norm):
    """A model layer's life: packed prompts (rotated, appended, attended), a second chunk that reads
    the cached beginning back, then single tokens over the cache; each output against the oracle
    on what the cache holds."""
    rng = np.random.default_rng(21)
    q_heads, kv_heads = 4, 2
    prompt, chunk, steps = [70, 1, 131], [20, 33, 1], 3
    total = [a + b + steps for a, b in zip(prompt, chunk)]
    pool = Pool(total, kv_heads, page, dim)
    rope = planner.rope_table(max(total), dim)
    norms = dict(q_norm=torch.rand(dim, device="cuda") + 0.5, k_norm=torch.rand(dim, device="cuda") + 0.5) if norm else {}
    scale = dim ** -0.5

    def projected(n):
        x = bf16(rng.standard_normal((n, q_heads + 2 * kv_heads, dim))).cuda()
        return x[:, :q_heads], x[:, q_heads:q_heads + kv_heads], x[:, q_heads + kv_heads:]

    def against(out, q, lens_q, lens_k, keys, values):
        a = b = 0
        for n, m in zip(lens_q, lens_k):
            want, _, mag, s_abs = paged.softmax_rows(f64(q[a:a + n]), f64(keys[b:b + m]), f64(values[b:b + m]),
                                                     paged.limits(n, m, 1), scale)
            assert np.all(np.abs(f64(out[a:a + n]) - want) <= tolerance(want, mag, s_abs, m, dim))
            a, b = a + n, b + m

    # the prompts: attention on the rotated bf16 keys
    q, k, v = projected(sum(prompt))
    qr, kr = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(k.shape, dtype=q.dtype, device="cuda")
    planner.rope_append_kv8(q, k, v, rope, cu_of(prompt), i32([0] * 3), pool.cache, qr, k_out=kr, **norms)
    out, _ = call(planner, qr, kr, v, prompt, prompt)
    against(out, qr, prompt, prompt, kr, v)
    # a second chunk: everything cached is read back
    q, k, v = projected(sum(chunk))
    qr = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    planner.rope_append_kv8(q, k, v, rope, cu_of(chunk), i32(prompt), pool.cache, qr, **norms)
    lens = [a + b for a, b in zip(prompt, chunk)]
    keys = torch.empty(sum(lens), kv_heads, dim, dtype=torch.bfloat16, device="cuda")
    values = torch.empty_like(keys)
    planner.kv8_read(pool.cache, cu_of(lens), i32([0] * 3), keys, values)
    out, _ = call(planner, qr, keys, values, chunk, lens)
    against(out, qr, chunk, lens, keys, values)
    # what was read back is the chunk's own rotated keys to half an e4m3 step of their block
    assert torch.mean(torch.abs(values[lens[0] - chunk[0]:lens[0]].float() - v[:chunk[0]].float())) < 0.05
    # single tokens
    ws = torch.empty(planner.attention_kv8_workspace(pool.cache), dtype=torch.uint8, device="cuda")
    for t in range(steps):
        q, k, v = projected(3)
        qr = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        planner.rope_append_kv8(q, k, v, rope, cu_of([1] * 3), i32([n + t for n in lens]), pool.cache, qr, **norms)
        now = [n + t + 1 for n in lens]
        ref = [pool.values(s, n) for s, n in enumerate(now)]
        check_attention(planner, pool, ref, now, 1, q_heads, True, seed=0, q=qr.view(3, 1, q_heads, dim), workspace=ws)
