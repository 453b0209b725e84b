"""Workloads of the 8-bit paged key/value cache and the attention operators around it.

Four operators, grouped in three kinds of case:
  * "append": queries and keys are normalised per head and rotated, keys and values go to the
    pages of an 8-bit cache (e4m3 codes, one power-of-two scale per page, head and k / v), and
    the touched pages are read back as bf16 values;
  * "cached": attention of one or a few new tokens per sequence over that cache;
  * "prompt": attention of whole packed prompts, causal or causal over frames, grouped heads.

``run`` computes a case in plain torch operations (``own`` false) or through the library.
"""
import functools
import math
import random

import torch

own = False

LOG_SCALE_MIN, LOG_SCALE_MAX = -40, 40   # exponents a block's scale may take
E4M3_MAX = 448.0


# ---- cases -------------------------------------------------------------------------------

def listed():
    return [
        # one robot, one new token: all of it is latency
        dict(name="append_1_token", kind="append", batch=1, new_lo=1, new_hi=1, old_lo=300, old_hi=300,
             q_heads=16, kv_heads=16, dim=64, page=16, rot=32, interleaved=True, norm=False, mix=1),
        # one serving step of a batch, sequences of all lengths
        dict(name="append_step_64", kind="append", batch=64, new_lo=1, new_hi=1, old_lo=0, old_hi=4096,
             q_heads=32, kv_heads=8, dim=128, page=64, rot=128, interleaved=False, norm=True, mix=2),
        # one frame of 258 tokens for each of 24 candidates of the predictor's own head layout
        dict(name="append_frames_24", kind="append", batch=24, new_lo=258, new_hi=258, old_lo=258,
             old_hi=258, q_heads=16, kv_heads=16, dim=64, page=32, rot=64, interleaved=False,
             norm=False, mix=3),
        # packed prompts of different lengths
        dict(name="append_prompts", kind="append", batch=9, new_lo=100, new_hi=4500, old_lo=0,
             old_hi=700, q_heads=32, kv_heads=8, dim=128, page=64, rot=128, interleaved=False,
             norm=True, mix=4),
        # one sequence of a few frames: latency
        dict(name="cached_1x517", kind="cached", batch=1, tq=1, len_lo=517, len_hi=517, q_heads=16,
             kv_heads=16, dim=64, page=32, causal=True, mix=5),
        # a serving batch of ragged lengths
        dict(name="cached_32_ragged", kind="cached", batch=32, tq=1, len_lo=100, len_hi=8000, q_heads=32,
             kv_heads=8, dim=128, page=64, causal=True, mix=6),
        # two long contexts
        dict(name="cached_2_long", kind="cached", batch=2, tq=1, len_lo=100001, len_hi=130001,
             q_heads=64, kv_heads=8, dim=128, page=128, causal=True, mix=7),
        # action and state token of 256 candidates over three frames of 258 tokens
        dict(name="cached_candidates", kind="cached", batch=256, tq=2, len_lo=776, len_hi=776, q_heads=16,
             kv_heads=16, dim=64, page=16, causal=False, mix=8),
        # one short prompt
        dict(name="prompt_1x200", kind="prompt", batch=1, q_lo=200, q_hi=200, pre_lo=0, pre_hi=0,
             q_heads=16, kv_heads=16, dim=64, frame=1, mix=9),
        # ragged packed prompts
        dict(name="prompt_ragged", kind="prompt", batch=12, q_lo=33, q_hi=2900, pre_lo=0, pre_hi=300,
             q_heads=32, kv_heads=8, dim=128, frame=1, mix=10),
        # three frames of 258 tokens for 32 problems, causal over frames, the predictor's heads
        dict(name="prompt_frames", kind="prompt", batch=32, q_lo=774, q_hi=774, pre_lo=0, pre_hi=0,
             q_heads=16, kv_heads=16, dim=64, frame=258, mix=11),
        # one long prompt
        dict(name="prompt_1x10007", kind="prompt", batch=1, q_lo=10007, q_hi=10007, pre_lo=0, pre_hi=0,
             q_heads=32, kv_heads=8, dim=128, frame=1, mix=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    kind = rng.choice(("append", "cached", "prompt"))
    while True:
        dim = rng.choice((64, 128))
        kv = rng.choice((1, 2, 3, 4, 5, 8, 16))
        group = rng.choice((1, 1, 2, 3, 4, 6, 7, 8))
        case = dict(kind=kind, q_heads=kv * group, kv_heads=kv, dim=dim, mix=rng.randrange(1 << 20))
        if kind == "append":
            long = rng.random() < 0.5
            lo = _log_int(rng, 1, 400) if long else 1
            case.update(batch=_log_int(rng, 1, 12 if long else 256), new_lo=lo,
                        new_hi=lo + _log_int(rng, 1, 4000) if long else rng.choice((1, 1, 2, 3)),
                        old_lo=0, old_hi=_log_int(rng, 1, 4000), page=rng.choice((16, 32, 64, 128)),
                        rot=16 * rng.randint(1, dim // 16), interleaved=rng.random() < 0.5,
                        norm=rng.random() < 0.5)
        elif kind == "cached":
            lo = _log_int(rng, 1, 60000)
            case.update(batch=_log_int(rng, 1, 256), tq=rng.choice((1, 1, 1, 2, 3, 4, 8)), len_lo=lo,
                        len_hi=lo + _log_int(rng, 1, 60000), page=rng.choice((16, 32, 64, 128)),
                        causal=rng.random() < 0.7)
        else:
            lo = _log_int(rng, 1, 4000)
            case.update(batch=_log_int(rng, 1, 32), q_lo=lo, q_hi=lo + _log_int(rng, 1, 4000), pre_lo=0,
                        pre_hi=rng.choice((0, 0, _log_int(rng, 1, 2000))),
                        frame=rng.choice((1, 1, 1, 66, 258)))
        w, top = work(case), _largest()[kind]
        if w["bytes"] <= top[0] and w["flops"] <= top[1] and _padded(case) <= top[2]:
            return case


@functools.lru_cache(None)
def _largest():
    """By kind: the most bytes, flops and padded elements that a listed case has."""
    top = {}
    for c in listed():
        w, t = work(c), top.get(c["kind"], (0, 0, 0))
        top[c["kind"]] = (max(t[0], w["bytes"]), max(t[1], w["flops"]), max(t[2], _padded(c)))
    return top


def _padded(case):
    """Elements of the plain form's largest intermediate, which pads sequences to the longest."""
    if case["kind"] == "prompt":
        nq, nk = _prompt_lengths(case)
        return case["batch"] * case["q_heads"] * max(nq) * max(nk)
    if case["kind"] == "cached":
        return case["batch"] * case["kv_heads"] * max(_cached_lengths(case)) * case["dim"]
    return sum(_append_lengths(case)[0]) * (case["q_heads"] + case["kv_heads"]) * case["dim"]


def _spread(lo, hi, n, mix):
    """n lengths between lo and hi; the longest is among them."""
    r = random.Random(mix)
    got = [r.randint(lo, hi) for _ in range(n)]
    got[r.randrange(n)] = hi
    return got


def _append_lengths(case):
    new = _spread(case["new_lo"], case["new_hi"], case["batch"], case["mix"])
    old = _spread(case["old_lo"], case["old_hi"], case["batch"], case["mix"] + 1)
    return new, old


def _cached_lengths(case):
    return _spread(case["len_lo"], case["len_hi"], case["batch"], case["mix"])


def _prompt_lengths(case):
    nq = _spread(case["q_lo"], case["q_hi"], case["batch"], case["mix"])
    pre = _spread(case["pre_lo"], case["pre_hi"], case["batch"], case["mix"] + 1)
    return nq, [a + b for a, b in zip(nq, pre)]


def _visible(nq, nk, frame):
    """Visible (query, key) pairs of one sequence: query i sees the keys of its own frame and
    of earlier ones."""
    total, first = 0, nk - nq
    for f in range(first // frame, (nk - 1) // frame + 1):
        rows = min(nk, (f + 1) * frame) - max(first, f * frame)
        total += max(0, rows) * min(nk, (f + 1) * frame)
    return total


def work(case):
    d, hq, hkv = case["dim"], case["q_heads"], case["kv_heads"]
    if case["kind"] == "append":
        new, old = _append_lengths(case)
        n = sum(new)
        read = sum(a + o % case["page"] for a, o in zip(new, old))
        byts = n * (2 * (hq + 2 * hkv) * d + 2 * hq * d + 2 * hkv * d + 4 * case["rot"])
        byts += read * (2 * hkv * d + 4 * hkv * d)
        return {"bytes": byts, "flops": 8 * n * (hq + 2 * hkv) * d}
    if case["kind"] == "cached":
        lens = _cached_lengths(case)
        rows = case["batch"] * case["tq"] * hq
        seen = 0
        for n in lens:
            first = n - case["tq"]
            seen += sum(max(0, first + t + 1) if case["causal"] else n for t in range(case["tq"]))
        byts = sum(lens) * 2 * hkv * d + rows * d * 4 + rows * 4
        byts += sum(-(-n // case["page"]) for n in lens) * (8 * hkv + 4)
        return {"bytes": byts, "flops": 4 * d * hq * seen}
    nq, nk = _prompt_lengths(case)
    byts = sum(nq) * (4 * hq * d + 4 * hq) + sum(nk) * 4 * hkv * d
    return {"bytes": byts, "flops": 4 * d * hq * sum(_visible(a, b, case["frame"]) for a, b in zip(nq, nk))}


# ---- inputs ------------------------------------------------------------------------------

def _i32(values):
    return torch.tensor(list(values), dtype=torch.int32, device="cuda")


def _cumulative(lengths):
    total, out = 0, [0]
    for n in lengths:
        total += n
        out.append(total)
    return _i32(out)


def _heads(gen, n, heads, dim):
    """Rows of n tokens whose heads have magnitudes of their own, as projections give them."""
    size = torch.rand(heads, 1, device="cuda", generator=gen) * 1.5 + 0.25
    return (torch.randn(n, heads, dim, device="cuda", generator=gen) * size).to(torch.bfloat16)


def _pool(gen, pages, heads, page, dim):
    """Pages already filled: e4m3 codes and the power-of-two scale of each page and head."""
    codes = torch.empty(pages, heads, page, dim, dtype=torch.uint8, device="cuda")
    scale = torch.empty(pages, heads, dtype=torch.float32, device="cuda")
    size = torch.rand(1, heads, 1, 1, device="cuda", generator=gen) * 1.5 + 0.25
    step = max(1, (1 << 27) // (heads * page * dim))
    for a in range(0, pages, step):
        x = torch.randn(min(step, pages - a), heads, page, dim, device="cuda", generator=gen) * size
        s = _block_scale(x.abs().amax((2, 3)))
        codes[a:a + step] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scale[a:a + step] = s
    return codes, scale


def _tables(gen, lengths, page):
    """A page table that hands out the pages of a pool in random order; -1 where there is none."""
    need = [-(-n // page) for n in lengths]
    total, most = sum(need), max(1, max(need))
    order = torch.randperm(max(1, total), device="cuda", generator=gen).to(torch.int32)
    table = torch.full((len(lengths), most), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return table, max(1, total)


def _rotary_table(positions, rot, base=10000.0):
    """cos in columns [0, rot/2), sin in [rot/2, rot), for positions 0 .. positions - 1."""
    inv = base ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float()


@functools.lru_cache(None)
def _planner():
    from cem_search_transformer_gb300 import binding, synthetic
    return binding.Planner(synthetic.PRESETS["small"])


def _handle(st):
    from cem_search_transformer_gb300 import binding
    return binding.KvCache8(st["kc"], st["vc"], st["ks"], st["vs"], st["table"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    d, hq, hkv = case["dim"], case["q_heads"], case["kv_heads"]
    st = dict(case=case)
    if case["kind"] == "prompt":
        nq, nk = _prompt_lengths(case)
        st.update(q=_heads(gen, sum(nq), hq, d), k=_heads(gen, sum(nk), hkv, d), v=_heads(gen, sum(nk), hkv, d),
                  cu_q=_cumulative(nq), cu_k=_cumulative(nk), max_q=max(nq), max_k=max(nk),
                  out=torch.empty(sum(nq), hq, d, dtype=torch.bfloat16, device="cuda"),
                  lse=torch.empty(sum(nq), hq, device="cuda"))
        if own:
            _planner()
        return st
    page = case["page"]
    if case["kind"] == "append":
        new, old = _append_lengths(case)
        lens = [a + b for a, b in zip(new, old)]
        first = [o // page * page for o in old]
        window = [n - f for n, f in zip(lens, first)]
        qkv = _heads(gen, sum(new), hq + 2 * hkv, d)   # one projection's rows: strided q, k, v
        st.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], cu=_cumulative(new),
                  start=_i32(old), first=_i32(first), cu_window=_cumulative(window),
                  rope=_rotary_table(max(lens), case["rot"]), q_norm=None, k_norm=None,
                  q_out=torch.empty(sum(new), hq, d, dtype=torch.bfloat16, device="cuda"),
                  k_read=torch.empty(sum(window), hkv, d, dtype=torch.bfloat16, device="cuda"),
                  v_read=torch.empty(sum(window), hkv, d, dtype=torch.bfloat16, device="cuda"))
        if case["norm"]:
            st["q_norm"] = 1 + 0.2 * torch.randn(d, device="cuda", generator=gen)
            st["k_norm"] = 1 + 0.2 * torch.randn(d, device="cuda", generator=gen)
    else:
        lens = _cached_lengths(case)
        rows = (case["batch"], case["tq"], hq)
        q = torch.randn(*rows, d, device="cuda", generator=gen).to(torch.bfloat16)
        st.update(q=q, kv_len=_i32(lens), max_len=max(lens), out=torch.empty_like(q),
                  lse=torch.empty(rows, device="cuda"))
    st["table"], pages = _tables(gen, lens, page)
    st["kc"], st["ks"] = _pool(gen, pages, hkv, page, d)
    st["vc"], st["vs"] = _pool(gen, pages, hkv, page, d)
    if own:
        st["cache"] = _handle(st)
        if case["kind"] == "cached":
            n = _planner().attention_kv8_workspace(st["cache"])
            st["work"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return st


# ---- plain forms -------------------------------------------------------------------------

def _block_scale(amax):
    """2^e with the least e for which amax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    m, e = torch.frexp(amax.float())
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(amax == 0, torch.full_like(e, LOG_SCALE_MIN), e).clamp(LOG_SCALE_MIN, LOG_SCALE_MAX)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _codes(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _norm_rotate(x, weight, cos, sin, interleaved, eps=1e-6):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight
    half = cos.shape[-1]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    c, s = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        r = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([r, rest], -1)


def _owners(cu, n):
    """Sequence and index within it of each of n packed tokens."""
    at = torch.arange(n, device=cu.device)
    seq = torch.searchsorted(cu.long(), at, right=True) - 1
    return seq, at - cu.long()[seq]


def _append_one(x, codes, scale, page_of, off, st, page):
    """Tokens x [n, heads, dim] into the pages; earlier tokens of a page keep their values, on
    the page's new scale."""
    pages = scale.shape[0]
    dump = torch.full_like(page_of, pages)
    old = torch.cat([scale, scale[:1]])
    grown = old.clone()
    grown[torch.where(off == 0, page_of, dump)] = 2.0 ** LOG_SCALE_MIN     # pages begun by this call
    grown = grown.scatter_reduce(0, page_of[:, None].expand(-1, x.shape[1]), _block_scale(x.abs().amax(-1)),
                                 "amax", include_self=True)
    start = st["start"].long()
    tail = start % page
    begun = st["cu"][1:] > st["cu"][:-1]
    held = torch.where(begun & (tail > 0), st["table"].gather(1, (start // page).clamp(max=st["table"].shape[1] - 1)[:, None])[:, 0].long(), pages)
    spare = torch.cat([codes, codes[:1]])
    factor = old[held] / grown[held]
    kept = torch.arange(page, device=x.device)[None, :] < tail[:, None]
    before = spare[held]
    after = _codes(_values(before) * factor[:, :, None, None])
    spare[held] = torch.where(kept[:, None, :, None], after, before)
    spare[page_of, :, off] = _codes(x / grown[page_of][:, :, None])
    codes.copy_(spare[:pages])
    scale.copy_(grown[:pages])


def _read_one(codes, scale, page_of, off):
    return (_values(codes[page_of, :, off]) * scale[page_of][:, :, None]).to(torch.bfloat16)


def _append_plain(st):
    case, page = st["case"], st["case"]["page"]
    seq, i = _owners(st["cu"], st["q"].shape[0])
    pos = st["start"].long()[seq] + i
    cos, sin = st["rope"][pos].chunk(2, -1)
    q = _norm_rotate(st["q"], st["q_norm"], cos, sin, case["interleaved"]).to(torch.bfloat16)
    k = _norm_rotate(st["k"], st["k_norm"], cos, sin, case["interleaved"])
    page_of, off = st["table"][seq, pos // page].long(), pos % page
    _append_one(k, st["kc"], st["ks"], page_of, off, st, page)
    _append_one(st["v"].float(), st["vc"], st["vs"], page_of, off, st, page)
    seq, i = _owners(st["cu_window"], st["k_read"].shape[0])
    pos = st["first"].long()[seq] + i
    page_of, off = st["table"][seq, pos // page].long(), pos % page
    return {"q": q, "k": _read_one(st["kc"], st["ks"], page_of, off), "v": _read_one(st["vc"], st["vs"], page_of, off)}


def _softmax_product(s, v):
    """softmax(s) @ v over the last axis of s, zero rows where every score is -inf; and the
    logarithm of the rows' sums."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l == 0, torch.ones_like(l), l)
    return o, (m + torch.log(l))[..., 0]


def _cached_plain(st):
    case = st["case"]
    b, tq, hq, d = st["q"].shape
    hkv, page = case["kv_heads"], case["page"]
    rows = st["table"].long().clamp(min=0)
    def dense(codes, scale):
        x = _values(codes[rows]) * scale[rows][..., None, None]          # [b, pages, heads, page, d]
        return x.transpose(1, 2).reshape(b, hkv, -1, d)
    k, v = dense(st["kc"], st["ks"]), dense(st["vc"], st["vs"])
    q = st["q"].float().reshape(b, tq, hkv, -1, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    s = torch.matmul(q, k.transpose(2, 3)) * d ** -0.5
    n = st["kv_len"].long()[:, None]
    t = torch.arange(tq, device=n.device)[None, :]
    lim = (n - tq + t + 1) if case["causal"] else n.expand(-1, tq)
    lim = lim.repeat_interleave(hq // hkv, 1)[:, None, :, None]
    s = torch.where(torch.arange(s.shape[-1], device=n.device) < lim, s, -math.inf)
    v = torch.where((torch.arange(v.shape[2], device=n.device)[None, :] < n)[:, None, :, None], v, 0.0)
    o, lse = _softmax_product(s, v)
    o = o.reshape(b, hkv, tq, -1, d).permute(0, 2, 1, 3, 4).reshape(b, tq, hq, d)
    lse = lse.reshape(b, hkv, tq, -1).permute(0, 2, 1, 3).reshape(b, tq, hq)
    return {"out": o.to(torch.bfloat16), "lse": lse}


def _prompt_plain(st):
    case = st["case"]
    hkv, d, frame = case["kv_heads"], case["dim"], case["frame"]
    cu_q, cu_k = st["cu_q"].long(), st["cu_k"].long()
    nq, nk = (cu_q[1:] - cu_q[:-1])[:, None], (cu_k[1:] - cu_k[:-1])[:, None]
    i = torch.arange(st["max_q"], device="cuda")[None, :]
    j = torch.arange(st["max_k"], device="cuda")[None, :]
    def padded(x, cu, at):
        return x[(cu[:-1, None] + at).clamp(max=x.shape[0] - 1)].float()
    b, g = nq.shape[0], case["q_heads"] // hkv
    q = padded(st["q"], cu_q, i).reshape(b, -1, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    k = padded(st["k"], cu_k, j).transpose(1, 2)
    v = padded(st["v"], cu_k, j).transpose(1, 2)
    p = i + nk - nq
    lim = torch.where(p >= 0, torch.minimum(nk, (p.div(frame, rounding_mode="floor") + 1) * frame), 0)
    seen = (j[:, None, :] < lim[:, :, None])[:, None, None]               # [b, 1, 1, max_q, max_k]
    s = torch.matmul(q, k.transpose(2, 3)) * d ** -0.5
    s = s.view(b, hkv, g, -1, s.shape[-1]).masked_fill_(~seen, -math.inf).view_as(s)
    o, lse = _softmax_product(s, v)
    seq, at = _owners(st["cu_q"], st["q"].shape[0])
    o = o.view(b, hkv, g, -1, d)[seq, :, :, at].reshape(-1, hkv * g, d)
    lse = lse.view(b, hkv, g, -1)[seq, :, :, at].reshape(-1, hkv * g)
    return {"out": o.to(torch.bfloat16), "lse": lse}


def run(state):
    st, case = state, state["case"]
    kind = case["kind"]
    if not own:
        return {"append": _append_plain, "cached": _cached_plain, "prompt": _prompt_plain}[kind](st)
    p = _planner()
    if kind == "append":
        p.rope_append_kv8(st["q"], st["k"], st["v"], st["rope"], st["cu"], st["start"], st["cache"], st["q_out"],
                          q_norm=st["q_norm"], k_norm=st["k_norm"], interleaved=case["interleaved"])
        p.kv8_read(st["cache"], st["cu_window"], st["first"], st["k_read"], st["v_read"])
        return {"q": st["q_out"], "k": st["k_read"], "v": st["v_read"]}
    if kind == "cached":
        p.attention_kv8(st["q"], st["cache"], st["kv_len"], st["out"], case["dim"] ** -0.5, st["work"],
                        causal=case["causal"], lse=st["lse"])
    else:
        p.attention_packed(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], st["out"], case["dim"] ** -0.5,
                           frame=case["frame"], lse=st["lse"])
    return {"out": st["out"], "lse": st["lse"]}


# ---- the definitions in 64 bits -----------------------------------------------------------

def _power(e):
    """2^e in 64 bits for whole numbers e, from its bits (a library's pow may be off by one)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(x):
    """x in 64 bits rounded to the nearest e4m3 value (ties to even), saturating."""
    _, e = torch.frexp(x)
    step = _power((e - 4).clamp(min=-9))
    return ((x / step).round() * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_append(case, st):
    new, old = _append_lengths(case)
    page, rot = case["page"], case["rot"]
    inv = 10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))

    def rotated(x, w, pos):
        x = x.double()
        if w is not None:
            x = x * w.double() / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6) ** 0.5
        a = (pos[:, None] * inv)[:, None, :]
        y = x.clone()
        y[..., first] = x[..., first] * a.cos() - x[..., second] * a.sin()
        y[..., second] = x[..., second] * a.cos() + x[..., first] * a.sin()
        return y

    qs, ks, vs, at = [], [], [], 0
    for s, (n, o) in enumerate(zip(new, old)):
        pos = torch.arange(o, o + n, device="cuda", dtype=torch.float64)
        rows = slice(at, at + n)
        at += n
        qs.append(rotated(st["q"][rows], st["q_norm"], pos))
        for x, codes, scale, got in ((rotated(st["k"][rows], st["k_norm"], pos), st["kc"], st["ks"], ks),
                                     (st["v"][rows].double(), st["vc"], st["vs"], vs)):
            lo, hi = o // page, -(-(o + n) // page)
            ids = st["table"][s, lo:hi].long()
            held = _values(codes[ids]).double().transpose(1, 2)            # [pages, page, heads, d]
            before = scale[ids].double()                                   # [pages, heads]
            full = torch.zeros((hi - lo) * page, *x.shape[1:], dtype=torch.float64, device="cuda")
            full[o - lo * page:o - lo * page + n] = x
            full = full.view(hi - lo, page, *x.shape[1:])
            most = full.abs().amax((1, 3))
            e = torch.ceil(torch.log2(most.clamp(min=2.0 ** -60) / E4M3_MAX)).clamp(LOG_SCALE_MIN, LOG_SCALE_MAX)
            e = torch.where(most <= E4M3_MAX * _power(e - 1), e - 1, e).clamp(min=LOG_SCALE_MIN)
            after = _power(e)
            if o % page:
                after[0] = torch.maximum(after[0], before[0])
            vals = _e4m3(full / after[:, None, :, None]) * after[:, None, :, None]
            vals = vals.reshape(-1, *x.shape[1:])
            if o % page:
                was = held[0, :o % page]
                back = _e4m3(was * (before[0] / after[0])[None, :, None]) * after[0][None, :, None]
                vals[:o % page] = back
            got.append(vals[:o + n - lo * page])
    return {"q": torch.cat(qs), "k": torch.cat(ks), "v": torch.cat(vs)}


def _exact_rows(q, k, v, lim, factor):
    """One sequence: q [n, hq, d], k, v [m, hkv, d], query i sees keys [0, lim[i])."""
    g = q.shape[1] // k.shape[1]
    out, lse = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    hidden = torch.arange(k.shape[0], device="cuda")[None, :] >= lim[:, None]
    some = lim > 0
    step = max(1, (1 << 27) // max(1, k.shape[0]))
    for h in range(q.shape[1]):
        for a in range(0, q.shape[0], step):
            rows = slice(a, a + step)
            s = (q[rows, h].double() @ k[:, h // g].double().T * factor).masked_fill(hidden[rows], -math.inf)
            lse[rows, h] = torch.logsumexp(s, -1)
            w = torch.where(some[rows, None], torch.exp(s - lse[rows, h, None]), 0.0)
            out[rows, h] = w @ v[:, h // g].double()
    return out, lse


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "append":
        return _exact_append(case, st)
    outs, lses = [], []
    if case["kind"] == "prompt":
        at_q = at_k = 0
        for a, b in zip(*_prompt_lengths(case)):
            p = torch.arange(b - a, b, device="cuda")
            lim = torch.clamp((torch.div(p, case["frame"], rounding_mode="floor") + 1) * case["frame"], max=b)
            o, l = _exact_rows(st["q"][at_q:at_q + a], st["k"][at_k:at_k + b], st["v"][at_k:at_k + b], lim, case["dim"] ** -0.5)
            outs.append(o)
            lses.append(l)
            at_q, at_k = at_q + a, at_k + b
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}
    for s, n in enumerate(_cached_lengths(case)):
        ids = st["table"][s, :-(-n // case["page"])].long()
        k, v = ((_values(c[ids]).double() * sc[ids].double()[:, :, None, None]).transpose(1, 2).reshape(-1, case["kv_heads"], case["dim"])[:n]
                for c, sc in ((st["kc"], st["ks"]), (st["vc"], st["vs"])))
        t = torch.arange(case["tq"], device="cuda")
        lim = (n - case["tq"] + 1 + t).clamp(min=0) if case["causal"] else torch.full_like(t, n)
        o, l = _exact_rows(st["q"][s], k, v, lim, case["dim"] ** -0.5)
        outs.append(o)
        lses.append(l)
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
