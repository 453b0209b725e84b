"""Workloads of the 4-bit paged key/value cache, its eviction, and the norm ahead of 8-bit products.

Four kinds of case:
  * "norm": residual addition, RMS norm and e4m3 codes with a scale a row, as the 8-bit linear
    layers take them;
  * "append": queries and keys are normalised per head and rotated, keys and values go into a paged
    cache as e2m1 codes with an e4m3 scale for every 16 elements, and are read back as bf16;
  * "cached": attention of one or a few new tokens per sequence over that cache, and, where asked for, the
    weight that each cached token received, added to what it had before;
  * "evict": the tokens with the largest weights and the latest ones move to fresh pages, and are
    read back.

``run`` computes a case in plain torch operations (``own`` false) or through the library.
"""
import functools
import math
import random

import torch

own = False

E2M1_MAX, E4M3_MAX = 6.0, 448.0
BLOCK = 16                                # elements that share a scale
SCALE_MIN = 2.0 ** -9                     # the least e4m3 value above zero
NORM_EPS = 1e-6


# ---- cases -------------------------------------------------------------------------------

def listed():
    return [
        # one token ahead of a projection: latency
        dict(name="norm_1x1024", kind="norm", rows=1, cols=1024, x="f32", delta="bf16", half=False),
        # 24 frames of 258 tokens of the full predictor's width, behind an fp32 projection
        dict(name="norm_frames_24", kind="norm", rows=6192, cols=1024, x="f32", delta="f32", half=False),
        # packed prompts of a wide model with a bf16 residual, the bf16 rows wanted as well
        dict(name="norm_4099x8192", kind="norm", rows=4099, cols=8192, x="bf16", delta="bf16", half=True),
        # one serving step of a batch, sequences of all lengths
        dict(name="append_step_64", kind="append", batch=64, new_lo=1, new_hi=1, old_lo=0, old_hi=4096,
             q_heads=32, kv_heads=8, dim=128, page=64, rot=128, interleaved=False, norm=True, mix=2),
        # packed prompts of different lengths
        dict(name="append_prompts", kind="append", batch=9, new_lo=100, new_hi=4500, old_lo=0,
             old_hi=700, q_heads=32, kv_heads=8, dim=128, page=64, rot=128, interleaved=False,
             norm=True, mix=4),
        # one sequence of a few frames: latency
        dict(name="cached_1x517", kind="cached", batch=1, tq=1, len_lo=517, len_hi=517, q_heads=16,
             kv_heads=16, dim=64, page=32, causal=True, weights=False, mix=5),
        # a serving batch of ragged lengths
        dict(name="cached_32_ragged", kind="cached", batch=32, tq=1, len_lo=100, len_hi=8000, q_heads=32,
             kv_heads=8, dim=128, page=64, causal=True, weights=False, mix=6),
        # two long contexts
        dict(name="cached_2_long", kind="cached", batch=2, tq=1, len_lo=100001, len_hi=130001,
             q_heads=64, kv_heads=8, dim=128, page=128, causal=True, weights=False, mix=7),
        # action and state token of 256 candidates over three frames of 258 tokens, weights kept
        dict(name="cached_candidates_w", kind="cached", batch=256, tq=2, len_lo=776, len_hi=776, q_heads=16,
             kv_heads=16, dim=64, page=16, causal=False, weights=True, mix=8),
        # ragged long sequences whose caches are going to be cut: weights kept
        dict(name="cached_16_w", kind="cached", batch=16, tq=1, len_lo=4000, len_hi=30000, q_heads=32,
             kv_heads=8, dim=128, page=64, causal=True, weights=True, mix=9),
        # eight episodes of a few frames back to two frames' worth
        dict(name="evict_8", kind="evict", batch=8, len_lo=517, len_hi=2001, kv_heads=16, dim=64, page=32,
             keep=516, recent=258, mix=10),
        # long contexts back to a budget; the shortest is within it
        dict(name="evict_6_long", kind="evict", batch=6, len_lo=5001, len_hi=70001, kv_heads=8, dim=128, page=64,
             keep=8192, recent=513, mix=11),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    kind = rng.choice(("norm", "append", "cached", "cached", "evict"))
    while True:
        dim = rng.choice((64, 128))
        kv = rng.choice((1, 2, 3, 4, 5, 8, 16))
        group = rng.choice((1, 1, 2, 3, 4, 6, 7, 8))
        case = dict(kind=kind, mix=rng.randrange(1 << 20))
        if kind == "norm":
            case.update(rows=_log_int(rng, 1, 20000), cols=16 * _log_int(rng, 1, 1024),
                        x=rng.choice(("f32", "bf16")), delta=rng.choice(("f32", "bf16", "none")),
                        half=rng.random() < 0.5)
        else:
            case.update(kv_heads=kv, dim=dim, page=rng.choice((16, 32, 64, 128)))
        if kind == "append":
            long = rng.random() < 0.5
            lo = _log_int(rng, 1, 400) if long else 1
            case.update(batch=_log_int(rng, 1, 12 if long else 256), new_lo=lo,
                        new_hi=lo + _log_int(rng, 1, 4000) if long else rng.choice((1, 1, 2, 3)),
                        old_lo=0, old_hi=_log_int(rng, 1, 4000), q_heads=kv * group,
                        rot=16 * rng.randint(1, dim // 16), interleaved=rng.random() < 0.5,
                        norm=rng.random() < 0.5)
        elif kind == "cached":
            lo = _log_int(rng, 1, 60000)
            case.update(batch=_log_int(rng, 1, 256), tq=rng.choice((1, 1, 1, 2, 3, 4, 8)), len_lo=lo,
                        len_hi=lo + _log_int(rng, 1, 60000), q_heads=kv * group,
                        causal=rng.random() < 0.7, weights=rng.random() < 0.5)
        elif kind == "evict":
            lo, keep = _log_int(rng, 1, 40000), _log_int(rng, 1, 16000)
            case.update(batch=_log_int(rng, 1, 128), len_lo=lo, len_hi=lo + _log_int(rng, 1, 40000),
                        keep=keep, recent=rng.choice((0, 1, keep, rng.randint(0, keep))))
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
    if case["kind"] == "norm":
        return case["rows"] * case["cols"]
    if case["kind"] == "append":
        return sum(_append_lengths(case)[0]) * (case["q_heads"] + case["kv_heads"]) * case["dim"]
    lens = _lengths(case)
    if case["kind"] == "cached":
        return case["batch"] * case["kv_heads"] * max(lens) * case["dim"]
    return case["batch"] * case["kv_heads"] * max(max(lens), min(case["keep"], max(lens)) * case["dim"])


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


def _lengths(case):
    return _spread(case["len_lo"], case["len_hi"], case["batch"], case["mix"])


def _kept(case):
    return [min(n, case["keep"]) for n in _lengths(case)]


def work(case):
    if case["kind"] == "norm":
        size = {"f32": 4, "bf16": 2, "none": 0}
        n = case["rows"] * case["cols"]
        byts = n * (2 * size[case["x"]] + size[case["delta"]] + 1 + 2 * case["half"])
        return {"bytes": byts + 4 * case["rows"] + 4 * case["cols"], "flops": 7 * n}
    d, hkv = case["dim"], case["kv_heads"]
    held = 2 * hkv * (d // 2 + d // BLOCK)                   # bytes of a cached token
    if case["kind"] == "append":
        n, hq = sum(_append_lengths(case)[0]), case["q_heads"]
        byts = n * (2 * (hq + 2 * hkv) * d + 2 * hq * d + held + 4 * case["rot"] + 4 * hkv * d)
        return {"bytes": byts, "flops": 8 * n * (hq + 2 * hkv) * d}
    lens = _lengths(case)
    if case["kind"] == "evict":
        n = sum(_kept(case))
        byts = 4 * hkv * sum(lens) + n * (2 * held + 4 * hkv * d + 4 * hkv)
        return {"bytes": byts, "flops": 4 * hkv * sum(lens)}
    hq = case["q_heads"]
    rows = case["batch"] * case["tq"] * hq
    seen = sum(max(0, n - case["tq"] + t + 1) if case["causal"] else n for n in lens for t in range(case["tq"]))
    byts = sum(lens) * (held + 8 * hkv * case["weights"]) + rows * d * 4 + rows * 4
    byts += sum(-(-n // case["page"]) for n in lens) * 4
    return {"bytes": byts, "flops": 4 * d * hq * seen}


# ---- inputs ------------------------------------------------------------------------------

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


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


def _units(gen, heads):
    """Powers of two near the heads' magnitudes, as a calibration leaves them."""
    return 2.0 ** torch.randint(-2, 2, (heads,), device="cuda", generator=gen).float()


def _pool(gen, pages, heads, page, dim, unit):
    """Pages already filled: packed codes and scales."""
    codes = torch.empty(pages, heads, page, dim // 2, dtype=torch.uint8, device="cuda")
    scale = torch.empty(pages, heads, page, dim // BLOCK, dtype=torch.float8_e4m3fn, device="cuda")
    size = torch.rand(1, heads, 1, 1, device="cuda", generator=gen) * 1.5 + 0.25
    step = max(1, (1 << 26) // (heads * page * dim))
    for a in range(0, pages, step):
        x = torch.randn(min(step, pages - a), heads, page, dim, device="cuda", generator=gen) * size
        codes[a:a + step], scale[a:a + step] = _quantise(x, unit[:, None, None])
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


def _handle(st, table):
    from cem_search_transformer_gb300 import binding
    return binding.KvCache4(st["kc"], st["vc"], st["ks"], st["vs"], table, st["k_unit"], st["v_unit"])


def _scratch(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case=case)
    if own:
        _planner()
    if case["kind"] == "norm":
        rows, cols = case["rows"], case["cols"]
        size = torch.exp(0.7 * torch.randn(rows, 1, device="cuda", generator=gen))   # tokens differ in magnitude
        st["x"] = (torch.randn(rows, cols, device="cuda", generator=gen) * size).to(_TYPES[case["x"]])
        st["delta"] = None
        if case["delta"] != "none":
            st["delta"] = (0.3 * torch.randn(rows, cols, device="cuda", generator=gen)).to(_TYPES[case["delta"]])
        st["w"] = 1 + 0.2 * torch.randn(cols, device="cuda", generator=gen)
        st["x_out"] = torch.empty_like(st["x"])
        st["codes"] = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
        st["scales"] = torch.empty(rows, device="cuda")
        st["y"] = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda") if case["half"] else None
        return st
    d, hkv, page = case["dim"], case["kv_heads"], case["page"]
    st["k_unit"], st["v_unit"] = _units(gen, hkv), _units(gen, hkv)
    if case["kind"] == "append":
        hq = case["q_heads"]
        new, old = _append_lengths(case)
        lens = [a + b for a, b in zip(new, old)]
        qkv = _heads(gen, sum(new), hq + 2 * hkv, d)   # one projection's rows: strided q, k, v
        st.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], cu=_cumulative(new),
                  start=_i32(old), rope=_rotary_table(max(lens), case["rot"]), q_norm=None, k_norm=None,
                  q_out=torch.empty(sum(new), hq, d, dtype=torch.bfloat16, device="cuda"),
                  k_read=torch.empty(sum(new), hkv, d, dtype=torch.bfloat16, device="cuda"),
                  v_read=torch.empty(sum(new), hkv, d, dtype=torch.bfloat16, device="cuda"))
        if case["norm"]:
            st["q_norm"] = 1 + 0.2 * torch.randn(d, device="cuda", generator=gen)
            st["k_norm"] = 1 + 0.2 * torch.randn(d, device="cuda", generator=gen)
    else:
        lens = _lengths(case)
        st.update(kv_len=_i32(lens), max_len=max(lens))
    st["table"], pages = _tables(gen, lens, page)
    there = st["table"].shape[1] * page
    if case["kind"] == "cached":
        rows = (case["batch"], case["tq"], case["q_heads"])
        q = torch.randn(*rows, d, device="cuda", generator=gen).to(torch.bfloat16)
        st.update(q=q, out=torch.empty_like(q), lse=torch.empty(rows, device="cuda"))
        if case["weights"]:
            st["mass"] = torch.rand(case["batch"], hkv, there, device="cuda", generator=gen) * 0.01
            st["mass_out"] = torch.zeros_like(st["mass"])
    if case["kind"] == "evict":
        # weights of many magnitudes; some tokens were never looked at, some alike
        mass = torch.exp(2.5 * torch.randn(case["batch"], hkv, there, device="cuda", generator=gen))
        st["mass"] = torch.where(mass < 0.1, 0.0, torch.where(mass < 0.2, 0.125, mass))
        kept = _kept(case)
        table, more = _tables(gen, kept, page)
        st["to_table"] = torch.where(table >= 0, table + pages, table)
        pages += more
        st.update(first=torch.zeros_like(st["kv_len"]), cu=_cumulative(kept), len_out=torch.zeros_like(st["kv_len"]),
                  mass_out=torch.zeros(case["batch"], hkv, table.shape[1] * page, device="cuda"),
                  k_read=torch.empty(sum(kept), hkv, d, dtype=torch.bfloat16, device="cuda"),
                  v_read=torch.empty(sum(kept), hkv, d, dtype=torch.bfloat16, device="cuda"))
    st["kc"], st["ks"] = _pool(gen, pages, hkv, page, d, st["k_unit"])
    st["vc"], st["vs"] = _pool(gen, pages, hkv, page, d, st["v_unit"])
    if own:
        st["cache"] = _handle(st, st["table"])
        if case["kind"] == "cached":
            st["work"] = _scratch(_planner().attention_kv4_workspace(st["cache"]))
        if case["kind"] == "evict":
            st["to"] = _handle(st, st["to_table"])
            st["work"] = _scratch(_planner().kv4_evict_workspace(st["cache"], case["keep"]))
    return st


# ---- plain forms -------------------------------------------------------------------------

def _quantise(x, unit):
    """Packed e2m1 codes (the even element in the low half of a byte) and e4m3 scales of rows x
    [..., dim] in fp32, `unit` broadcast against [..., dim / 16]."""
    b = x.unflatten(-1, (-1, BLOCK))
    s = (b.abs().amax(-1).double() / E2M1_MAX / unit).float()      # a sixth by a product in 32 bits leaves ties to chance
    s = s.clamp(SCALE_MIN, E4M3_MAX).to(torch.float8_e4m3fn)
    y = b / (s.float() * unit)[..., None]
    m = y.abs()
    c = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
         + 8 * (y < 0)).to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), s


def _values(codes, scale, unit):
    """What packed codes [..., dim / 2] with scales [..., dim / 16] stand for, in fp32."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat([table, -table])
    x = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)
    return (x.unflatten(-1, (-1, BLOCK)) * (scale.float() * unit)[..., None]).flatten(-2)


def _norm_plain(st):
    s = st["x"].float()
    if st["delta"] is not None:
        s = s + st["delta"].float()
    y = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + NORM_EPS) * st["w"]
    top = y.abs().amax(-1, keepdim=True)
    scale = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    codes = (y * torch.where(top > 0, E4M3_MAX / top, torch.ones_like(top))).clamp(-E4M3_MAX, E4M3_MAX)
    got = {"x": s.to(st["x"].dtype), "codes": codes.to(torch.float8_e4m3fn), "scales": scale[:, 0]}
    if st["y"] is not None:
        got["y"] = y.to(torch.bfloat16)
    return got


def _norm_rotate(x, weight, cos, sin, interleaved):
    """Heads x [n, heads, dim] in fp32. The norm's factor is computed in 64 bits and rounded once: what
    is quantised next lies next to borders."""
    x = x.float()
    if weight is not None:
        r = torch.rsqrt((x.double() ** 2).mean(-1, keepdim=True) + NORM_EPS).float()
        x = x * (r * weight)
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


def _append_plain(st):
    case, page = st["case"], st["case"]["page"]
    seq, i = _owners(st["cu"], st["q"].shape[0])
    pos = st["start"].long()[seq] + i
    cos, sin = st["rope"][pos].chunk(2, -1)
    q = _norm_rotate(st["q"], st["q_norm"], cos, sin, case["interleaved"]).to(torch.bfloat16)
    k = _norm_rotate(st["k"], st["k_norm"], cos, sin, case["interleaved"])
    page_of, off = st["table"][seq, pos // page].long(), pos % page
    ku, vu = st["k_unit"][:, None], st["v_unit"][:, None]
    st["kc"][page_of, :, off], st["ks"].view(torch.uint8)[page_of, :, off] = _bytes(_quantise(k, ku))
    st["vc"][page_of, :, off], st["vs"].view(torch.uint8)[page_of, :, off] = _bytes(_quantise(st["v"].float(), vu))
    return {"q": q, "k": _read(st["kc"], st["ks"], ku, page_of, off), "v": _read(st["vc"], st["vs"], vu, page_of, off)}


def _bytes(quantised):
    return quantised[0], quantised[1].view(torch.uint8)


def _read(codes, scale, unit, page_of, off):
    scale = scale.view(torch.uint8)[page_of, :, off].view(torch.float8_e4m3fn)
    return _values(codes[page_of, :, off], scale, unit).to(torch.bfloat16)


def _cached_plain(st):
    case = st["case"]
    b, tq, hq, d = st["q"].shape
    hkv = case["kv_heads"]
    rows = st["table"].long().clamp(min=0)

    def dense(codes, scale, unit):
        scale = scale.view(torch.uint8)[rows].view(torch.float8_e4m3fn)
        x = _values(codes[rows], scale, unit[:, None, None])                 # [b, pages, heads, page, d]
        return x.transpose(1, 2).reshape(b, hkv, -1, d)
    q = st["q"].float().reshape(b, tq, hkv, -1, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    s = torch.matmul(q, dense(st["kc"], st["ks"], st["k_unit"]).transpose(2, 3)) * d ** -0.5
    n = st["kv_len"].long()[:, None]
    j = torch.arange(s.shape[-1], device=n.device)
    t = torch.arange(tq, device=n.device)[None, :]
    lim = (n - tq + t + 1) if case["causal"] else n.expand(-1, tq)
    lim = lim.repeat_interleave(hq // hkv, 1)[:, None, :, None]
    s = torch.where(j < lim, s, -math.inf)
    v = dense(st["vc"], st["vs"], st["v_unit"])
    there = j < n                                                            # [b, keys]
    v = torch.where(there[:, None, :, None], v, 0.0)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    w = p / torch.where(l == 0, torch.ones_like(l), l)
    o = torch.matmul(w, v).reshape(b, hkv, tq, -1, d).permute(0, 2, 1, 3, 4).reshape(b, tq, hq, d)
    lse = (m + torch.log(l))[..., 0].reshape(b, hkv, tq, -1).permute(0, 2, 1, 3).reshape(b, tq, hq)
    got = {"out": o.to(torch.bfloat16), "lse": lse}
    if case["weights"]:
        got["mass"] = torch.where(there[:, None, :], 0.98 * st["mass"] + w.sum(2), st["mass_out"])
    return got


def _evict_plain(st):
    case, page = st["case"], st["case"]["page"]
    n = st["kv_len"].long()[:, None]
    j = torch.arange(st["mass"].shape[-1], device=n.device)[None, :]
    keep = n.clamp(max=case["keep"])
    late = j >= n - case["recent"]
    rank = torch.where(late[:, None], math.inf, st["mass"])
    rank = torch.where((j < n)[:, None], rank, -1.0)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices        # ties: the lowest first
    place = torch.arange(st["mass_out"].shape[-1], device=n.device)
    order = torch.nn.functional.pad(order, (0, max(0, place.numel() - order.shape[-1])))[..., :place.numel()]
    inside = (place[None, :] < keep)[:, None]                                 # [b, 1, kept]
    token = torch.sort(torch.where(inside, order, j.shape[-1]), -1).values    # [b, heads, kept]
    token = torch.where(inside, token, 0)
    mass = torch.where(inside, st["mass"].gather(-1, token), 0.0)
    seq, i = _owners(st["cu"], st["k_read"].shape[0])
    token = token[seq, :, i]                                                  # [kept in all, heads]
    head = torch.arange(case["kv_heads"], device=n.device)[None, :]
    page_of, off = st["table"][seq[:, None], token // page].long(), token % page

    def moved(codes, scale, unit):
        scale = scale.view(torch.uint8)[page_of, head, off].view(torch.float8_e4m3fn)
        return _values(codes[page_of, head, off], scale, unit[:, None]).to(torch.bfloat16)
    return {"k": moved(st["kc"], st["ks"], st["k_unit"]), "v": moved(st["vc"], st["vs"], st["v_unit"]),
            "mass": mass, "len": keep[:, 0].to(torch.int32)}


def run(state):
    st, case = state, state["case"]
    kind = case["kind"]
    if not own:
        return {"norm": _norm_plain, "append": _append_plain, "cached": _cached_plain, "evict": _evict_plain}[kind](st)
    p = _planner()
    if kind == "norm":
        p.add_rmsnorm_fp8(st["x"], st["delta"], st["w"], st["x_out"], st["codes"], st["scales"], eps=NORM_EPS, y=st["y"])
        got = {"x": st["x_out"], "codes": st["codes"], "scales": st["scales"]}
        return {**got, "y": st["y"]} if case["half"] else got
    if kind == "append":
        p.rope_append_kv4(st["q"], st["k"], st["v"], st["rope"], st["cu"], st["start"], st["cache"], st["q_out"],
                          q_norm=st["q_norm"], k_norm=st["k_norm"], norm_eps=NORM_EPS, interleaved=case["interleaved"])
        p.kv4_read(st["cache"], st["cu"], st["start"], st["k_read"], st["v_read"])
        return {"q": st["q_out"], "k": st["k_read"], "v": st["v_read"]}
    if kind == "cached":
        got = {"out": st["out"], "lse": st["lse"]}
        if not case["weights"]:
            p.attention_kv4(st["q"], st["cache"], st["kv_len"], st["out"], case["dim"] ** -0.5, st["work"],
                            causal=case["causal"], lse=st["lse"])
            return got
        p.attention_kv4(st["q"], st["cache"], st["kv_len"], st["out"], case["dim"] ** -0.5, st["work"],
                        causal=case["causal"], lse=st["lse"], mass=st["mass"], mass_out=st["mass_out"], decay=0.98)
        return {**got, "mass": st["mass_out"]}
    p.kv4_evict(st["cache"], st["kv_len"], st["mass"], case["keep"], case["recent"], st["to"], st["len_out"],
                st["mass_out"], st["work"])
    p.kv4_read(st["to"], st["cu"], st["first"], st["k_read"], st["v_read"])
    return {"k": st["k_read"], "v": st["v_read"], "mass": st["mass_out"], "len": st["len_out"]}


# ---- the definitions in 64 bits -----------------------------------------------------------

def _e4m3(x):
    """x >= 0 in 64 bits rounded to the nearest e4m3 value (ties to even), saturating."""
    _, e = torch.frexp(x)
    e = (e - 4).clamp(min=-9)
    step = ((e.long() + 1023) << 52).view(torch.float64)      # 2^e from its bits: a library's pow may be off by one
    return ((x / step).round() * step).clamp(-E4M3_MAX, E4M3_MAX)


def _block_values(x, unit):
    """x [n, heads, dim] in 64 bits as the cache holds it."""
    out = torch.empty_like(x)
    for b in range(x.shape[-1] // BLOCK):
        part = x[..., BLOCK * b:BLOCK * (b + 1)]
        s = _e4m3(part.abs().amax(-1, keepdim=True) / (6 * unit)).clamp(min=SCALE_MIN) * unit
        m = (part / s).abs()
        step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).double()
        out[..., BLOCK * b:BLOCK * (b + 1)] = torch.sign(part) * ((m / step).round() * step).clamp(max=6) * s
    return out


def _unpacked(codes, scale, unit):
    """Values in 64 bits of packed codes [n, heads, dim / 2], arithmetic in place of a table."""
    c = torch.stack([codes % 16, codes // 16], -1).flatten(-2).double()
    sign, m = 1 - 2 * (c >= 8).double(), c % 8
    mag = torch.where(m < 2, m / 2, (2 + m % 2) * 2.0 ** ((m // 2) - 2))
    return sign * mag * scale.double().repeat_interleave(BLOCK, -1) * unit.double()[:, None]


def _exact_norm(case, st):
    s = st["x"].double() + (st["delta"].double() if st["delta"] is not None else 0)
    y = s * st["w"].double() / ((s ** 2).sum(-1, keepdim=True) / s.shape[-1] + NORM_EPS) ** 0.5
    top = y.abs().max(-1, keepdim=True).values
    codes = y / top * E4M3_MAX
    got = {"x": s, "codes": torch.sign(codes) * _e4m3(codes.abs()), "scales": top[:, 0] / E4M3_MAX}
    return {**got, "y": y} if case["half"] else got


def _exact_append(case, st):
    new, old = _append_lengths(case)
    rot = case["rot"]
    inv = 10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
    pos = torch.cat([torch.arange(o, o + n, device="cuda", dtype=torch.float64) for n, o in zip(new, old)])
    a = (pos[:, None] * inv)[:, None, :]

    def rotated(x, w):
        x = x.double()
        if w is not None:
            x = x * w.double() / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + NORM_EPS) ** 0.5
        y = x.clone()
        y[..., first] = x[..., first] * a.cos() - x[..., second] * a.sin()
        y[..., second] = x[..., second] * a.cos() + x[..., first] * a.sin()
        return y
    return {"q": rotated(st["q"], st["q_norm"]), "k": _block_values(rotated(st["k"], st["k_norm"]), st["k_unit"].double()[:, None]),
            "v": _block_values(st["v"].double(), st["v_unit"].double()[:, None])}


def _sequence(st, s, n):
    """Keys and values of sequence s in 64 bits, [n, heads, dim] each."""
    page = st["case"]["page"]
    ids = st["table"][s, :-(-n // page)].long()

    def one(codes, scale, unit):
        c = codes[ids].transpose(1, 2).flatten(0, 1)[:n]
        e = scale.view(torch.uint8)[ids].view(torch.float8_e4m3fn).transpose(1, 2).flatten(0, 1)[:n]
        return _unpacked(c, e, unit)
    return one(st["kc"], st["ks"], st["k_unit"]), one(st["vc"], st["vs"], st["v_unit"])


def _exact_cached(case, st):
    tq, g = case["tq"], case["q_heads"] // case["kv_heads"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(out.shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    mass = st["mass_out"].double() if case["weights"] else None
    for s, n in enumerate(_lengths(case)):
        k, v = _sequence(st, s, n)
        t = torch.arange(tq, device="cuda")
        lim = (n - tq + 1 + t).clamp(min=0) if case["causal"] else torch.full_like(t, n)
        lim = lim.repeat_interleave(g)[None, :, None]
        q = st["q"][s].double().unflatten(1, (-1, g)).transpose(0, 1).flatten(1, 2)      # [heads, tq g, dim]
        z = torch.einsum("hrd,nhd->hrn", q, k) / case["dim"] ** 0.5
        z = z.masked_fill(torch.arange(n, device="cuda") >= lim, -math.inf)
        l = torch.logsumexp(z, -1)
        w = torch.where(lim > 0, torch.exp(z - l[..., None]), 0.0)
        out[s] = torch.einsum("hrn,nhd->hrd", w, v).unflatten(1, (tq, g)).transpose(0, 1).flatten(1, 2)
        lse[s] = l.unflatten(1, (tq, g)).transpose(0, 1).flatten(1, 2)
        if case["weights"]:
            mass[s, :, :n] = 0.98 * st["mass"][s, :, :n].double() + w.sum(1)
    return {"out": out, "lse": lse, "mass": mass} if case["weights"] else {"out": out, "lse": lse}


def _exact_evict(case, st):
    ks, vs, mass = [], [], torch.zeros(st["mass_out"].shape, dtype=torch.float64, device="cuda")
    for s, n in enumerate(_lengths(case)):
        k, v = _sequence(st, s, n)
        keep, late = min(n, case["keep"]), min(n, case["recent"])
        m = st["mass"][s, :, :n].double()
        need, chosen = keep - late, torch.ones(m.shape, dtype=torch.bool, device="cuda")
        if keep < n:
            old = m[:, :n - late]
            border = torch.sort(old, -1, descending=True).values[:, need - 1:need] if need else torch.full_like(old[:, :1], math.inf)
            above = old > border
            equal = (old == border) if need else torch.zeros_like(above)
            chosen[:, :n - late] = above | (equal & (equal.cumsum(-1) <= need - above.sum(-1, keepdim=True)))
        at = chosen.nonzero()[:, 1].view(case["kv_heads"], keep)
        heads = torch.arange(case["kv_heads"], device="cuda")[:, None]
        ks.append(k[at, heads].transpose(0, 1))
        vs.append(v[at, heads].transpose(0, 1))
        mass[s, :, :keep] = m.gather(1, at)
    return {"k": torch.cat(ks), "v": torch.cat(vs), "mass": mass,
            "len": torch.tensor([min(n, case["keep"]) for n in _lengths(case)], device="cuda")}


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "cached": _exact_cached, "evict": _exact_evict}[case["kind"]](case, st)
