"""Residual addition, RMS norm and e4m3 codes against the oracle in 64 bits.

Tolerances, derived before the first run. e = 2^-24, half a step of fp32.
  * s = x + delta: one rounding, e; as bf16 2^-8 more.
  * The mean of squares: the squares' sums are chains of at most 8 fused products, four partial sums
    and a tree of at most 5 + 31 additions (warps, then up to 32 of them), all positive, so at most 48 e of the sum, with
    s's own rounding (2 e) and the division; half of that after the root: 26 e, and two more for root
    and reciprocal. y: 2 e for the products. In all 32 e |y|.
  * scale = max|y| / 448: 34 e. A code stands for y / scale rounded to half a step, 2^-4 relative or 2^-10
    absolute below 2^-6; the quotient itself carries 4 e. So code * scale is off by 2^-4 |y| + 2^-10
    scale + 40 e |y|."""
import numpy as np
import pytest
import torch

from gpu_helpers import make_planner  # noqa: F401 (the suite's helpers are importable)
from oracle import four_bit

pytestmark = pytest.mark.gpu

E, BF16 = 2.0 ** -24, 2.0 ** -8
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def planner():
    from cem_search_transformer_gb300 import binding, synthetic
    p = binding.Planner(synthetic.PRESETS["tiny"])       # an fp32 context serves as well
    yield p
    p.close()


def f64(t):
    return t.detach().double().cpu().numpy()


def run(planner, x, delta, w, eps=1e-6, half=True, codes=True, in_place=False, stream=None):
    rows, cols = x.shape
    x_out = x if in_place else torch.full((rows, cols), 9.0, dtype=x.dtype, device="cuda")
    c = torch.full((rows, cols), 0x55, dtype=torch.uint8, device="cuda") if codes else None
    s = torch.full((rows,), 9.0, device="cuda") if codes else None
    y = torch.full((rows, cols), 9.0, dtype=torch.bfloat16, device="cuda") if half else None
    planner.add_rmsnorm_fp8(x, delta, w, x_out, c, s, eps=eps, y=y, stream=stream)
    return x_out, c, s, y


def check(x, delta, w, got, eps=1e-6):
    x_out, c, s, y = got
    want, norm = four_bit.add_rmsnorm(f64(x), None if delta is None else f64(delta), f64(w), eps)
    tol = np.abs(want) * (E if x_out.dtype == torch.float32 else BF16 + E)
    assert np.all(np.abs(f64(x_out) - want) <= tol)
    if y is not None:
        assert np.all(np.abs(f64(y) - norm) <= (BF16 + 32 * E) * np.abs(norm) + 1e-38)
    if c is not None:
        scale, top = f64(s), np.abs(norm).max(-1)
        assert np.all(np.abs(scale - np.where(top > 0, top / 448, 1)) <= 34 * E * top / 448)   # 1 for a row of zeros
        value = f64(c.view(torch.float8_e4m3fn).float()) * scale[:, None]
        assert np.all(np.abs(value - norm) <= (2.0 ** -4 + 40 * E) * np.abs(norm) + 2.0 ** -10 * scale[:, None])


def inputs(rows, cols, x, delta, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = torch.randn(rows, cols, device="cuda", generator=g) * torch.exp(torch.randn(rows, 1, device="cuda", generator=g))
    d = None if delta == "none" else torch.randn(rows, cols, device="cuda", generator=g).to(TYPES[delta])
    return a.to(TYPES[x]), d, 1 + 0.3 * torch.randn(cols, device="cuda", generator=g)


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 32), (1, 1024), (9, 1040), (33, 384), (700, 1024), (5, 4096),
                                       (2, 4112), (37, 8192), (3, 16000), (2, 16400), (3, 32768)])
@pytest.mark.parametrize("x,delta", [("f32", "bf16"), ("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "none")])
def test_matches_oracle(planner, rows, cols, x, delta):
    a, d, w = inputs(rows, cols, x, delta, seed=rows + cols)
    check(a, d, w, run(planner, a, d, w))
    planner.sync_check()


@pytest.mark.parametrize("half,codes", [(True, False), (False, True)])
def test_outputs_left_out(planner, half, codes):
    a, d, w = inputs(40, 512, "f32", "bf16")
    check(a, d, w, run(planner, a, d, w, half=half, codes=codes))
    full = run(planner, a, d, w)
    planner.add_rmsnorm_fp8(a, d, w, None, full[1], full[2])
    check(a, d, w, full)


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_in_place_and_columns_of_wider_rows(planner, x):
    wide, d, w = inputs(21, 3 * 256, x, "bf16", seed=4)
    a = wide[:, 256:512]
    others = wide.clone()
    want = run(planner, a, d[:, 512:], w[:256].clone())
    check(a, d[:, 512:], w[:256], want)
    got = run(planner, a, d[:, 512:], w[:256].clone(), in_place=True)
    for g, r in zip((a, *got[1:]), want):
        assert torch.equal(g, r)
    assert torch.equal(wide[:, :256], others[:, :256]) and torch.equal(wide[:, 512:], others[:, 512:])


def test_zeros_and_far_magnitudes(planner):
    a, _, w = inputs(6, 256, "f32", "none", seed=2)
    a = a / a.abs().amax(1, keepdim=True)
    a *= torch.tensor([0.0, 1e-30, 1e-12, 1.0, 1e12, 1e18], device="cuda")[:, None]
    check(a, None, w, run(planner, a, None, w))
    got = run(planner, a, None, w)
    assert not (got[1][0] & 0x7f).any() and got[2][0] == 1.0        # zeros of either sign
    tiny = a[3:4] * 1e-37                                    # 448 / max|s w| has no fp32 value
    x_out, c, s, y = run(planner, tiny, None, w)
    _, norm = four_bit.add_rmsnorm(f64(tiny), None, f64(w), 1e-6)
    # the sum of squares vanishes and eps stands alone; a code's step is 2^-126 r at most, 2^-3 relative
    value = f64(c.view(torch.float8_e4m3fn).float()) * f64(s)[:, None]
    assert np.all(np.abs(value - norm) <= 2.0 ** -4 * (1 + 2.0 ** -20) * np.abs(norm) + 2.0 ** -136 * 1000 * 1.001)


def test_rows_that_are_not_finite_stay_alone(planner):
    a, d, w = inputs(5, 2048, "f32", "bf16", seed=3)
    want = run(planner, a, d, w)
    a[1, 77], a[3, 5] = float("nan"), float("inf")
    x_out, c, s, y = run(planner, a, d, w)
    planner.sync_check()
    for i in (0, 2, 4):
        for g, r in zip((x_out, c, s, y), want):
            assert torch.equal(g[i], r[i])
    value = c.view(torch.float8_e4m3fn).float() * s[:, None]
    assert torch.isnan(value[1]).all() and torch.isnan(y[1]).all()
    other = torch.arange(2048, device="cuda") != 5               # x / inf, and inf / inf
    assert torch.isnan(value[3, 5]) and not value[3, other].any()


def test_captured_on_another_stream_and_fed_to_the_fp8_product(planner):
    from cem_search_transformer_gb300 import binding, synthetic
    p = binding.Planner(synthetic.PRESETS["small"])
    a, d, w = inputs(130, 512, "f32", "bf16", seed=6)
    weight = torch.randn(256, 512, device="cuda")
    wc, ws = torch.empty(256, 512, dtype=torch.uint8, device="cuda"), torch.empty(256, device="cuda")
    p.quantize_rows_fp8(weight, 256, 512, wc, ws)
    x_out, c, s, y = run(p, a, d, w)
    out = torch.empty(130, 256, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        p.add_rmsnorm_fp8(a, d, w, x_out, c, s, y=y, stream=torch.cuda.current_stream())
        p.linear_fp8(c, s, wc, ws, None, 130, 256, 512, 0, out, stream=torch.cuda.current_stream())
    for seed in (7, 8):
        b, e, _ = inputs(130, 512, "f32", "bf16", seed=seed)
        a.copy_(b)
        d.copy_(e)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        check(a, d, w, (x_out, c, s, y))
        codes = f64(c.view(torch.float8_e4m3fn).float()) * f64(s)[:, None]
        want = codes @ (f64(wc.view(torch.float8_e4m3fn).float()) * f64(ws)[:, None]).T
        assert np.abs(f64(out) - want).max() <= 2e-5 * np.abs(want).max()
    p.sync_check()
    p.close()


def test_refusals(planner):
    from cem_search_transformer_gb300 import binding
    a, d, w = inputs(4, 64, "f32", "bf16")
    c, s = torch.empty(4, 64, dtype=torch.uint8, device="cuda"), torch.empty(4, device="cuda")
    ok = dict(x=a, delta=d, weight=w, x_out=torch.empty_like(a), codes=c, scales=s)
    planner.add_rmsnorm_fp8(**ok)
    wide = torch.zeros(4, 72, device="cuda")
    for change, match in ((dict(codes=None), "bad argument"), (dict(codes=None, scales=None), "bad argument"),
                          (dict(scales=s[:3]), "elements"), (dict(weight=w[:60]), "elements"), (dict(delta=d[:, :48]), "fit"),
                          (dict(x_out=d), "x_out"), (dict(x=a.half()), "dtype"), (dict(eps=-1.0), "bad argument"),
                          (dict(eps=float("nan")), "bad argument"), (dict(x=a.t()), "contiguous"),
                          (dict(x=wide[:, 1:65]), "bad argument"),                        # rows 4 bytes off
                          (dict(x=torch.zeros(4, 68, device="cuda")[:, :64]), "bad argument")):     # stride 68
        with pytest.raises(binding.JepaError, match=match):
            planner.add_rmsnorm_fp8(**{**ok, **change})
    for cols, match in ((24, "bad argument"), (32784, "columns")):
        x = torch.zeros(2, cols, device="cuda")
        with pytest.raises(binding.JepaError, match=match):
            planner.add_rmsnorm_fp8(x, None, torch.ones(cols, device="cuda"), x, torch.empty(2, cols, dtype=torch.uint8, device="cuda"),
                                    torch.empty(2, device="cuda"))
    planner.sync_check()
