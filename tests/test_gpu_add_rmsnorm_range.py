"""Residual addition, RMS norm and codes of rows whose squares leave fp32, against the oracle in 64 bits: the tolerances of
test_gpu_add_rmsnorm.py, of which nothing depends on the rows' magnitude."""
import numpy as np
import pytest
import torch

from oracle import four_bit
from test_gpu_add_rmsnorm import E, TYPES, check, f64, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def planner():
    from cem_search_transformer_gb300 import binding, synthetic
    p = binding.Planner(synthetic.PRESETS["tiny"])
    yield p
    p.close()


def far_rows(rows, cols, x, seed):
    """Rows of 1e19 to 3e38, some with one far element among ordinary ones, ordinary ones in between."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = torch.randn(rows, cols, device="cuda", generator=g)
    a /= a.abs().amax(1, keepdim=True)
    sizes = [1e19, 1.0, 3e19, 1e30, 3e38, 1.0, 1e25, 2.0 ** 55]
    a *= torch.tensor([sizes[i % len(sizes)] for i in range(rows)], device="cuda")[:, None]
    for i in range(5, rows, 8):
        a[i, (37 * i) % cols] = (-1) ** i * 1e38
    for i in range(2, rows, 8):
        a[i, :cols // 2] *= 2.0 ** -100                       # the far half beside the ordinary one
    return a.to(TYPES[x])


@pytest.mark.parametrize("rows,cols", [(9, 16), (17, 256), (9, 272), (8, 512), (19, 1024), (11, 4096), (8, 8192), (8, 16000), (6, 32768)])
@pytest.mark.parametrize("x,delta", [("f32", "none"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
def test_rows_past_the_squares_of_fp32(planner, rows, cols, x, delta):
    a = far_rows(rows, cols, x, rows + cols)
    d = None if delta == "none" else (0.25 * far_rows(rows, cols, "f32", 1)).to(TYPES[delta]) * 0.5
    w = 1 + 0.3 * torch.randn(cols, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    got = run(planner, a, d, w)
    planner.sync_check()
    check(a, d, w, got)
    again = run(planner, a.clone(), d, w, in_place=True)
    for g, r in zip(again, got):
        assert torch.equal(g, r)


@pytest.mark.parametrize("cols", [16, 256, 512, 1024, 4096, 8192, 16384, 32768])
@pytest.mark.parametrize("eps", [0.0, 1e-36])
def test_rows_below_them_without_an_epsilon(planner, cols, eps):
    g = torch.Generator(device="cuda").manual_seed(cols)
    a = torch.randn(8, cols, device="cuda", generator=g)
    a /= a.abs().amax(1, keepdim=True)
    a *= torch.tensor([1.0, 1e-12, 1e-20, 1e-25, 1e-36, 2e-38, 1e20, 3e38], device="cuda")[:, None]
    w = 1 + 0.3 * torch.randn(cols, device="cuda", generator=g)
    got = run(planner, a, None, w, eps=eps)
    planner.sync_check()
    check(a, None, w, got, eps=float(np.float32(eps)))


def test_rows_beside_far_ones_are_as_without_them(planner):
    """Rows that share a CTA, at every number of threads a row."""
    for cols in (256, 512, 1024):
        g = torch.Generator(device="cuda").manual_seed(cols)
        a, w = torch.randn(16, cols, device="cuda", generator=g), torch.ones(cols, device="cuda")
        want = run(planner, a, None, w)
        b = a.clone()
        b[::2] *= 1e30
        got = run(planner, b, None, w)
        for x, y in zip(got, want):
            assert torch.equal(x[1::2], y[1::2])
        zeros = torch.zeros(2, cols, device="cuda")                   # 0 / 0
        x_out, c, s, y = run(planner, zeros, None, w, eps=0.0)
        planner.sync_check()
        assert torch.isnan(y).all() and torch.isnan(c.view(torch.float8_e4m3fn).float()).all()
        _, norm = four_bit.add_rmsnorm(f64(b), None, f64(w), 1e-6)
        assert np.all(np.abs(f64(got[3]) - norm) <= (2.0 ** -8 + 32 * E) * np.abs(norm) + 1e-38)
