"""The append to the 4-bit cache at the ends of the number range, against the oracle.

What decides a code is defined in fp32 operation by operation, so codes and scales are compared for equality
(test_gpu_kv4.py)."""
import numpy as np
import pytest
import torch

from oracle import four_bit
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
