"""The e4m3 decode where its operands' 8-bit terms show (tests/fp8_cases.py
has the cases and derives the tolerances)."""
import numpy as np
import pytest
import torch

from tests import fp8_cases as c
from tests.test_gpu_fp8 import check_decode, make_cache, run_decode

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def decode(q, k, s, **kw):
    cache, table = c.place(k)
    out, _, flags = run_decode(q, cache, np.full(len(cache) // 64, s, np.float32), table, (len(k),), 64, scale=c.SCALE, **kw)
    assert flags == 0
    return out[0].astype(np.float64)


@pytest.mark.parametrize("heads", [16, 40, 128])
@pytest.mark.parametrize("ratio", [2.0 ** 8, 2.0 ** 12, 2.0 ** 13, 2.0 ** 14, 2.0 ** 17])
def test_decode_one_feature_far_above_the_others(ratio, heads):
    q, k = c.wide_query(heads, ratio)
    for split in (True, False):
        c.check_scores(decode(q, k, 2.0 ** -6, split=split), q[0].double().numpy(), k, 2.0 ** -6, heads,
                       f"{heads} heads, ratio {ratio:.0f}, split={split}")


@pytest.mark.parametrize("heads", [8, 48])
def test_decode_features_spread_over_2_to_the_14(heads):
    rng = np.random.default_rng(heads)
    lens = (300, 70)
    cache, scales, table = make_cache(rng, lens, 64)
    q = torch.from_numpy(rng.standard_normal((2, heads, 576)) * np.exp2(rng.integers(-14, 1, (2, heads, 576)))).bfloat16()
    got = run_decode(q, cache, scales, table, lens, 64)
    check_decode(got, q, cache, scales, table, lens, 64, what=f"{heads} heads, spread 2^14")


@pytest.mark.parametrize("heads", [16, 40, 128])
@pytest.mark.parametrize("n,gap", [(500, 9.0), (2000, 14.0), (2000, 16.5), (8192, 30.0), (8192, 60.0)])
def test_decode_weights_of_zero_add_nothing(n, gap, heads):
    q, k, s = c.alternating_tail(heads, n, gap)
    for split in (True, False):
        c.check_alternating(decode(q, k, s, split=split), q[0].double().numpy(), k, s, f"{heads} heads, gap {gap}, split={split}")


@pytest.mark.parametrize("heads", [16, 40, 128])
@pytest.mark.parametrize("n,gap", [(3000, 6.0), (3000, 9.0), (20000, 10.4), (20000, 11.1), (20000, 12.0), (20000, 13.0)])
def test_decode_keeps_a_flat_tail(n, gap, heads):
    q, k, s = c.peak_over_tail(heads, n, gap)
    for split in (True, False):
        c.check_tail(decode(q, k, s, split=split), q[0].double().numpy(), k, s, f"{heads} heads, {gap} over {n}, split={split}")
