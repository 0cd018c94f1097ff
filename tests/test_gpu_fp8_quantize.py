"""The e4m3 quantiser where its quotients are delicate: codes and scales equal
the oracle's, which divides in float32."""
import numpy as np
import pytest
import torch

import mla_attention_nvfp4_gb300 as mla
from oracle import fp8
from tests.helpers import f32

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
DEV = "cuda:0"


def check(t):
    codes, scales = mla.mla_nvfp4_fp8_quantize(t.to(DEV))
    rc, rs = fp8.quantize(f32(t))
    assert np.array_equal(scales.cpu().numpy(), rs)
    got = codes.cpu().view(torch.uint8).numpy()
    assert np.array_equal(got, rc), f"{int((got != rc).sum())} codes differ"


def test_quantize_keeps_the_sign_of_zero():
    # among other numbers, alone in a group, and beside an infinity
    x = torch.randn(6, 512).bfloat16()
    x[:, ::3] = -0.0
    x[:, 1::3] = 0.0
    x[1, :128] = -0.0
    x[2, 5] = float("inf")
    check(x)


@pytest.mark.parametrize("power", [-133, -126, -118, -116, -113, -110, -100, -84, -57, -55, -30])
def test_quantize_tiny_groups(power):
    # quotients beside the midpoints of two codes: 17/16, 19/16 and 21/16 of a power of two, and values between
    rng = np.random.default_rng(-power)
    M = 2000
    amax = f32(torch.from_numpy(2.0 ** power * (1 + rng.integers(0, 128, M) / 128)).bfloat16()).astype(np.float64)[:, None]
    mid = rng.choice([17, 19, 21], (M, 128)) / 16 * 2.0 ** rng.integers(-9, 9, (M, 128)) / 448
    x = np.where(rng.random((M, 128)) < 0.5, mid, rng.uniform(0, 1, (M, 128))) * amax
    x = np.minimum(x, amax) * rng.choice([-1, 1], (M, 128))
    x[:, 5] = amax[:, 0]
    t = torch.from_numpy(x).bfloat16()
    check(t)
