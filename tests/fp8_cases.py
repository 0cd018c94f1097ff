"""Cases of the e4m3 decode where its operands' 8-bit terms show, and a
float64 model of those terms.

The kernel holds a query feature x (divided by 2^e, the smallest power that
brings its head's largest to at most 448) as e4m3(x) + e4m3(16 (x - e4m3(x))) / 16.
"""
import math

import numpy as np
import torch

from oracle import fp8
from tests.helpers import bf16_half_ulp

SCALE = 1.0 / math.sqrt(192.0)


def _cast(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).double().numpy()


def e4m3(x):
    return _cast(x, torch.float8_e4m3fn)


def f16(x):
    return _cast(x, torch.float16)


def query_model(q, gain=16.0):
    """What the terms hold of q [..., 576]; gain 1 is a second term without its factor."""
    amax = np.abs(q).max(-1, keepdims=True)
    e = np.ceil(np.log2(np.maximum(amax, 1e-300) / 448))
    x = f16(q * 2.0 ** -e)
    q1 = e4m3(x)
    return (q1 + e4m3(gain * (x - q1)) / gain) * 2.0 ** e


def query_floor(q):
    """How far query_model may be from q: where a feature is below 2^-6 of the scaled head, its first term has a step of
    2^-9 and the second one of 2^-13, so half of that, and half a step of f16's, 2^-24; nothing elsewhere."""
    amax = np.abs(q).max(-1, keepdims=True)
    up = 2.0 ** np.ceil(np.log2(np.maximum(amax, 1e-300) / 448))
    return np.where(np.abs(q) < 2.0 ** -6 * up, (2.0 ** -14 + 2.0 ** -25) * up, 0)


def wide_query(heads, ratio):
    """Queries [1, heads, 576] with one feature `ratio` times the others, which lie in [1, 2), and codes [300, 576] of
    keys that are zero there.  Up to a ratio of 2^13 every feature is exact in its two terms: 224 < largest 2^-e, so that
    a scaled feature is above 2^-6, and of one in [2^E, 2^(E + 1)) the first term leaves up to eight steps of 2^(E - 7):
    16 times that is a multiple of e4m3's smallest step, 2^-9."""
    rng = np.random.default_rng(int(ratio) + heads)
    q = rng.choice([-1.0, 1.0], (1, heads, 576)) * (1 + rng.integers(0, 128, (1, heads, 576)) / 128)
    at = rng.integers(0, 576, heads)
    q[0, np.arange(heads), at] = ratio
    k = e4m3(rng.standard_normal((300, 576)) * 32)
    k[:, at] = 0
    return torch.from_numpy(q).bfloat16(), k


def place(k, page=64):
    """Codes k [n, 576] in a cache: (bytes, table)."""
    n = len(k)
    blocks = -(-n // page) * page // 64
    cache = np.zeros((blocks * 64, 576), np.uint8)
    cache[:n] = fp8.encode(k)
    return cache, np.arange(-(-n // page), dtype=np.int32)[None]


def check_scores(out, q, k, s, heads, what):
    """out [heads, 512] of q over codes k of one scale s.  Off by at most bf16's rounding, the weights' 2^-8 and their
    absolute floor (tests/test_gpu_fp8.py derives both), and what the scores' errors move: fp32 sums, and query_floor."""
    x = (q @ k.T) * (s * SCALE)
    p = np.exp(x - x.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    v = k[:, :512] * s
    o, oabs = p @ v, p @ np.abs(v)
    d = (np.abs(q) @ np.abs(k).T).max(1) * (s * SCALE) * 2.0 ** -24 * 584 + (query_floor(q) @ np.abs(k).T).max(1) * (s * SCALE)
    tol = np.maximum(bf16_half_ulp(o), bf16_half_ulp(out)) + (2.0 ** -8 + 2 * np.expm1(d))[:, None] * oabs
    tol = tol + 2.0 ** -17 * p.max(1)[:, None] * np.abs(v).sum(0)
    worst = float(np.max(np.abs(out - o) / tol))
    print(f"[fp8 decode] {what}: {worst:.3f} of the tolerance, relative 2-norm {np.linalg.norm(out - o) / np.linalg.norm(o):.2e}")
    assert worst <= 1, f"{what}: {worst:.2f} times the tolerance"
