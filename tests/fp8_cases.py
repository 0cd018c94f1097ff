"""Cases of the e4m3 decode where its operands' 8-bit terms show, and a
float64 model of those terms.

The kernel holds a query feature x (divided by 2^e, the smallest power that
brings its head's largest to at most 448) as e4m3(x) + e4m3(16 (x - e4m3(x))) / 16,
and a weight p = s 2^(x - m), rounded to f16, whose largest is 2^4 or more, as p1 = e4m3(p) and
  up to 32 heads: e4m3(16 (p - p1 + o)) / 16,
  more heads:     e5m2 of p - p1 + o rounded to a multiple of 2^-13 (where below 2^-4),
with an offset o that runs evenly through a step of 2^-13 over 32 keys.
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


def e5m2(x):
    return _cast(x, torch.float8_e5m2)


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


# the kernel's order: the lane's five bits reversed
OFFSET = (np.array([int(f"{i:05b}"[::-1], 2) for i in range(32)]) + 0.5) / 32 - 0.5


def weight_model(p, heads, steps=True, offsets=True):
    """What the terms hold of p [heads, n] (key j in lane j % 32).  steps False: without the multiples of 2^-13; offsets
    False: without o."""
    o = OFFSET[np.arange(p.shape[-1]) % 32] * (2.0 ** -13 if offsets else 0)
    p = f16(p)
    p1 = e4m3(p)
    if heads <= 32:
        return p1 + e4m3(f16(16 * (p - p1) + 16 * o)) / 16
    r = f16(p - p1 + o)
    if steps:
        r = f16(f16(r + 0.1875) - 0.1875)
    return p1 + e5m2(r)


def decode_model(q, k, s, heads, tail=None, **kw):
    """Attention of q [heads, 576] over codes k [n, 576] of one scale s, its weights through their terms; out in bf16."""
    x = (q @ k.T) * (s * SCALE)
    w = np.exp(x - x.max(1, keepdims=True))
    p = weight_model(16 * w, heads, **kw) / 16
    if tail is not None:  # key 17 is the peak
        p = np.where(np.arange(p.shape[1]) == 17, p, tail * p)
    return torch.from_numpy(p @ k[:, :512] * s / w.sum(1, keepdims=True)).bfloat16().double().numpy()


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


def peak_over_tail(heads, n, gap):
    """Key 17 `gap` above n - 1 of equal score, all values around a common vector; (q, codes, scale)."""
    rng = np.random.default_rng(n + heads)
    k = np.zeros((n, 576))
    k[:, :512] = e4m3(rng.standard_normal((1, 512)) * 60 + rng.standard_normal((n, 512)) * 20)
    k[17, 512] = 448
    s = 2.0 ** -7
    q = np.zeros((1, heads, 576))
    q[:, :, 512] = gap / (448 * s * SCALE)
    return torch.from_numpy(q).bfloat16(), k, s


def check_tail(out, q, k, s, what):
    """The tail's part P of the softmax, from what of out [heads, 512] the peak's part p0 does not explain, along the
    tail's mean value u: (out - p0 v0) . u / u . u.  Off by at most
      the output's rounding     sum |u_i| half_ulp(out_i) / u . u
      relative errors           2^-8 + 2^-12 (two terms, f16) and 2 (e^d - 1) (scores off by d) of P and p0 |v0 . u| / u . u
      the terms' absolute step  2^-13 of a largest weight of 2^4 or more.  Of 32 equal weights the 32 offsets take the
                                nearest number up: their sum is within half a step.  The last 32 keys and the peak's count
                                a step each, and a key's own error, a step at most, counts as far as its value along u
                                differs from the mean's."""
    x = (q @ k.T) * (s * SCALE)
    p = np.exp(x - x.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    v = k[:, :512] * s
    tail = np.delete(np.arange(len(k)), 17)
    u = v[tail].mean(0)
    along = v @ u / (u @ u)
    part, peak = p[:, tail].sum(1), p[:, 17]
    got = out @ u / (u @ u) - peak * along[17]
    d = (np.abs(q) @ np.abs(k).T).max(1) * (s * SCALE) * 2.0 ** -24 * 584
    tol = (np.maximum(bf16_half_ulp(out), bf16_half_ulp(p @ v)) @ np.abs(u) / (u @ u)
           + (2.0 ** -8 + 2.0 ** -12 + 2 * np.expm1(d)) * (part + peak * abs(along[17]))
           + 2.0 ** -17 * peak * (len(k) / 64 + 64 + np.abs(along[tail] - 1).sum()))
    worst = float(np.max(np.abs(got - part) / tol))
    print(f"[fp8 decode] {what}: a tail of {part[0]:.4f} off by {float(np.max(np.abs(got / part - 1))):.4f} of it, tolerance "
          f"{float(np.max(tol / part)):.4f}, {worst:.3f} of the tolerance")
    assert worst <= 1, f"{what}: the tail is off by {worst:.2f} times the tolerance"


def alternating_tail(heads, n, gap):
    """One key `gap` above n - 1 whose values follow the sign of their lane's offset; (q, codes, scale)."""
    k = np.zeros((n, 576))
    k[:, :512] = np.where(OFFSET[np.arange(n) % 32] > 0, 448.0, -448.0)[:, None]
    k[17, :512] = e4m3(np.random.default_rng(n).uniform(1, 2, 512))
    k[17, 512] = 448
    s = 2.0 ** -7
    q = np.zeros((1, heads, 576))
    q[:, :, 512] = gap / (448 * s * SCALE)
    return torch.from_numpy(q).bfloat16(), k, s


def check_alternating(out, q, k, s, what):
    """out [heads, 512] of such keys.  A weight w (of a largest of 2^4) is within 2^-8 of itself and f16's rounding, and
    where the terms' step is absolute within that step, 2^-13: half of it by rounding, half by the offset.  One below
    2^-19 is zero: the largest offset, 31/64 of the step, does not take it to half of one."""
    x = (q @ k.T) * (s * SCALE)
    w = 16 * np.exp(x - x.max(1, keepdims=True))
    v = k[:, :512] * s
    o = w @ v / w.sum(1, keepdims=True)
    off = np.where(w < 2.0 ** -19, w, (2.0 ** -8 + 2.0 ** -12) * w + 2.0 ** -25 + np.where(w < 2.0 ** -5, 2.0 ** -13, 0))
    tol = np.maximum(bf16_half_ulp(o), bf16_half_ulp(out)) + off @ np.abs(v) / w.sum(1, keepdims=True)
    worst = float(np.max(np.abs(out - o) / tol))
    print(f"[fp8 decode] {what}: {worst:.3f} of the tolerance")
    assert worst <= 1, f"{what}: {worst:.2f} times the tolerance"
