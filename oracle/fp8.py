"""The 8-bit path: the e4m3 latent cache with one power-of-two scale per
block of 64 tokens, attention over it, and the e4m3 quantiser and GEMM with
scales per block of 128.  Codes and scales evaluate their definition in
float32 (as the NVFP4 oracle does); everything else is float64."""
from __future__ import annotations

import math

import numpy as np

from . import nvfp4

BLOCK = 64
GROUP = 128
_GRID = nvfp4.e4m3_decode(np.arange(0x7F))  # 0 .. 448, ascending
_MIDS = (_GRID[:-1] + _GRID[1:]) / 2


def encode(x) -> np.ndarray:
    """x to e4m3 codes: nearest, ties to the even code, saturating; NaN is 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    lo = np.searchsorted(_MIDS, a, side="left")  # a at a midpoint goes to the lower code ...
    tie = (lo < len(_MIDS)) & (a == _MIDS[np.minimum(lo, len(_MIDS) - 1)])
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo)  # ... unless that one is odd
    return np.where(np.isnan(x), 0x7F, code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def decode_codes(codes) -> np.ndarray:
    c = np.asarray(codes, dtype=np.uint8)
    v = nvfp4.e4m3_decode(np.where((c & 0x7F) == 0x7F, 0, c))
    return np.where((c & 0x7F) == 0x7F, np.nan, v)


def rotate(x, cos_sin, interleaved: bool) -> np.ndarray:
    """float32 x [..., 64] turned by cos_sin [..., 64], every product and sum rounded to float32."""
    x = np.asarray(x, dtype=np.float32)
    c, s = np.asarray(cos_sin, np.float32)[..., :32], np.asarray(cos_sin, np.float32)[..., 32:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    u, v = a * c - b * s, b * c + a * s
    if interleaved:
        return np.stack([u, v], -1).reshape(x.shape)
    return np.concatenate([u, v], -1)


def block_scale(amax: float) -> float:
    e = -60
    while e < 60 and not amax <= 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(cache, scales, kv_c, k_pe, cos_sin, cu, ctx, table, page_size, interleaved) -> None:
    """In place on cache (uint8 [slots, 576]) and scales (float32)."""
    for b in range(len(ctx)):
        n = int(cu[b + 1] - cu[b])
        pos = int(ctx[b]) + np.arange(n)
        key = np.concatenate([np.asarray(kv_c[cu[b]:cu[b + 1]], np.float32),
                              rotate(k_pe[cu[b]:cu[b + 1]], cos_sin[pos], interleaved)], 1)
        for blk in sorted(set((pos // BLOCK).tolist())):
            rows = key[pos // BLOCK == blk]
            first = int(pos[pos // BLOCK == blk][0])
            slot = int(table[b][first // page_size]) * page_size + first % page_size
            g, off = slot // BLOCK, slot % BLOCK
            a = np.abs(rows)
            need = block_scale(float(np.max(np.where(np.isnan(a), 0, a))))
            was = float(scales[g])
            keep = off > 0 and 2.0 ** -60 <= was <= 2.0 ** 60
            new = max(was, need) if keep else need
            if keep and new != was:
                old = cache[slot - off:slot]
                cache[slot - off:slot] = encode(decode_codes(old) * (was / new))
            scales[g] = new
            cache[slot:slot + len(rows)] = encode(rows.astype(np.float64) / new)


def decode(q, cache, scales, softmax_scale, table, lens, page_size):
    """(out, lse, softmax @ |v|, largest p s times the sum of |k8|) in float64; q float [B, H, 576]."""
    B, H, _ = q.shape
    out, lse, oabs, flat = np.zeros((B, H, 512)), np.full((B, H), -np.inf), np.zeros((B, H, 512)), np.zeros((B, H, 512))
    for b in range(B):
        keys = []
        for t in range(int(lens[b])):
            page = int(table[b][t // page_size])
            slot = page * page_size + t % page_size
            if page < 0 or slot // BLOCK >= len(scales) or not 2.0 ** -60 <= scales[slot // BLOCK] <= 2.0 ** 60:
                continue
            keys.append(slot)
        if not keys:
            continue
        keys = np.asarray(keys)
        k = decode_codes(cache[keys]) * np.asarray(scales, np.float64)[keys // BLOCK][:, None]
        s = np.asarray(q[b], np.float64) @ k.T * softmax_scale
        m = s.max(1, keepdims=True)
        p = np.exp(s - m)
        z = p.sum(1, keepdims=True)
        out[b], oabs[b] = p @ k[:, :512] / z, p @ np.abs(k[:, :512]) / z
        lse[b] = (m + np.log(z))[:, 0]
        s = np.asarray(scales, np.float64)[keys // BLOCK]
        flat[b] = np.max(p / z * s, 1)[:, None] * np.abs(k[:, :512] / s[:, None]).sum(0)
    return out, lse, oabs, flat


def quantize(x):
    """(codes uint8, scales float32) of x [M, K]: float32 quotients."""
    x = np.asarray(x, np.float32)
    M, K = x.shape
    codes, scales = np.zeros((M, K), np.uint8), np.zeros((M, math.ceil(K / GROUP)), np.float32)
    for j in range(scales.shape[1]):
        g = x[:, GROUP * j:GROUP * (j + 1)]
        a = np.abs(g)
        with np.errstate(invalid="ignore", divide="ignore"):
            s = np.maximum(np.max(np.where(np.isnan(a), 0, a), 1) / np.float32(448), np.float32(2.0 ** -126))
            codes[:, GROUP * j:GROUP * (j + 1)] = encode(g / s[:, None])
        scales[:, j] = s
    return codes, scales


def gemm(a, a_scales, w, w_scales):
    """(product, product of magnitudes) in float64."""
    K, N = a.shape[1], w.shape[0]
    sa = np.repeat(np.asarray(a_scales, np.float64), GROUP, 1)[:, :K]
    sw = np.repeat(np.repeat(np.asarray(w_scales, np.float64), GROUP, 0)[:N], GROUP, 1)[:, :K]
    x, y = decode_codes(a) * sa, decode_codes(w) * sw
    return x @ y.T, np.abs(x) @ np.abs(y).T
