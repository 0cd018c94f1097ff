"""The 8-bit oracle against closed forms and torch's float8_e4m3fn cast."""
import numpy as np
import torch

from oracle import fp8


def test_encode_against_torch_cast():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * np.exp2(rng.integers(-12, 9, 20000)), fp8._MIDS, -fp8._MIDS,
                        fp8._GRID, [0.0, -0.0]]).astype(np.float32)
    x = np.clip(x, -448, 448)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp8.encode(x), ref)
    assert list(fp8.encode([500.0, -np.inf, np.nan])) == [0x7E, 0xFE, 0x7F]


def test_decode_codes_all():
    c = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(fp8.decode_codes(c), ref, equal_nan=True)


def test_block_scale():
    for amax, e in ((0.0, -60), (448.0, 0), (448.0001, 1), (224.0, -1), (1.0, -8), (1e30, 60), (np.inf, 60)):
        assert fp8.block_scale(amax) == 2.0 ** e


def test_rotation_is_a_turn():
    rng = np.random.default_rng(1)
    x, a = rng.standard_normal((5, 64)), rng.standard_normal((5, 32))
    cs = np.concatenate([np.cos(a), np.sin(a)], 1)
    il, hs = fp8.rotate(x, cs, True), fp8.rotate(x, cs, False)
    z = (x[:, 0::2] + 1j * x[:, 1::2]) * np.exp(1j * a)
    assert np.allclose(il[:, 0::2], z.real, atol=1e-5) and np.allclose(il[:, 1::2], z.imag, atol=1e-5)
    order = np.concatenate([np.arange(0, 64, 2), np.arange(1, 64, 2)])
    assert np.allclose(fp8.rotate(x[:, order], cs, False), il[:, order], atol=1e-5)
    assert np.allclose(np.linalg.norm(hs, axis=1), np.linalg.norm(x, axis=1), rtol=1e-5)


def test_append_grows_and_restarts():
    cs = np.tile(np.concatenate([np.ones(32), np.zeros(32)]), (256, 1)).astype(np.float32)
    cache, scales = np.zeros((128, 576), np.uint8), np.zeros(2, np.float32)
    table = np.array([[1]])
    one = np.ones((1, 512), np.float32)
    pe = np.ones((1, 64), np.float32)
    fp8.append(cache, scales, one, pe, cs, [0, 1], [0], table, 64, True)
    assert scales[1] == 2.0 ** -8 and np.all(fp8.decode_codes(cache[64]) == 256)
    fp8.append(cache, scales, 1000 * one, pe, cs, [0, 1], [1], table, 64, True)  # 1000 <= 448 * 4
    assert scales[1] == 4 and np.all(fp8.decode_codes(cache[64]) * 4 == 1)
    assert np.all(fp8.decode_codes(cache[65, :512]) * 4 == 1024)  # 250 to e4m3: 256
    fp8.append(cache, scales, one, pe, cs, [0, 1], [0], table, 64, True)  # the first token again: anew
    assert scales[1] == 2.0 ** -8 and scales[0] == 0


def test_gemm_and_quantize_close():
    rng = np.random.default_rng(2)
    x, y = rng.standard_normal((3, 300)), rng.standard_normal((130, 300))
    a, sa = fp8.quantize(x)
    w = np.zeros((130, 300), np.uint8)
    sw = np.zeros((2, 3), np.float32)
    for i in range(2):
        for j in range(3):
            blk = y[128 * i:128 * (i + 1), 128 * j:128 * (j + 1)]
            sw[i, j] = np.abs(blk).max() / 448
            w[128 * i:128 * (i + 1), 128 * j:128 * (j + 1)] = fp8.encode(blk / sw[i, j])
    c, mag = fp8.gemm(a, sa, w, sw)
    assert np.all(np.abs(c - x @ y.T) <= 2 * 2.0 ** -4 * mag * 1.2)


def test_decode_against_brute_force():
    rng = np.random.default_rng(3)
    cache, scales = fp8.encode(rng.standard_normal((128, 576)) * 50), np.array([2.0 ** -6, 2.0 ** -5], np.float32)
    q = rng.standard_normal((1, 2, 576))
    out, lse, _, _ = fp8.decode(q, cache, scales, 0.05, np.array([[1, 0]]), [100], 64)
    k = fp8.decode_codes(cache) * np.repeat(scales, 64)[:, None]
    k = np.concatenate([k[64:], k[:36]])
    w = np.exp(q[0] @ k.T * 0.05)
    assert np.allclose(out[0], w @ k[:, :512] / w.sum(1, keepdims=True)) and np.allclose(lse[0], np.log(w.sum(1)))
