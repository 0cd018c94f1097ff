"""The oracle of eviction, key weights and positions against their definition, by small cases worked by hand."""
import math

import numpy as np

from oracle import fp8


def test_choose_takes_the_most_recent_and_the_heaviest_in_order():
    w = np.array([3, 1, 3, 9, 0, 2, 0.5])
    assert fp8.choose(w, 7, 3, 0).tolist() == [0, 2, 3]
    assert fp8.choose(w, 7, 3, 2).tolist() == [3, 5, 6]
    assert fp8.choose(w, 7, 4, 2).tolist() == [0, 3, 5, 6]  # of the two 3s the earlier
    assert fp8.choose(w, 7, 2, 2).tolist() == [5, 6]
    assert fp8.choose(w, 2, 3, 2).tolist() == [0, 1]
    assert fp8.choose(w, 0, 3, 2).tolist() == []


def test_choose_orders_special_values():
    w = np.array([math.nan, -1, -math.inf, math.inf, -0.0, 0.0])
    assert fp8.choose(w, 6, 1, 0).tolist() == [3]
    assert fp8.choose(w, 6, 2, 0).tolist() == [3, 4]  # -0 equals 0
    assert fp8.choose(w, 6, 5, 0).tolist() == [1, 2, 3, 4, 5]


def test_evict_scales_and_codes():
    rng = np.random.default_rng(0)
    cache = fp8.encode(rng.standard_normal((256, 576)) * 64)
    scales = np.array([2.0 ** -3, 2.0 ** -9, 1, 1], np.float32)
    before = cache.copy()
    w = np.zeros((1, 128), np.float32)
    w[0, [3, 70]] = 1
    kept, lens, nw = fp8.evict(cache, scales, w, [[0, 1]], [128], [[3]], 3, 1, 64)
    assert kept.tolist() == [[3, 70, 127]] and lens.tolist() == [3] and nw.tolist() == [[1, 1, 0]]
    assert np.array_equal(cache[:192], before[:192]) and np.array_equal(cache[195:], before[195:])
    old = fp8.decode_codes(before[[3, 70, 127]]) * np.array([2.0 ** -3, 2.0 ** -9, 2.0 ** -9])[:, None]
    s = float(scales[3])
    assert math.log2(s) % 1 == 0 and np.abs(old).max() <= 448 * s and np.abs(old).max() > 448 * s / 2
    # rounded again: half a step of e4m3 (2^-4 relative, 2^-10 below its normal range) in the new scale
    assert np.all(np.abs(fp8.decode_codes(cache[192:195]) * s - old) <= np.maximum(2.0 ** -4 * np.abs(old), 2.0 ** -10 * s))


def test_key_weights_of_one_head_sum_to_one():
    rng = np.random.default_rng(1)
    cache, scales = fp8.encode(rng.standard_normal((128, 576)) * 64), np.full(2, 2.0 ** -6, np.float32)
    q = rng.standard_normal((1, 3, 576))
    lse = fp8.decode(q, cache, scales, 0.07, [[1, 0]], [100], 64)[1]
    out, tol = fp8.key_weights(q, cache, scales, 0.07, lse, [[1, 0]], [100], 64, np.zeros((1, 120)))
    assert abs(out.sum() - 3) < 1e-12 and np.all(out[0, 100:] == 0) and np.all(tol[0, 100:] == 0) and np.all(tol[0, :100] > 0)


def test_append_at_turns_by_position():
    rng = np.random.default_rng(2)
    cs = np.concatenate([np.cos(np.arange(50)[:, None] * np.ones(32)), np.sin(np.arange(50)[:, None] * np.ones(32))], 1)
    cs = cs.astype(np.float32)
    kv, pe = rng.standard_normal((2, 512)), rng.standard_normal((2, 64))
    a, b = (np.zeros((64, 576), np.uint8) for _ in range(2))
    sa, sb = np.ones(1, np.float32), np.ones(1, np.float32)
    fp8.append(a, sa, kv, pe, cs, [0, 2], [7], [[0]], 64, True, positions=[30])
    fp8.append(b, sb, kv, pe, np.roll(cs, -23, 0), [0, 2], [7], [[0]], 64, True)
    assert np.array_equal(a, b) and np.array_equal(sa, sb)
