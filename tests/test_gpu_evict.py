"""Key weights and eviction from the e4m3 cache on the GPU, and the append
that goes on after it.

Eviction's choice, codes, scales and weights equal the oracle's: it evaluates a
definition of comparisons and float32 products by powers of two.  Key weights
are off by at most what oracle.fp8.key_weights derives (fp32 sums of exact
products, the hardware's exp2), and of what the queries' two 8-bit terms leave:
exact down to 2^-13 of a head's largest feature, 2^-21 of it below
(tests/fp8_cases.py states and tests that)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import mla_attention_nvfp4_gb300 as mla
from oracle import fp8
from tests.fp8_cases import query_floor
from tests.helpers import f32
from tests.test_gpu_fp8 import (DEV, F8, SCALE, angles, check_decode, errw, make_cache, pages_for, run_decode, same_codes,
                                u8)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def i32(a):
    return torch.tensor(list(a), dtype=torch.int32, device=DEV)


# -------------------------------------------------------------- key weights
def weigh(q, cache, scales, table, lens, page, lse, weights, out=None, scale=SCALE):
    e = errw()
    w = None if weights is None else t(np.asarray(weights, np.float32))
    o = mla.mla_nvfp4_fp8_key_weights(q.to(DEV), t(cache).view(F8), t(scales), scale, t(np.asarray(lse, np.float32)),
                                      page_table=t(table), seq_lens=i32(lens), page_size=page, weights=w,
                                      out=w if out is None and w is not None else out, error_word=e)
    torch.cuda.synchronize()
    return o.cpu().numpy(), int(e.item())


def check_weights(got, q, cache, scales, table, lens, page, lse, weights, what, scale=SCALE):
    ref, tol = fp8.key_weights(f32(q), cache, scales, scale, lse, table, lens, page, weights)
    # features below 2^-13 of their head's largest: part of the score's error
    floor = query_floor(f32(q))
    if floor.any():
        d = scale * floor.sum(2).max() * 448 * float(np.max(scales))
        tol = tol + 2 * np.expm1(d) * np.abs(ref)
    there = np.arange(ref.shape[1])[None] < np.asarray(lens)[:, None]
    assert np.array_equal(got[~there], np.asarray(weights, np.float32)[~there]), f"{what}: written past a length"
    worst = float(np.max(np.abs(got - ref)[there] / np.maximum(tol[there], 1e-37), initial=0))
    print(f"[key weights] {what}: {worst:.3f} of the tolerance")
    assert np.all(np.isfinite(got)) and worst <= 1, f"{what}: {worst:.2f} times the tolerance"


def step(rng, heads, lens, page, spread=0):
    cache, scales, table = make_cache(rng, lens, page, spread)
    q = torch.from_numpy(rng.standard_normal((len(lens), heads, 576))).bfloat16()
    lse = fp8.decode(f32(q), cache, scales, SCALE, table, lens, page)[1].astype(np.float32)
    return q, cache, scales, table, lse


@pytest.mark.parametrize("heads", [1, 5, 16, 31, 32, 33, 64, 65, 128, 130, 200])
def test_key_weights_heads(heads):
    rng = np.random.default_rng(heads)
    lens = (1, 0, 63, 64, 65, 127, 128, 129, 700)
    q, cache, scales, table, lse = step(rng, heads, lens, 64)
    w = rng.random((len(lens), 720)).astype(np.float32)
    got, flags = weigh(q, cache, scales, table, lens, 64, lse, w)
    assert flags == 0
    check_weights(got, q, cache, scales, table, lens, 64, lse, w, f"{heads} heads")


@pytest.mark.parametrize("page", [64, 128, 192, 1024])
@pytest.mark.parametrize("lens", [(5000,), (1, 3000, 77), (0, 0), (64,) * 40, (2, 0, 4097) * 3, (1,) * 160, (129,) * 330])
def test_key_weights_lengths(page, lens):
    rng = np.random.default_rng(page + len(lens))
    q, cache, scales, table, lse = step(rng, 24, lens, page, spread=3)
    w = np.zeros((len(lens), max(lens) + 1), np.float32)
    got, flags = weigh(q, cache, scales, table, lens, page, lse, w)
    assert flags == 0
    check_weights(got, q, cache, scales, table, lens, page, lse, w, f"page {page}, {len(lens)} sequences")


def test_key_weights_of_the_decode_sum_to_the_heads():
    rng = np.random.default_rng(3)
    lens = (3000, 17, 900)
    q, cache, scales, table, _ = step(rng, 16, lens, 64)
    lse = run_decode(q, cache, scales, table, lens, 64)[1]
    got, _ = weigh(q, cache, scales, table, lens, 64, lse, np.zeros((3, 3000), np.float32))
    # (the lse's own error, below 1e-4, moves every part by as much)
    assert np.allclose(got.sum(1), 16, rtol=1e-3)


def test_key_weights_outputs():
    rng = np.random.default_rng(4)
    lens = (200, 0, 65)
    q, cache, scales, table, lse = step(rng, 16, lens, 64)
    zero = np.zeros((3, 200), np.float32)
    base, _ = weigh(q, cache, scales, table, lens, 64, lse, zero)
    # nothing before it, a new result as wide as the page table
    alone, _ = weigh(q, cache, scales, table, lens, 64, lse, None)
    assert alone.shape == (3, table.shape[1] * 64) and np.array_equal(alone[:, :200], base) and not alone[:, 200:].any()
    # inside a wider tensor, apart from weights
    wide = torch.full((3, 300), 9.0, device=DEV)
    w = rng.random((3, 200)).astype(np.float32)
    e = errw()
    r = mla.mla_nvfp4_fp8_key_weights(q.to(DEV), t(cache).view(F8), t(scales), SCALE, t(lse), page_table=t(table),
                                      seq_lens=i32(lens), weights=t(w), out=wide[:, 50:250], error_word=e)
    torch.cuda.synchronize()
    assert r.data_ptr() == wide[:, 50:].data_ptr() and int(e.item()) == 0
    got = wide.cpu().numpy()
    assert np.all(got[:, :50] == 9) and np.all(got[:, 250:] == 9) and np.all(got[1] == 9)
    for b, n in enumerate(lens):
        assert np.all(got[b, 50 + n:250] == 9) and np.array_equal(got[b, 50:50 + n], w[b, :n] + base[b, :n])


def test_key_weights_bad_entries():
    rng = np.random.default_rng(5)
    lens = (200, 300, 150)
    q, cache, scales, table, lse = step(rng, 20, lens, 64)
    w = rng.random((3, 300)).astype(np.float32)
    good, _ = weigh(q, cache, scales, table, lens, 64, lse, w)
    for change in ("page", "page_neg", "scale", "length", "row"):
        tab, sc, ln, ww = table.copy(), scales.copy(), list(lens), w
        skipped = range(64, 128)
        if change == "page":
            tab[1, 1] = len(cache) // 64
        elif change == "page_neg":
            tab[1, 1] = -1
        elif change == "scale":
            sc[table[1, 1]] = 2.0 ** 61
        elif change == "length":
            tab, skipped = table[:, :4].copy(), range(256, 300)
        else:
            ww, skipped = w[:, :256].copy(), range(256, 256)
        got, flags = weigh(q, cache, sc, tab, ln, 64, lse, ww)
        assert flags == (4 if change == "scale" else 1), change
        ref = good[:, :ww.shape[1]].copy()
        ref[1, list(skipped)] = w[1, list(skipped)]
        assert np.array_equal(got, ref), change


def test_key_weights_nan_and_infinity():
    rng = np.random.default_rng(6)
    lens = (200, 300)
    q, cache, scales, table, lse = step(rng, 20, lens, 64)
    zero = np.zeros((2, 300), np.float32)
    good, _ = weigh(q, cache, scales, table, lens, 64, lse, zero)
    bad = cache.copy()
    bad[int(table[0][1]) * 64 + 7, 100] = 0x7F  # key 71 of sequence 0
    got, flags = weigh(q, bad, scales, table, lens, 64, lse, zero)
    assert flags == 0 and np.isnan(got[0, 71])
    assert np.array_equal(np.delete(got[0], 71), np.delete(good[0], 71)) and np.array_equal(got[1], good[1])
    for value in (float("inf"), float("nan")):
        qq, ln = q.clone(), lse.copy()
        qq[1, 3, 9] = value
        ln[1, 3] = np.nan  # what the decode says of that head
        got, _ = weigh(qq, cache, scales, table, lens, 64, ln, zero)
        assert np.all(np.isnan(got[1])) and np.array_equal(got[0], good[0])


def test_key_weights_of_queries_and_scales_of_any_size():
    # scores of a few tens whatever the factors: 2^e in the queries, 2^-e in the blocks' scales
    rng = np.random.default_rng(7)
    for e in (-60, -9, 40, 57):
        cache, scales, table = make_cache(rng, (400,), 64)
        scales = (scales * 2.0 ** -e).astype(np.float32).clip(2.0 ** -60, 2.0 ** 60)
        q = torch.from_numpy(rng.standard_normal((1, 16, 576)) * 2.0 ** e).bfloat16()
        lse = fp8.decode(f32(q), cache, scales, SCALE, table, (400,), 64)[1].astype(np.float32)
        w = np.zeros((1, 400), np.float32)
        got, flags = weigh(q, cache, scales, table, (400,), 64, lse, w)
        assert flags == 0
        check_weights(got, q, cache, scales, table, (400,), 64, lse, w, f"queries times 2^{e}")


def test_key_weights_in_a_graph_and_on_two_streams():
    rng = np.random.default_rng(8)
    lens = (5000, 300, 64, 1)
    q, cache, scales, table, lse = step(rng, 40, lens, 64)
    a = dict(page_table=t(table), seq_lens=i32(lens))
    args = (q.to(DEV), t(cache).view(F8), t(scales), SCALE, t(lse))
    plain = mla.mla_nvfp4_fp8_key_weights(*args, **a)
    outs, streams = [torch.zeros_like(plain) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for o, st in zip(outs, streams):
            with torch.cuda.stream(st):
                mla.mla_nvfp4_fp8_key_weights(*args, **a, out=o)
    torch.cuda.synchronize()
    total = torch.zeros_like(plain)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.mla_nvfp4_fp8_key_weights(*args, **a, weights=total, out=total)
    total.zero_()
    g.replay()
    a["seq_lens"][0] = 4000  # a replay reads the lengths anew
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, plain) for o in outs)
    assert torch.equal(total[1:], 2 * plain[1:]) and torch.equal(total[0, :4000], 2 * plain[0, :4000])
    assert torch.equal(total[0, 4000:], plain[0, 4000:])


# ------------------------------------------------------------------ eviction
def make_evict(rng, lens, keep, page, kind="spread"):
    left = [min(n, keep) for n in lens]
    both, pages = pages_for(rng, [n for n in lens] + left, page)
    table, new = both[:len(lens)].copy(), both[len(lens):].copy()
    cache = rng.integers(0, 256, (pages * page, 576), dtype=np.uint8)
    scales = np.exp2(rng.integers(-12, -3, pages * page // 64)).astype(np.float32)
    W = max(max(lens), 1)
    w = {"spread": np.exp(3 * rng.standard_normal((len(lens), W))), "ties": rng.integers(0, 4, (len(lens), W)),
         "equal": np.ones((len(lens), W)), "signs": rng.standard_normal((len(lens), W)) * 1e-40}[kind].astype(np.float32)
    return dict(table=table, new=new, cache=cache, scales=scales, w=w, lens=lens, page=page)


def evict(c, keep, recent, cache=None, scales=None, w=None, **kw):
    e = errw()
    cache = t(c["cache"]) if cache is None else cache
    scales = t(c["scales"]) if scales is None else scales
    kept, lens, nw = mla.mla_nvfp4_fp8_cache_evict(
        cache.view(F8), scales, t(c["w"]) if w is None else w, page_table=t(c["table"]), seq_lens=i32(c["lens"]),
        new_page_table=t(c["new"]), keep=keep, recent=recent, page_size=c["page"], error_word=e, **kw)
    torch.cuda.synchronize()
    return kept.cpu().numpy(), lens.cpu().numpy(), nw.cpu().numpy(), u8(cache), scales.cpu().numpy(), int(e.item())


def check_evict(c, got, keep, recent, what):
    cache, scales = c["cache"].copy(), c["scales"].copy()
    kept, lens, nw = fp8.evict(cache, scales, c["w"], c["table"], c["lens"], c["new"], keep, recent, c["page"])
    assert got[5] == 0, what
    assert np.array_equal(got[1], lens) and np.array_equal(got[0], kept), what
    assert np.array_equal(got[2], nw, equal_nan=True), what
    assert np.array_equal(got[4], scales), f"{what}: scales"
    same_codes(got[3], cache, what)


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "signs"])
@pytest.mark.parametrize("lens,keep,recent,page", [
    ((1000,), 256, 32, 64), ((1,), 1, 0, 64), ((1, 0, 2, 63, 64, 65, 129), 64, 7, 64), ((300, 5, 128), 130, 130, 128),
    ((300, 301), 1, 0, 64), ((300, 301), 1, 1, 192), ((5000, 1023, 1024, 1025), 1000, 1, 64), ((20000, 100), 3001, 500, 256),
    ((70,) * 50, 69, 3, 64), ((0, 0), 5, 2, 64), ((130, 64), 2000, 0, 64)])
def test_evict(lens, keep, recent, page, kind):
    rng = np.random.default_rng(sum(lens) + keep)
    c = make_evict(rng, lens, keep, page, kind)
    check_evict(c, evict(c, keep, recent), keep, recent, f"{kind} {keep} of {lens[:4]}")


@pytest.mark.parametrize("n", [8191, 8192, 8193, 16384, 16385, 32768, 40000, 65536, 70001, 140000])
def test_evict_long(n):
    rng = np.random.default_rng(n)
    for keep, recent, kind in ((n // 3, 100, "spread"), (n - 1, 0, "ties"), (7, 3, "spread"), (n // 2, n // 2, "equal")):
        c = make_evict(rng, (n,), keep, 64, kind)
        check_evict(c, evict(c, keep, recent), keep, recent, f"{kind} {keep} of {n}")


def test_evict_of_a_large_batch_with_one_long_sequence():
    # one CTA a sequence, which does not hold all its weights at once
    rng = np.random.default_rng(20)
    lens = (40000,) + (100, 0, 63) * 30
    for kind, keep in (("spread", 300), ("ties", 90)):
        c = make_evict(rng, lens, keep, 64, kind)
        check_evict(c, evict(c, keep, 10), keep, 10, f"91 sequences, {kind}")


def test_calls_in_a_row_read_what_the_work_ahead_wrote():
    # queries, cache, lengths and weights of every call are written by the kernels just before it
    rng = np.random.default_rng(21)
    lens, keep = (700, 64, 3000), 200
    sets = []
    for _ in range(3):
        q, cache, scales, table, lse = step(rng, 16, lens, 64)
        sets.append((q.to(DEV), t(cache), t(scales), t(lse), t(rng.random((3, 3000)).astype(np.float32))))
    blocks = sets[0][2].numel()
    new = torch.arange(blocks, blocks + 3 * 4, dtype=torch.int32, device=DEV).view(3, 4)
    tab, ln = t(table), i32(lens)
    grow = lambda s: (s[0], torch.cat([s[1], s[1].new_zeros(3 * 4 * 64, 576)]), torch.cat([s[2], s[2].new_ones(12)]), s[3], s[4])  # noqa: E731
    # (the sets' page tables differ; every set is read through the last one's)
    sets = [grow(s) for s in sets]
    clean = lambda c: torch.where((c & 0x7F) == 0x7F, 0x30, c)  # noqa: E731
    sets = [(s[0], clean(s[1]), s[2], s[3], s[4]) for s in sets]

    def both(q, cache, scales, lse, w):
        mla.mla_nvfp4_fp8_key_weights(q, cache.view(F8), scales, SCALE, lse, page_table=tab, seq_lens=ln, weights=w, out=w)
        return mla.mla_nvfp4_fp8_cache_evict(cache.view(F8), scales, w, page_table=tab, seq_lens=ln, new_page_table=new,
                                             keep=keep, recent=20)

    ref = []
    for s in sets:
        held = [x.clone() for x in s]
        torch.cuda.synchronize()
        out = both(*held)
        torch.cuda.synchronize()
        ref.append([x.clone() for x in (*out, held[1], held[2], held[4])])
    held, got = [x.clone() for x in sets[0]], []
    for i in range(60):
        for h, s in zip(held, sets[i % 3]):
            h.copy_(s)
        out = both(*held)
        got.append([x.clone() for x in (*out, held[1], held[2], held[4])])
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, ref[i % 3])), i


def test_evict_special_weights():
    rng = np.random.default_rng(9)
    c = make_evict(rng, (500, 400), 100, 64)
    c["w"][0, ::3], c["w"][0, 1::7], c["w"][0, 2::11], c["w"][1] = np.nan, np.inf, -np.inf, np.nan
    c["w"][0, 5::13] = -0.0
    for keep, recent in ((100, 0), (450, 10), (499, 0), (200, 200)):
        c["cache"] = rng.integers(0, 256, (64 * 40, 576), dtype=np.uint8)
        c["scales"] = np.ones(40, np.float32)
        c["table"] = np.arange(16).reshape(2, 8).astype(np.int32)
        c["new"] = (20 + np.arange(16)).reshape(2, 8).astype(np.int32)
        check_evict(c, evict(c, keep, recent), keep, recent, f"special {keep} {recent}")


def test_evict_strides_and_given_outputs():
    rng = np.random.default_rng(10)
    lens, keep = (300, 90, 700), 128
    c = make_evict(rng, lens, keep, 64)
    ref = evict(c, keep, 16)
    wide = torch.full((3, 900), float("nan"), device=DEV)
    wide[:, 100:800] = t(c["w"])
    out_w = torch.full((3, 400), 5.0, device=DEV)
    kept, nl = torch.empty((3, keep), dtype=torch.int32, device=DEV), torch.empty(3, dtype=torch.int32, device=DEV)
    got = evict(c, keep, 16, w=wide[:, 100:800], kept=kept, new_lens=nl, new_weights=out_w[:, 50:350])
    assert np.array_equal(got[0], ref[0]) and np.array_equal(kept.cpu().numpy(), ref[0]) and np.array_equal(got[3], ref[3])
    o = out_w.cpu().numpy()
    assert np.array_equal(o[:, 50:50 + keep], ref[2]) and not o[:, 50 + keep:350].any()  # a wider row's rest is zero
    assert np.all(o[:, :50] == 5) and np.all(o[:, 350:] == 5)


def test_evict_keeps_more_than_there_can_be():
    # new blocks end with the tokens and the new pages, kept's entries with -1
    rng = np.random.default_rng(31)
    c = make_evict(rng, (130, 0, 64), 1 << 16, 64)
    check_evict(c, evict(c, 1 << 16, 3), 1 << 16, 3, "of few")
    e = errw()
    pages = i32([0, 1, 2])[:, None]
    cache, sc = torch.zeros((6 * 64, 576), dtype=torch.uint8, device=DEV), torch.ones(6, device=DEV)
    kept, n, nw = mla.mla_nvfp4_fp8_cache_evict(
        cache.view(F8), sc, torch.empty((3, 0), device=DEV), page_table=pages, seq_lens=i32([0, 0, 0]), new_page_table=pages + 3,
        keep=5, error_word=e)
    assert kept.eq(-1).all() and n.eq(0).all() and nw.eq(0).all() and int(e.item()) == 0


def test_a_cache_past_32_bits_of_bytes():
    # the same keys in the first pages and beyond 2^32 bytes: the same results
    rng = np.random.default_rng(32)
    lens, keep = (300, 129), 100
    c = make_evict(rng, lens, keep, 64)
    c["cache"] &= 0xF7  # (no NaN)
    pages = len(c["cache"]) // 64
    first = (1 << 32) // (576 * 64) + 1
    cache = torch.empty(((first + pages) * 64, 576), dtype=torch.uint8, device=DEV)
    scales = torch.zeros(first + pages, device=DEV)
    cache[first * 64:], scales[first:] = t(c["cache"]), t(c["scales"])
    far = {**c, "table": c["table"] + first, "new": c["new"] + first}
    q = torch.from_numpy(rng.standard_normal((2, 16, 576))).bfloat16().to(DEV)

    def calls(cache, scales, c):
        e = errw()
        a = dict(page_table=t(c["table"]), seq_lens=i32(lens), error_word=e)
        out, lse = mla.mla_nvfp4_fp8_decode_shared(q, cache.view(F8), scales, SCALE, shared_len=0, return_lse=True, **a)
        w = mla.mla_nvfp4_fp8_key_weights(q, cache.view(F8), scales, SCALE, lse, **a)
        got = evict(c, keep, 10, cache=cache, scales=scales)
        assert int(e.item()) == 0 and got[5] == 0
        return f32(out), f32(lse), w.cpu().numpy(), got

    near = calls(t(c["cache"]), t(c["scales"]), c)
    there = calls(cache, scales, far)
    for x, y in zip(near[:3] + near[3][:3], there[:3] + there[3][:3]):
        assert np.all(np.isfinite(x)) and np.array_equal(x, y)
    assert np.array_equal(near[3][3], there[3][3][first * 64:]) and np.array_equal(near[3][4], there[3][4][first:])


def test_evict_bad_entries():
    rng = np.random.default_rng(11)
    lens, keep = (300, 200), 150
    for change in ("page", "page_neg", "scale", "length", "row", "new page", "new page neg", "new room"):
        c = make_evict(rng, lens, keep, 64)
        ref_c = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in c.items()}
        if change in ("page", "page_neg"):
            c["table"][0, 1] = ref_c["table"][0, 1] = len(c["cache"]) // 64 if change == "page" else -1
        elif change == "scale":
            c["scales"][c["table"][0, 1]] = ref_c["scales"][c["table"][0, 1]] = np.nan
        elif change == "length":
            c["table"] = c["table"][:, :4].copy()
            ref_c["lens"] = (256, 200)
        elif change == "row":
            c["w"] = c["w"][:, :250].copy()
            ref_c["lens"] = (250, 200)
        elif change in ("new page", "new page neg"):
            c["new"][0, 1] = ref_c["new"][0, 1] = len(c["cache"]) // 64 if change == "new page" else -1
        else:  # 128 of 150 fit
            c["new"] = c["new"][:, :2].copy()
        got = evict(c, keep, 20)
        if change == "new room":
            k, l, w = (fp8.evict(ref_c["cache"], ref_c["scales"], c["w"], c["table"], lens, c["new"], 128, 20, 64))
            assert got[1].tolist() == [128, 128] and np.array_equal(got[0][:, :128], k) and np.all(got[0][:, 128:] == -1)
        else:
            k, l, w = fp8.evict(ref_c["cache"], ref_c["scales"], ref_c["w"], ref_c["table"], ref_c["lens"], ref_c["new"],
                                keep, 20, 64)
            assert np.array_equal(got[0], k) and np.array_equal(got[1], l), change
        assert got[5] == (4 if change == "scale" else 1), change
        same_codes(got[3], ref_c["cache"], change)
        assert np.array_equal(got[4], ref_c["scales"], equal_nan=True), change


def test_evict_moves_nan_codes_and_zero_keys():
    rng = np.random.default_rng(12)
    c = make_evict(rng, (200,), 100, 64)
    c["cache"][:] = np.where(rng.random(c["cache"].shape) < 0.2, 0x7F, 0)
    check_evict(c, evict(c, 100, 0), 100, 0, "NaN codes and zeros")


def test_evict_in_a_graph_repeats_and_reads_lengths_anew():
    rng = np.random.default_rng(13)
    lens, keep, recent = (9000, 300), 700, 64
    c = make_evict(rng, lens, keep, 64)
    cache, scales, w = t(c["cache"]), t(c["scales"]), t(c["w"])
    tab, new, ln = t(c["table"]), t(c["new"]), i32(lens)
    mla.mla_nvfp4_fp8_cache_evict(cache.view(F8), scales, w, page_table=tab, seq_lens=ln, new_page_table=new, keep=keep,
                                  recent=recent)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept, nl, nw = mla.mla_nvfp4_fp8_cache_evict(cache.view(F8), scales, w, page_table=tab, seq_lens=ln,
                                                     new_page_table=new, keep=keep, recent=recent)
    for now in ((9000, 300), (5000, 1), (0, 299)):
        cache.copy_(t(c["cache"]))
        scales.copy_(t(c["scales"]))
        ln.copy_(i32(now))
        g.replay()
        torch.cuda.synchronize()
        got = kept.cpu().numpy(), nl.cpu().numpy(), nw.cpu().numpy(), u8(cache), scales.cpu().numpy(), 0
        check_evict({**c, "lens": now}, got, keep, recent, f"replay {now}")


# ------------------------------------------------------------- a run of them
def test_append_at_positions():
    rng = np.random.default_rng(14)
    new, ctx, pos, heads = (3, 70, 1, 5), (60, 0, 128, 10), (1000, 7, 128, 400), 4
    table, pages = pages_for(rng, [a + b for a, b in zip(new, ctx)], 64)
    T, cs = sum(new), angles(1100)
    kv, pe = (torch.from_numpy(rng.standard_normal((T, d))).bfloat16() for d in (512, 64))
    q = torch.from_numpy(rng.standard_normal((T, heads, 64))).bfloat16()
    cache, scales = rng.integers(0, 256, (pages * 64, 576), dtype=np.uint8), np.full(pages, 2.0 ** -7, np.float32)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    for interleaved in (True, False):
        e, dc, ds = errw(), t(cache), t(scales)
        got = mla.mla_nvfp4_fp8_cache_append(kv.to(DEV), pe.to(DEV), t(cs), t(cu), i32(ctx), t(table), dc.view(F8), ds,
                                             interleaved=interleaved, q_pe=q.to(DEV), positions=i32(pos), error_word=e)
        torch.cuda.synchronize()
        rc, rs = cache.copy(), scales.copy()
        fp8.append(rc, rs, f32(kv), f32(pe), cs, cu, ctx, table, 64, interleaved, positions=pos)
        assert int(e.item()) == 0 and np.array_equal(ds.cpu().numpy(), rs)
        same_codes(u8(dc), rc, "append at")
        at = np.concatenate([np.arange(p, p + n) for p, n in zip(pos, new)])
        assert np.array_equal(f32(got), f32(torch.from_numpy(fp8.rotate(f32(q), cs[at][:, None], interleaved)).bfloat16()))


def test_append_at_bad_positions():
    rng = np.random.default_rng(15)
    table, pages = pages_for(rng, (70, 70), 64)
    kv, pe = (torch.from_numpy(rng.standard_normal((6, d))).bfloat16() for d in (512, 64))
    cache, scales = np.zeros((pages * 64, 576), np.uint8), np.full(pages, 2.0 ** -7, np.float32)
    cs, cu = angles(100), np.array([0, 3, 6], np.int32)
    for pos, rows in (((-1, 50), (0, 3)), ((98, 50), (2, 3)), ((100, 50), (0, 3)), ((2 ** 31 - 1, 50), (0, 3))):
        e, dc, ds = errw(), t(cache), t(scales)
        mla.mla_nvfp4_fp8_cache_append(kv.to(DEV), pe.to(DEV), t(cs), t(cu), i32((10, 20)), t(table), dc.view(F8), ds,
                                       positions=i32(pos), error_word=e)
        torch.cuda.synchronize()
        assert int(e.item()) == 1
        got = u8(dc)
        for b, n in enumerate(rows):
            s = int(table[b][0]) * 64 + (10, 20)[b]
            assert np.all(got[s:s + n].any(1)) and not got[s + n:s + 3].any()


def test_decode_weigh_evict_append_decode():
    """A generation that keeps its cache within a budget: each step appends a token, decodes, adds to the weights, and evicts
    where the budget is passed; every result against the oracle on the oracle's own cache."""
    rng = np.random.default_rng(16)
    B, H, page, budget, keep, recent = 3, 16, 64, 160, 96, 32
    lens, pos = np.array([150, 159, 100]), np.array([150, 159, 100])
    pages = 2 * B * 3
    free = list(rng.permutation(pages))
    take = lambda n: [int(free.pop()) for _ in range(n)]  # noqa: E731
    table = np.zeros((B, 3), np.int32)
    for b in range(B):
        table[b] = take(3)
    cache, scales, _ = make_cache(rng, (pages * 64,), 64)
    cache = cache[:pages * 64]
    cache[(cache & 0x7F) == 0x7F] = 0x30
    scales = scales[:pages]
    w, cs = np.zeros((B, 192), np.float32), angles(200)
    rc, rs = cache.copy(), scales.copy()
    dc, ds, dw, dtab = t(cache), t(scales), t(w), t(table)
    evictions = 0
    for _ in range(12):
        kv, pe = (torch.from_numpy(rng.standard_normal((B, d))).bfloat16() for d in (512, 64))
        q = torch.from_numpy(rng.standard_normal((B, H, 576))).bfloat16()
        cu, e = np.arange(B + 1, dtype=np.int32), errw()
        dq = q.to(DEV)
        mla.mla_nvfp4_fp8_cache_append(kv.to(DEV), pe.to(DEV), t(cs), t(cu), i32(lens), dtab, dc.view(F8), ds,
                                       q_pe=dq[:, :, 512:], q_out=dq[:, :, 512:], positions=i32(pos), error_word=e)
        fp8.append(rc, rs, f32(kv), f32(pe), cs, cu, lens, table, page, True, positions=pos)
        lens, pos = lens + 1, pos + 1
        out, lse = mla.mla_nvfp4_fp8_decode(dq, dc.view(F8), ds, SCALE, page_table=dtab, seq_lens=i32(lens), return_lse=True,
                                            error_word=e)
        mla.mla_nvfp4_fp8_key_weights(dq, dc.view(F8), ds, SCALE, lse, page_table=dtab, seq_lens=i32(lens), weights=dw,
                                      out=dw, error_word=e)
        torch.cuda.synchronize()
        assert int(e.item()) == 0 and np.array_equal(ds.cpu().numpy(), rs)
        same_codes(u8(dc), rc, "cache")
        check_decode((f32(out), f32(lse)), dq.cpu(), rc, rs, table, lens, page, what="step")
        check_weights(dw.cpu().numpy(), dq.cpu(), rc, rs, table, lens, page, f32(lse), w, "step")
        w = dw.cpu().numpy()
        if lens.max() > budget:
            evictions += 1
            new = np.stack([take(3) for _ in range(B)]).astype(np.int32)
            dnew = t(new)
            dw2 = torch.full_like(dw, 3.0)
            kept, nl, _ = mla.mla_nvfp4_fp8_cache_evict(dc.view(F8), ds, dw, page_table=dtab, seq_lens=i32(lens),
                                                        new_page_table=dnew, keep=keep, recent=recent, new_weights=dw2,
                                                        error_word=e)
            torch.cuda.synchronize()
            rk, rl, rw = fp8.evict(rc, rs, w, table, lens, new, keep, recent, page)
            assert int(e.item()) == 0 and np.array_equal(kept.cpu().numpy(), rk) and np.array_equal(nl.cpu().numpy(), rl)
            free += [int(x) for x in table.reshape(-1)]
            lens, table, dtab, dw = rl.astype(int), new, dnew, dw2
            w = np.zeros_like(w)
            w[:, :keep] = rw
            assert np.array_equal(dw.cpu().numpy(), w)
    assert evictions == 1


_FIRST_CALLS = """
import torch
import mla_attention_nvfp4_gb300 as mla
D = "cuda"
cache = torch.zeros((640, 576), dtype=torch.uint8, device=D).view(torch.float8_e4m3fn)
scales, gs = torch.ones(10, device=D), torch.ones(1, device=D)
table = torch.arange(4, dtype=torch.int32, device=D).view(2, 2)
a = dict(page_table=table, seq_lens=torch.tensor([100, 90], dtype=torch.int32, device=D))
codes, sf = torch.full((512, 512), 0x21, dtype=torch.uint8, device=D), torch.full((512 * 64,), 0x38, dtype=torch.uint8, device=D)
calls = []
for h in (16, 128):
    q, lse = torch.ones((2, h, 576), device=D).bfloat16(), torch.zeros((2, h), device=D)
    x = torch.ones((h // 8, 1024), device=D).bfloat16()
    calls += [lambda q=q: mla.mla_nvfp4_fp8_decode_shared(q, cache, scales, 0.1, shared_len=64, **a),
              lambda q=q, lse=lse: mla.mla_nvfp4_fp8_key_weights(q, cache, scales, 0.1, lse, **a),
              lambda x=x: mla.mla_nvfp4_gemv(x, codes, sf, gs)]
w = torch.rand((2, 128), device=D)
calls.append(lambda: mla.mla_nvfp4_fp8_cache_evict(cache, scales, w, new_page_table=table[:, :1] + 4, keep=40, **a)[0])
torch.cuda.synchronize()
for f in calls:
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = f()
    g.replay()
    assert torch.equal(r, f())
print("same")
"""


def test_a_process_may_capture_its_first_calls():
    r = subprocess.run([sys.executable, "-c", _FIRST_CALLS], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


@pytest.mark.parametrize("heads", [64, 72, 96, 128, 200])
def test_key_weights_repeat_themselves(heads):
    """Sequences of many tiles and of one, more of both than there are SMs: every call gives the same bits."""
    rng = np.random.default_rng(heads)
    lens = (2500, 1, 129, 0, 128, 1023) + (130, 64) * 80
    q, cache, scales, table, lse = step(rng, heads, lens, 64)
    w = rng.random((len(lens), 2500)).astype(np.float32)
    got, flags = weigh(q, cache, scales, table, lens, 64, lse, w)
    assert flags == 0
    check_weights(got, q, cache, scales, table, lens, 64, lse, w, f"{heads} heads, many sequences")
    args = (q.to(DEV), t(cache).view(F8), t(scales), SCALE, t(lse))
    kw = dict(page_table=t(table), seq_lens=i32(lens), weights=t(w))
    again = [mla.mla_nvfp4_fp8_key_weights(*args, **kw, out=t(w)) for _ in range(20)]
    torch.cuda.synchronize()
    assert all(np.array_equal(x.cpu().numpy(), got) for x in again)


def test_evict_wants_a_page_table_row_for_each_sequence():
    # (the decodes and the key weights take one row for all)
    c = make_evict(np.random.default_rng(40), (64, 64), 32, 64)
    for name in ("page_table", "new_page_table"):
        e, kw = errw(), dict(page_table=t(c["table"]), new_page_table=t(c["new"]))
        kw[name] = kw[name][:1].expand(2, -1)
        before = t(c["cache"])
        with pytest.raises(ValueError, match="a row for each sequence"):
            mla.mla_nvfp4_fp8_cache_evict(before.view(F8), t(c["scales"]), t(c["w"]), seq_lens=i32((64, 64)), keep=32,
                                          error_word=e, **kw)
        torch.cuda.synchronize()
        assert int(e.item()) == 0 and np.array_equal(before.cpu().numpy(), c["cache"])


def test_weights_beside_their_results_in_one_matrix():
    rng = np.random.default_rng(41)
    lens = (300, 0, 129)
    q, cache, scales, table, lse = step(rng, 16, lens, 64)
    w = rng.random((3, 320)).astype(np.float32)
    ref, _ = weigh(q, cache, scales, table, lens, 64, lse, w)
    both = torch.full((3, 700), 7.0, device=DEV)
    both[:, :320] = t(w)
    mla.mla_nvfp4_fp8_key_weights(q.to(DEV), t(cache).view(F8), t(scales), SCALE, t(lse), page_table=t(table),
                                  seq_lens=i32(lens), weights=both[:, :320], out=both[:, 320:640])
    got = both.cpu().numpy()
    assert np.array_equal(got[:, :320], w) and np.all(got[:, 640:] == 7)
    for b, n in enumerate(lens):
        assert np.array_equal(got[b, 320:320 + n], ref[b, :n]) and np.all(got[b, 320 + n:] == 7)
    c = make_evict(rng, lens, 100, 64)
    ref = evict(c, 100, 10)
    n = c["w"].shape[1]
    both = torch.full((3, n + 150), 7.0, device=DEV)
    both[:, :n] = t(c["w"])
    got = evict(c, 100, 10, w=both[:, :n], new_weights=both[:, n:n + 120])
    assert all(np.array_equal(a, b) for i, (a, b) in enumerate(zip(got, ref)) if i != 2)
    assert np.array_equal(got[2][:, :100], ref[2]) and not got[2][:, 100:].any()
    assert np.array_equal(both[:, :n].cpu().numpy(), c["w"]) and bool((both[:, n + 120:] == 7).all())
