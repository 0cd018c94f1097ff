"""The 8-bit path on the GPU against the float64 oracle: append to the e4m3
latent cache, attention over it, the quantiser and the GEMM.

Tolerances, for each output element:
  append, quantize  codes and scales equal: the kernels evaluate the float32
                    definition the oracle states.
  gemm              2^-8 |c| (rounding to bf16) + 2^-24 (K + 2 blocks) *
                    sum |a w| (fp32 sums of K exact products and one scaled
                    sum a block).
  decode            2^-8 |o| (bf16) + 2^-8 * sum p |v| / sum p (probabilities
                    carried as two 8-bit terms: for p in [2^e, 2^(e+1)) the
                    first leaves at most 2^(e-4), of which the second, e4m3 or
                    e5m2, leaves at most 2^(e-8)) + the scores' fp32 sums:
                    a score off by d moves p by a factor e^d, so
                    2 (e^d - 1) * sum p |v| / sum p with
                    d = 2^-24 (576 + 8) * max sum |q k| * scale
                    + f * max_j (p_j s_j) * sum_j |k8_j|, f = 2^-17: where
                    the two terms' step is absolute it is 2^-13, a weight
                    carries p_j s_j K with the largest at least 2^4, and a
                    weight's error (half a step, half a step of offset) times
                    |k8_j| / K enters the output.
  lse               d, plus 2^-22 |lse| (log2 and its rescaling in fp32), plus
                    2^-20 (exp2 of a difference), plus 2^-24 (n + n / 32 + 4)
                    for n keys: a sum of n positive terms in fp32 is at most
                    n - 1 half steps off, relative to itself, and each of its
                    at most n / 64 + 1 rescalings two more; ln(1 + x) <= x.
"""
import math

import numpy as np
import pytest
import torch

import mla_attention_nvfp4_gb300 as mla
from oracle import fp8
from tests.helpers import bf16_half_ulp, f32

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
DEV = "cuda:0"
SCALE = 1.0 / math.sqrt(192.0)
F8 = torch.float8_e4m3fn


def u8(t):
    return t.cpu().view(torch.uint8).numpy()


def errw():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def angles(n, base=10000.0):
    f = base ** (-np.arange(0, 64, 2) / 64)
    a = np.arange(n)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def pages_for(rng, lens, page, spare=2):
    """A permuted page table one page wider than needed (unused entries out of range), and the pages there are."""
    need = [-(-int(n) // page) for n in lens]
    ids = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max(max(need), 1) + 1), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, len(ids)


# ------------------------------------------------------------------- append
def make_append(rng, new, ctx, page, heads, pad=0, spread=1.0):
    lens = [a + b for a, b in zip(new, ctx)]
    table, pages = pages_for(rng, lens, page)
    T = sum(new) + pad
    slots = pages * page
    c = dict(table=table, page=page, cu=np.concatenate([[0], np.cumsum(new)]).astype(np.int32),
             ctx=np.asarray(ctx, np.int32), cs=angles(max(lens) + 1),
             kv=(torch.from_numpy(rng.standard_normal((T, 512)) * np.exp2(rng.uniform(-spread, spread, (T, 1))))
                 .bfloat16()),
             pe=torch.from_numpy(rng.standard_normal((T, 64))).bfloat16(),
             q=torch.from_numpy(rng.standard_normal((T, heads, 64))).bfloat16() if heads else None,
             # what a reused cache holds: any bytes, NaN codes among them, and scales of a running cache
             cache=rng.integers(0, 256, (slots, 576), dtype=np.uint8),
             scales=np.exp2(rng.integers(-9, -5, slots // 64)).astype(np.float32))
    return c


def run_append(c, interleaved=True, max_new=None, in_place=False, table=None, rows=slice(None)):
    d = {k: torch.from_numpy(c[k]).to(DEV) for k in ("cu", "ctx", "cs", "cache", "scales")}
    table = torch.from_numpy(c["table"]).to(DEV) if table is None else table
    q = c["q"].to(DEV) if c["q"] is not None else None
    e = errw()
    got = mla.mla_nvfp4_fp8_cache_append(c["kv"].to(DEV), c["pe"].to(DEV), d["cs"], d["cu"], d["ctx"], table,
                                         d["cache"].view(F8), d["scales"], page_size=c["page"],
                                         interleaved=interleaved, q_pe=q, q_out=q if in_place else None,
                                         max_new_tokens=max_new, error_word=e)
    torch.cuda.synchronize()
    return u8(d["cache"]), d["scales"].cpu().numpy(), None if got is None else f32(got), int(e.item())


def same_codes(got, ref, what):
    # a code that is NaN on both sides may carry either sign
    nan = ((got & 0x7F) == 0x7F) & ((ref & 0x7F) == 0x7F)
    assert np.array_equal(np.where(nan, 0x7F, got), np.where(nan, 0x7F, ref)), \
        f"{what}: {int(((got != ref) & ~nan).sum())} codes differ"


def check_append(c, got, interleaved, n_rows):
    cache, scales = c["cache"].copy(), c["scales"].copy()
    fp8.append(cache, scales, f32(c["kv"]), f32(c["pe"]), c["cs"], c["cu"], c["ctx"], c["table"], c["page"], interleaved)
    assert np.array_equal(got[1], scales), f"scales differ at {np.nonzero(got[1] != scales)[0][:8]}"
    same_codes(got[0], cache, "append")
    if c["q"] is not None:
        pos = np.concatenate([np.arange(a, a + n) for a, n in zip(c["ctx"], np.diff(c["cu"]))]).astype(int)
        ref = fp8.rotate(f32(c["q"][:n_rows]), c["cs"][pos][:, None], interleaved)
        assert np.array_equal(got[2][:n_rows], f32(torch.from_numpy(ref).bfloat16()))


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("new,ctx,page,heads", [
    ((1,), (0,), 64, 1), ((1,), (63,), 64, 16), ((1,), (64,), 64, 128), ((1, 1, 1), (5, 127, 1000), 64, 5),
    ((64,), (0,), 64, 2), ((65, 63), (0, 1), 128, 3), ((200, 1, 129), (30, 64, 191), 64, 7),
    ((700, 0, 3), (100, 77, 0), 192, 0), ((2, 2), (63, 62), 64, 33)])
def test_append(interleaved, new, ctx, page, heads):
    rng = np.random.default_rng(sum(new) + 7 * page)
    c = make_append(rng, new, ctx, page, heads)
    got = run_append(c, interleaved)
    assert got[3] == 0
    check_append(c, got, interleaved, sum(new))


def test_append_step_by_step_grows_and_equals_oracle():
    # one token a call over three blocks, magnitudes rising and falling by up
    # to 2^12: scales grow inside a block and start anew in the next
    rng = np.random.default_rng(5)
    c = make_append(rng, (1,), (190,), 64, 0)
    cache, scales = torch.from_numpy(c["cache"]).to(DEV), torch.from_numpy(c["scales"]).to(DEV)
    rc, rs = c["cache"].copy(), c["scales"].copy()
    table, cs = torch.from_numpy(c["table"]).to(DEV), torch.from_numpy(c["cs"]).to(DEV)
    cu = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    for p in range(190):
        kv = torch.from_numpy(rng.standard_normal((1, 512)) * 2.0 ** rng.integers(-6, 7)).bfloat16()
        pe = torch.from_numpy(rng.standard_normal((1, 64))).bfloat16()
        mla.mla_nvfp4_fp8_cache_append(kv.to(DEV), pe.to(DEV), cs, cu, torch.tensor([p], dtype=torch.int32, device=DEV),
                                       table, cache.view(F8), scales)
        fp8.append(rc, rs, f32(kv), f32(pe), c["cs"], [0, 1], [p], c["table"], 64, True)
    torch.cuda.synchronize()
    assert np.array_equal(scales.cpu().numpy(), rs)
    same_codes(u8(cache), rc, "steps")


def test_append_extreme_values():
    rng = np.random.default_rng(6)
    c = make_append(rng, (70, 3, 64), (0, 10, 64), 64, 1)
    kv = c["kv"].float()
    kv[0, 3], kv[1, 4], kv[2, 5] = math.inf, -math.inf, math.nan
    kv[71] = 1e38
    kv[73:137] = 0
    kv[80, 9] = 1e-30
    c["kv"] = kv.bfloat16()
    c["pe"][73:137] = 0
    c["scales"][int(c["table"][1][0])] = 2.0 ** -60
    got = run_append(c)
    assert got[3] == 0
    check_append(c, got, True, 137)


def test_append_strides_padding_and_in_place():
    rng = np.random.default_rng(7)
    new, ctx, pad = (5, 70, 1), (60, 3, 128), 9
    c = make_append(rng, new, ctx, 64, 4, pad=pad)
    ref = run_append(c)
    check_append(c, ref, True, 76)
    # rows of one wide projection, queries inside a wider tensor, a page table inside a wider one; the rows behind
    # the last sequence, and everything around the rotated part, stay as they are
    T = 76 + pad
    wide = torch.zeros(T, 1024, dtype=torch.bfloat16, device=DEV)
    wide[:, :512], wide[:, 512:576] = c["kv"].to(DEV), c["pe"].to(DEV)
    q = torch.randn(T, 4, 576, device=DEV).bfloat16()
    q[:, :, 512:] = c["q"].to(DEV)
    before = q.clone()
    tab = torch.full((3, 11), -5, dtype=torch.int32, device=DEV)
    tab[:, 2:2 + c["table"].shape[1]] = torch.from_numpy(c["table"]).to(DEV)
    d = {k: torch.from_numpy(c[k]).to(DEV) for k in ("cu", "ctx", "cs", "cache", "scales")}
    e = errw()
    r = mla.mla_nvfp4_fp8_cache_append(wide[:, :512], wide[:, 512:576], d["cs"], d["cu"], d["ctx"],
                                       tab[:, 2:2 + c["table"].shape[1]], d["cache"].view(F8), d["scales"],
                                       q_pe=q[:, :, 512:], q_out=q[:, :, 512:], max_new_tokens=70, error_word=e)
    torch.cuda.synchronize()
    assert r.data_ptr() == q[:, :, 512:].data_ptr() and int(e.item()) == 0
    assert np.array_equal(u8(d["cache"]), ref[0]) and np.array_equal(d["scales"].cpu().numpy(), ref[1])
    assert np.array_equal(f32(q[:76, :, 512:]), ref[2][:76])
    assert torch.equal(q[76:], before[76:]) and torch.equal(q[:, :, :512], before[:, :, :512])


def test_append_bad_entries_are_flagged_and_skipped():
    rng = np.random.default_rng(8)
    base = make_append(rng, (3, 4, 5), (64, 10, 60), 64, 2)

    def untouched(c, got, seqs):
        ok = np.ones(len(c["cache"]), bool)
        for b in seqs:
            # every block that takes a token: its earlier tokens are rounded again where its scale grows
            blocks = np.arange(c["ctx"][b] // 64, (c["ctx"][b] + c["cu"][b + 1] - c["cu"][b] - 1) // 64 + 1)
            for s in c["table"][b][blocks].astype(np.int64) * 64:
                ok[s:s + 64] = False
        assert np.array_equal(got[0][ok], c["cache"][ok])

    for change in ("page", "page_neg", "context", "cu", "max_new", "angles", "scale"):
        c = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in base.items()}
        kw = {}
        if change == "page":
            c["table"][1, 0] = len(c["cache"]) // 64
        elif change == "page_neg":
            c["table"][1, 0] = -1
        elif change == "context":
            c["ctx"][1] = -3
        elif change == "cu":
            c["cu"][3] = 13  # one row more than there are
        elif change == "max_new":
            kw["max_new"] = 3
        elif change == "angles":
            c["cs"] = c["cs"][:62]  # sequences 0 and 2 reach past it
        else:
            c["scales"][c["table"][1, 0]] = math.nan
        got = run_append(c, **kw)
        assert got[3] == (4 if change == "scale" else 1), change
        if change in ("page", "page_neg", "context"):
            untouched(base, got, (0, 2))
        if change == "cu":
            untouched(base, got, (0, 1))
        if change == "angles":
            untouched(base, got, (1, 2))
        # the other sequences' tokens are written as ever
        ref = run_append(base)
        if change in ("page", "context"):
            s = int(base["table"][0][1]) * 64
            assert np.array_equal(got[0][s:s + 3], ref[0][s:s + 3])


# ------------------------------------------------------------------- decode
def make_cache(rng, lens, page, spread=0):
    table, pages = pages_for(rng, lens, page)
    blocks = pages * page // 64
    # every byte any: NaN codes in rows that hold no key of a sequence
    cache = rng.integers(0, 256, (blocks * 64, 576), dtype=np.uint8)
    scales = np.exp2(rng.integers(-7 - spread, -6 + spread + 1, blocks)).astype(np.float32)
    for b, n in enumerate(lens):
        t = np.arange(n)
        slot = table[b][t // page].astype(np.int64) * page + t % page
        x = rng.standard_normal((n, 576))
        x[:, :512] *= np.where(rng.random((n, 512)) < 0.01, 20, 1)
        cache[slot] = fp8.encode(x * 128)
    return cache, scales, table


def run_decode(q, cache, scales, table, lens, page, scale=SCALE, **kw):
    e = errw()
    out, lse = mla.mla_nvfp4_fp8_decode(q.to(DEV), torch.from_numpy(cache).to(DEV).view(F8),
                                        torch.from_numpy(scales).to(DEV), scale,
                                        page_table=torch.from_numpy(table).to(DEV),
                                        seq_lens=torch.tensor(list(lens), dtype=torch.int32, device=DEV),
                                        page_size=page, return_lse=True, error_word=e, **kw)
    torch.cuda.synchronize()
    return f32(out), f32(lse), int(e.item())


def check_decode(got, q, cache, scales, table, lens, page, scale=SCALE, what="decode"):
    out, lse, oabs, flat = fp8.decode(f32(q), cache, scales, scale, table, lens, page)
    qa = np.abs(f32(q))
    d = np.zeros(qa.shape[:2])
    for b, n in enumerate(lens):
        t = np.arange(n)
        if n:
            page_id = table[b][t // page].astype(np.int64)
            slot = page_id * page + t % page
            slot = slot[(page_id >= 0) & (slot < len(cache))]
            s = np.asarray(scales, np.float64)[slot // 64]
            k = np.abs(np.nan_to_num(fp8.decode_codes(cache[slot]))) * np.where((s >= 2.0**-60) & (s <= 2.0**60), s, 0)[:, None]
            d[b] = (qa[b] @ k.T).max(1, initial=0) * scale * 2.0 ** -24 * 584
    tol = np.maximum(bf16_half_ulp(out), bf16_half_ulp(got[0])) + (2.0 ** -8 + 2 * np.expm1(d))[..., None] * oabs
    tol = tol + 2.0 ** -17 * flat
    err = np.abs(got[0] - out)
    assert np.all(np.isfinite(got[0])), f"{what}: not finite"
    worst = float(np.max(err / np.maximum(tol, 1e-30), initial=0))
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(got[1]), empty), f"{what}: -inf pattern"
    le = np.where(empty, 0, np.abs(np.where(empty, 0, got[1]) - np.where(empty, 0, lse)))
    terms = np.maximum(np.asarray(lens, np.float64), 0)[:, None]
    ltol = d + 2.0 ** -22 * np.abs(np.where(empty, 0, lse)) + 2.0 ** -20 + 2.0 ** -24 * (terms * (1 + 1 / 32) + 4)
    print(f"[fp8 decode] {what}: error {worst:.3f} of the tolerance, lse {float(np.max(le / ltol, initial=0)):.3f}; "
          f"relative 2-norm {np.linalg.norm(err) / max(np.linalg.norm(out), 1e-30):.2e}")
    assert worst <= 1, f"{what}: {worst:.2f} times the tolerance"
    assert np.all(le <= ltol), f"{what}: lse off by {le.max():.2e}"
    assert np.all(got[0][empty] == 0)


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("heads", [1, 16, 31, 32, 33, 64, 128, 130])
def test_decode_heads(heads, split):
    rng = np.random.default_rng(heads)
    lens = (1, 0, 63, 64, 65, 127, 128, 129, 700)
    cache, scales, table = make_cache(rng, lens, 64)
    q = torch.from_numpy(rng.standard_normal((len(lens), heads, 576))).bfloat16()
    got = run_decode(q, cache, scales, table, lens, 64, split=split)
    assert got[2] == 0
    check_decode(got, q, cache, scales, table, lens, 64, what=f"{heads} heads split={split}")


@pytest.mark.parametrize("page", [64, 128, 192, 1024])
@pytest.mark.parametrize("lens", [(5000,), (1, 3000, 77), (0, 0), (64,) * 40, (2, 0, 4097) * 3, (1,) * 160])
def test_decode_lengths(page, lens):
    rng = np.random.default_rng(page + len(lens))
    cache, scales, table = make_cache(rng, lens, page)
    q = torch.from_numpy(rng.standard_normal((len(lens), 24, 576))).bfloat16()
    got = run_decode(q, cache, scales, table, lens, page)
    assert got[2] == 0
    check_decode(got, q, cache, scales, table, lens, page, what=f"page {page}, {len(lens)} sequences")


def test_decode_many_short_sequences():
    rng = np.random.default_rng(11)
    lens = tuple(int(x) for x in rng.integers(0, 140, 400))
    cache, scales, table = make_cache(rng, lens, 64)
    q = torch.from_numpy(rng.standard_normal((len(lens), 3, 576))).bfloat16()
    got = run_decode(q, cache, scales, table, lens, 64)
    check_decode(got, q, cache, scales, table, lens, 64, what="400 short")


@pytest.mark.parametrize("growth", [0.02, 0.3, 2.0, -0.3])
def test_decode_scores_that_grow_or_fall(growth):
    # the keys' magnitude changes from block to block, so the running maximum
    # of every head moves many times
    rng = np.random.default_rng(12)
    lens = (1500, 900)
    cache, scales, table = make_cache(rng, lens, 64)
    for b, n in enumerate(lens):
        for blk in range(-(-n // 64)):
            scales[table[b][blk]] = 2.0 ** -7 * max(0.02, 1 + growth * blk)
    q = torch.from_numpy(rng.standard_normal((2, 40, 576))).bfloat16()
    got = run_decode(q, cache, scales, table, lens, 64)
    check_decode(got, q, cache, scales, table, lens, 64, what=f"growth {growth}")


@pytest.mark.parametrize("spread", [8, 20])
def test_decode_block_scales_far_apart(spread):
    rng = np.random.default_rng(13 + spread)
    lens = (1000, 130)
    cache, scales, table = make_cache(rng, lens, 64, spread=spread)
    q = torch.from_numpy(rng.standard_normal((2, 32, 576))).bfloat16()
    sc = SCALE * 2.0 ** -spread
    got = run_decode(q, cache, scales, table, lens, 64, scale=sc)
    check_decode(got, q, cache, scales, table, lens, 64, scale=sc, what=f"scales 2^+-{spread}")


@pytest.mark.parametrize("heads", [16, 40])
@pytest.mark.parametrize("n,gap", [(3000, 6.0), (3000, 9.0), (20000, 12.0)])
def test_decode_one_peak_over_a_flat_tail(n, gap, heads):
    # one key far above many of equal score: the tail's weights are far below
    # the peak's and all the same, so a one-sided rounding of theirs would
    # show in the output
    rng = np.random.default_rng(14)
    cache, scales, table = make_cache(rng, (n,), 64)
    scales[:] = 2.0 ** -7
    slot = table[0][np.arange(n) // 64].astype(np.int64) * 64 + np.arange(n) % 64
    cache[slot, 512:] = fp8.encode(np.zeros((n, 64)))
    cache[slot, :512] = fp8.encode(rng.standard_normal((1, 512)) * 60 + rng.standard_normal((n, 512)) * 20)
    cache[slot[17], 512] = 0x7E  # 448
    q = np.zeros((1, heads, 576))
    q[:, :, 512] = gap / (448 * 2.0 ** -7 * SCALE)
    q = torch.from_numpy(q).bfloat16()
    got = run_decode(q, cache, scales, table, (n,), 64)
    check_decode(got, q, cache, scales, table, (n,), 64, what=f"peak {gap} over {n}")


def test_decode_query_ranges():
    # queries of any magnitude, all zero, and with a few large features
    rng = np.random.default_rng(15)
    lens = (300,)
    cache, scales, table = make_cache(rng, lens, 64)
    x = rng.standard_normal((1, 8, 576))
    x[0, 0] = 0
    x[0, 1] *= 1e-6
    x[0, 2] *= 30
    x[0, 3, 5] = 60
    x[0, 4] *= np.exp2(rng.integers(-12, 1, 576))
    q = torch.from_numpy(x).bfloat16()
    got = run_decode(q, cache, scales, table, lens, 64)
    check_decode(got, q, cache, scales, table, lens, 64, what="query ranges")


@pytest.mark.parametrize("heads", [16, 40])
def test_decode_nan_and_infinity_stay_where_they_are(heads):
    # a query's make its head's results NaN, a key's those of its sequence
    rng = np.random.default_rng(23)
    lens = (300, 20000, 100, 65)
    cache, scales, table = make_cache(rng, lens, 64)
    q = torch.from_numpy(rng.standard_normal((4, heads, 576))).bfloat16()
    clean = run_decode(q, cache, scales, table, lens, 64)
    bad = q.clone()
    bad[0, 1, 3], bad[0, 2, 575], bad[1, 5, 0], bad[3, 0, 100] = math.nan, math.inf, -math.inf, math.nan
    cache[table[2][1] * 64 + 5, 570] = 0x7F  # the RoPE part of key 69
    got = run_decode(bad, cache, scales, table, lens, 64)
    nan = np.zeros((4, heads), bool)
    nan[0, 1] = nan[0, 2] = nan[1, 5] = nan[3, 0] = True
    nan[2] = True
    assert np.array_equal(np.isnan(got[1]), nan) and np.array_equal(np.isnan(got[0]), np.repeat(nan[..., None], 512, 2))
    assert np.array_equal(got[0][~nan], clean[0][~nan]) and np.array_equal(got[1][~nan], clean[1][~nan])
    assert got[2] == 0


@pytest.mark.parametrize("power", [-126, -100, 100, 126])
def test_decode_queries_near_the_ends_of_the_range(power):
    # scaled by a power of two, and the softmax's scale by its inverse (as far
    # as fp32 goes): the same results, within the bound
    rng = np.random.default_rng(24)
    lens = (200, 77)
    cache, scales, table = make_cache(rng, lens, 64)
    q = torch.from_numpy(rng.standard_normal((2, 20, 576))).bfloat16()
    up = 2.0 ** (power if power > 0 else power + 6)
    big = (q.double() * up).bfloat16()
    out, lse, flags = run_decode(big, cache, scales, table, lens, 64, scale=SCALE / up)
    assert flags == 0
    finite = torch.isfinite(big).all(2)  # (4 * 2^126 is an infinity)
    assert finite.float().mean() > 0.8 and np.array_equal(~np.isnan(lse), finite.numpy())
    h = finite.all(0).numpy()
    check_decode((out[:, h], lse[:, h]), big[:, h], cache, scales, table, lens, 64, scale=SCALE / up,
                 what=f"queries 2^{power}")


def test_decode_lengths_near_the_largest_integer():
    # pages of 2^30 tokens: the lengths and the blocks' indexes stay in range,
    # and what the cache does not hold is flagged and skipped
    rng = np.random.default_rng(26)
    cache, scales, _ = make_cache(rng, (128,), 64)
    cache, scales = cache[:128], scales[:2]
    cache[:] = fp8.encode(rng.standard_normal((128, 576)) * 100)
    table = np.array([[0, -1, 7], [0, 1, 2]], dtype=np.int32)
    q = torch.from_numpy(rng.standard_normal((2, 4, 576))).bfloat16()
    got = run_decode(q, cache, scales, table, (2 ** 31 - 1, 100), 2 ** 30)
    assert got[2] == 1
    check_decode(got, q, cache, scales, np.array([[0], [0]]), (128, 100), 128, what="2^31 - 1 keys")


def test_decode_more_sequences_than_threads():
    rng = np.random.default_rng(25)
    lens = tuple(int(x) for x in rng.integers(0, 70, 1100))
    cache, scales, table = make_cache(rng, lens, 64)
    q = torch.from_numpy(rng.standard_normal((len(lens), 2, 576))).bfloat16()
    for split in (True, False):
        got = run_decode(q, cache, scales, table, lens, 64, split=split)
        assert got[2] == 0
        check_decode(got, q, cache, scales, table, lens, 64, what=f"1100 sequences split={split}")


def test_decode_bad_entries_are_flagged_and_skipped():
    rng = np.random.default_rng(16)
    lens = (300, 200, 64)
    cache, scales, table = make_cache(rng, lens, 64)
    q = torch.from_numpy(rng.standard_normal((3, 16, 576))).bfloat16()
    t = table.copy()
    t[0, 1], t[0, 4], t[2, 0] = -1, len(scales), len(scales) + 5
    got = run_decode(q, cache, scales, t, lens, 64)
    assert got[2] == 1
    check_decode(got, q, cache, scales, t, lens, 64, what="bad pages")
    for bad in (0.0, -1.0, math.nan, math.inf, 2.0 ** 61, 2.0 ** -61):
        s = scales.copy()
        s[table[0, 2]] = bad
        s[table[2, 0]] = bad
        got = run_decode(q, cache, s, table, lens, 64)
        assert got[2] == 4, bad
        check_decode(got, q, cache, s, table, lens, 64, what=f"scale {bad}")
    # a length past the page table: the keys the table holds
    got = run_decode(q, cache, scales, table[:, :2].copy(), lens, 64)
    assert got[2] == 1
    check_decode(got, q, cache, scales, table[:, :2], [min(n, 128) for n in lens], 64, what="short table")
    got = run_decode(q, cache, scales, table, (-4, 200, -(2 ** 31)), 64)
    check_decode(got, q, cache, scales, table, (0, 200, 0), 64, what="negative lengths")


def test_decode_graph_streams_and_repeats():
    rng = np.random.default_rng(17)
    sets = []
    for i, lens in enumerate([(2000, 65, 1), (900, 0, 1500, 31)]):
        cache, scales, table = make_cache(rng, lens, 64)
        q = torch.from_numpy(rng.standard_normal((len(lens), 48, 576))).bfloat16().to(DEV)
        a = [torch.from_numpy(x).to(DEV) for x in (cache, scales, table)] + \
            [torch.tensor(lens, dtype=torch.int32, device=DEV)]
        ws = torch.randint(0, 256, (mla.mla_nvfp4_fp8_decode_workspace_size(len(lens), 48),), dtype=torch.uint8, device=DEV)
        out = torch.empty(len(lens), 48, 512, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(len(lens), 48, device=DEV)
        sets.append((q, a, ws, out, lse))

    def call(s):
        q, a, ws, out, lse = s
        mla.mla_nvfp4_fp8_decode(q, a[0].view(F8), a[1], SCALE, page_table=a[2], seq_lens=a[3], out=out, lse=lse,
                                 workspace=ws)

    refs = []
    for s in sets:
        call(s)
        torch.cuda.synchronize()
        refs.append((s[3].clone(), s[4].clone()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):  # two calls in one graph, the second on the first's workspace size or less
        for s in sets:
            call(s)
    for _ in range(3):
        for s in sets:
            s[3].zero_(), s[4].zero_(), s[2].fill_(255)
        g.replay()
        torch.cuda.synchronize()
        for s, r in zip(sets, refs):
            assert torch.equal(s[3], r[0]) and torch.equal(s[4], r[1])
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for s, st in zip(sets, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                s[3].zero_()
                call(s)
        torch.cuda.synchronize()
        for s, r in zip(sets, refs):
            assert torch.equal(s[3], r[0]) and torch.equal(s[4], r[1])


# ---------------------------------------------------------- quantize, GEMM
@pytest.mark.parametrize("M,K", [(1, 8), (1, 128), (3, 136), (5, 1000), (64, 7168), (257, 520), (1, 16384), (0, 128)])
def test_quantize(M, K):
    rng = np.random.default_rng(M + K)
    x = rng.standard_normal((M, K)) * np.exp2(rng.integers(-30, 31, (M, 1)))
    x[M // 2:, : min(K, 128)] = 0
    t = torch.from_numpy(x).bfloat16()
    codes, scales = mla.mla_nvfp4_fp8_quantize(t.to(DEV))
    torch.cuda.synchronize()
    rc, rs = fp8.quantize(f32(t))
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(u8(codes), rc)


def test_quantize_extreme_values_and_strides():
    x = torch.randn(6, 512).bfloat16()
    x[0, 3], x[1, 200], x[2, 300], x[3, 10] = math.inf, math.nan, -math.inf, 3e38
    x[4, :128] = 1e-40
    x[5, 128:256] = 2.0 ** -130
    wide = torch.zeros(6, 1024, dtype=torch.bfloat16)
    wide[:, 128:640] = x
    codes, scales = mla.mla_nvfp4_fp8_quantize(wide.to(DEV)[:, 128:640])
    torch.cuda.synchronize()
    rc, rs = fp8.quantize(f32(x))
    assert np.array_equal(scales.cpu().numpy(), rs)
    same_codes(u8(codes), rc, "quantize")


def make_gemm(rng, M, N, K, outliers=True):
    a = fp8.encode(rng.standard_normal((M, K)) * 100)
    w = fp8.encode(rng.standard_normal((N, K)) * 100)
    kb, nb = -(-K // 128), -(-N // 128)
    sa = np.exp2(rng.uniform(-9, 1, (M, kb))).astype(np.float32)
    sw = np.exp2(rng.uniform(-9, -4, (nb, kb))).astype(np.float32)
    return a, sa, w, sw


def run_gemm(a, sa, w, sw, **kw):
    d = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
    e = errw()
    out = mla.mla_nvfp4_fp8_gemm(d(a).view(F8), d(sa), d(w).view(F8), d(sw), error_word=e, **kw)
    torch.cuda.synchronize()
    assert int(e.item()) == 0
    return f32(out)


def check_gemm(got, a, sa, w, sw, what):
    c, mag = fp8.gemm(a, sa, w, sw)
    K = a.shape[1]
    tol = np.maximum(bf16_half_ulp(c), bf16_half_ulp(got)) + 2.0 ** -24 * (K + 2 * sa.shape[1]) * mag
    err = np.abs(got - c)
    print(f"[fp8 gemm] {what}: error {float(np.max(err / tol)):.3f} of the tolerance")
    assert np.all(err <= tol), f"{what}: {float(np.max(err / tol)):.2f} times the tolerance"


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 127, 128, 129, 200, 300])
@pytest.mark.parametrize("N,K", [(64, 128), (576, 512), (130, 144), (257, 1040), (1, 16), (1000, 2048)])
def test_gemm(M, N, K):
    rng = np.random.default_rng(M * 1000 + N + K)
    p = make_gemm(rng, M, N, K)
    check_gemm(run_gemm(*p), *p, what=f"{M}x{N}x{K}")


@pytest.mark.parametrize("M,N,K", [(1, 576, 7168), (8, 7168, 1536), (513, 1100, 4096), (1030, 640, 7168), (77, 129, 16384),
                                   (1300, 3601, 272), (2300, 2111, 400), (130, 40000, 144)])
def test_gemm_larger(M, N, K):
    rng = np.random.default_rng(M + N + K)
    p = make_gemm(rng, M, N, K)
    check_gemm(run_gemm(*p), *p, what=f"{M}x{N}x{K}")


@pytest.mark.parametrize("M,N,K", [(5, 200, 272), (150, 300, 400)])
def test_gemm_strides_and_neighbours(M, N, K):
    # operands inside wider tensors full of NaN codes; an output whose rows
    # are not 16-byte aligned, inside a wider tensor that stays as it is
    rng = np.random.default_rng(M)
    a, sa, w, sw = make_gemm(rng, M, N, K)
    wa = torch.full((M + 3, K + 64), 0x7F, dtype=torch.uint8, device=DEV)
    ww = torch.full((N + 3, K + 128), 0x7F, dtype=torch.uint8, device=DEV)
    wa[:M, 16:16 + K], ww[:N, 32:32 + K] = torch.from_numpy(a).to(DEV), torch.from_numpy(w).to(DEV)
    for left in (0, 3, 8):
        out = torch.full((M + 2, N + 13), 7.0, dtype=torch.bfloat16, device=DEV)
        got = mla.mla_nvfp4_fp8_gemm(wa.view(F8)[:M, 16:16 + K], torch.from_numpy(sa).to(DEV),
                                     ww.view(F8)[:N, 32:32 + K], torch.from_numpy(sw).to(DEV),
                                     out=out[:M, left:left + N])
        torch.cuda.synchronize()
        check_gemm(f32(got), a, sa, w, sw, f"strided, out at column {left}")
        rest = out.clone()
        rest[:M, left:left + N] = 7.0
        assert torch.all(rest == 7.0)


@pytest.mark.parametrize("N,wide,left", [(2104, 2112, 0), (2093, 2112, 16), (2104, 2104, 0), (2103, 2104, 1),
                                         (2101, 2103, 1)])
def test_gemm_large_tiles_outputs(N, wide, left):
    # rows of the output at multiples of 32 bytes, of 16, of 2: many rows, one
    # wave of large tiles, whose last ones are ragged in both directions
    M, K = 1300, 272
    rng = np.random.default_rng(N + left)
    a, sa, w, sw = make_gemm(rng, M, N, K)
    d = [torch.from_numpy(x).to(DEV) for x in (a, sa, w, sw)]
    out = torch.full((M + 2, wide), 7.0, dtype=torch.bfloat16, device=DEV)
    got = mla.mla_nvfp4_fp8_gemm(d[0].view(F8), d[1], d[2].view(F8), d[3], out=out[:M, left:left + N])
    torch.cuda.synchronize()
    check_gemm(f32(got), a, sa, w, sw, f"{M}x{N}x{K}, rows of {wide}")
    rest = out.clone()
    rest[:M, left:left + N] = 7.0
    assert torch.all(rest == 7.0)


@pytest.mark.parametrize("M", [16, 32, 64, 128, 640])
def test_gemm_many_blocks(M):
    # many K blocks a CTA in every form, so that each stage is filled several
    # times; ten tiles of weights, repeated
    rng = np.random.default_rng(M)
    a, sa, w, sw = make_gemm(rng, M, 1280, 4112)
    got = run_gemm(a, sa, np.tile(w, (20, 1)), np.tile(sw, (20, 1)))
    check_gemm(got[:, :1280], a, sa, w, sw, f"{M}x25600x4112")
    for i in range(1, 20):
        assert np.array_equal(got[:, :1280], got[:, 1280 * i:1280 * (i + 1)])


def test_gemm_graph_and_streams():
    rng = np.random.default_rng(21)
    ps = [make_gemm(rng, 9, 700, 1024), make_gemm(rng, 260, 520, 512)]
    d = [[torch.from_numpy(x).to(DEV) for x in p] for p in ps]
    outs = [torch.empty(p[0].shape[0], p[2].shape[0], dtype=torch.bfloat16, device=DEV) for p in ps]

    def call(i):
        a, sa, w, sw = d[i]
        mla.mla_nvfp4_fp8_gemm(a.view(F8), sa, w.view(F8), sw, out=outs[i])

    refs = []
    for i in range(2):
        call(i)
        torch.cuda.synchronize()
        refs.append(outs[i].clone())
        check_gemm(f32(outs[i]), *ps[i], what="before capture")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(0), call(1)
    for _ in range(2):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, r) for o, r in zip(outs, refs))
    streams = [torch.cuda.Stream() for _ in ps]
    for i, st in enumerate(streams):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            outs[i].zero_()
            call(i)
    torch.cuda.synchronize()
    assert all(torch.equal(o, r) for o, r in zip(outs, refs))


# ------------------------------------------------------------- as it is used
def test_a_layer_in_8_bits():
    """Prefill of two prompts, then two decode steps: hidden -> quantize ->
    gemm (latent and RoPE key) -> append -> decode -> quantize -> gemm, each
    step against the oracle on what the previous one gave."""
    rng = np.random.default_rng(31)
    hidden, H, B = 512, 8, 2
    w_kv = fp8.encode(rng.standard_normal((576, hidden)) * 60)
    s_kv = np.full((5, 4), 2.0 ** -11, np.float32)
    w_o = fp8.encode(rng.standard_normal((hidden, H * 512)) * 60)
    s_o = np.full((4, 32), 2.0 ** -12, np.float32)
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
    table, pages = pages_for(rng, (200, 130), 64)
    cache, scales = torch.zeros(pages * 64, 576, dtype=torch.uint8, device=DEV), torch.zeros(pages, device=DEV)
    rc, rs = np.zeros((pages * 64, 576), np.uint8), np.zeros(pages, np.float32)
    cs = angles(256)
    lens = np.zeros(B, np.int32)
    e = errw()
    for new in ((197, 64), (1, 1), (1, 1)):
        T = sum(new)
        x = torch.from_numpy(rng.standard_normal((T, hidden))).bfloat16().to(DEV)
        xa, xs = mla.mla_nvfp4_fp8_quantize(x)
        kv = mla.mla_nvfp4_fp8_gemm(xa, xs, d(w_kv).view(F8), d(s_kv))
        check_gemm(f32(kv), u8(xa), xs.cpu().numpy(), w_kv, s_kv, "latent")
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        q = torch.from_numpy(rng.standard_normal((T, H, 576)) * 0.3).bfloat16().to(DEV)
        qr = f32(q)
        mla.mla_nvfp4_fp8_cache_append(kv[:, :512], kv[:, 512:], d(cs), d(cu), d(lens), d(table), cache.view(F8), scales,
                                       q_pe=q[:, :, 512:], q_out=q[:, :, 512:], max_new_tokens=max(new), error_word=e)
        fp8.append(rc, rs, f32(kv[:, :512]), f32(kv[:, 512:]), cs, cu, lens, table, 64, True)
        assert np.array_equal(scales.cpu().numpy(), rs)
        same_codes(u8(cache), rc, "layer append")
        pos = np.concatenate([lens[b] + np.arange(new[b]) for b in range(B)])
        qr[:, :, 512:] = f32(torch.from_numpy(fp8.rotate(qr[:, :, 512:], cs[pos][:, None], True)).bfloat16())
        lens = lens + np.asarray(new, np.int32)
        last = cu[1:] - 1  # the newest token of each sequence attends to all its keys
        qd = q[torch.from_numpy(last).long().to(DEV)].contiguous()
        assert np.array_equal(f32(qd), qr[last])
        out, lse = mla.mla_nvfp4_fp8_decode(qd, cache.view(F8), scales, SCALE, page_table=d(table), seq_lens=d(lens),
                                            return_lse=True, error_word=e)
        torch.cuda.synchronize()
        check_decode((f32(out), f32(lse)), qd, rc, rs, table, lens, 64, what="layer")
        oa, os_ = mla.mla_nvfp4_fp8_quantize(out.view(B, H * 512))
        y = mla.mla_nvfp4_fp8_gemm(oa, os_, d(w_o).view(F8), d(s_o))
        check_gemm(f32(y), u8(oa), os_.cpu().numpy(), w_o, s_o, "output projection")
    assert int(e.item()) == 0


# ----------------------------------------------------------------- refusals
def test_calls_refuse_wrong_tensors():
    """Shapes, types, strides and pairs the calls do not take; nothing runs."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device=DEV)  # noqa: E731
    i32 = torch.int32
    cache, scales = z(128, 576, dt=torch.uint8).view(F8), z(2, dt=torch.float32)
    good = dict(kv_c=z(3, 512), k_pe=z(3, 64), cos_sin=z(8, 64, dt=torch.float32), cu_seqlens=z(2, dt=i32),
                context_lens=z(1, dt=i32), page_table=z(1, 2, dt=i32), cache=cache, scales=scales)
    for name, bad in dict(kv_c=z(3, 500), k_pe=z(2, 64), cos_sin=z(8, 32, dt=torch.float32), cu_seqlens=z(3, dt=i32),
                          context_lens=z(1, dt=torch.int64), page_table=z(2, 2, dt=i32), cache=z(100, 576, dt=torch.uint8).view(F8),
                          scales=z(3, dt=torch.float32)).items():
        with pytest.raises(ValueError):
            mla.mla_nvfp4_fp8_cache_append(**dict(good, **{name: bad}))
    for kw in (dict(q_out=z(3, 4, 64)), dict(q_pe=z(3, 4, 32)), dict(q_pe=z(2, 4, 64)), dict(page_size=96),
               dict(q_pe=z(3, 4, 64), q_out=z(3, 5, 64)), dict(kv_c=z(512, 3).t()), dict(error_word=z(1))):
        with pytest.raises(ValueError):
            mla.mla_nvfp4_fp8_cache_append(**dict(good, **kw))
    with pytest.raises(mla.MLAError):  # rows that are not 16-byte aligned
        mla.mla_nvfp4_fp8_cache_append(**dict(good, kv_c=z(3, 513)[:, :512]))
    dec = dict(q=z(1, 16, 576), cache=cache, scales=scales, softmax_scale=0.1, page_table=z(1, 2, dt=i32), seq_lens=z(1, dt=i32))
    for kw in (dict(q=z(1, 16, 512)), dict(q=z(1, 16, 1152)[:, :, :576]), dict(seq_lens=z(2, dt=i32)), dict(page_size=0),
               dict(out=z(1, 16, 576)), dict(lse=z(1, 8, dt=torch.float32)), dict(workspace=z(8, dt=torch.float32)),
               dict(split=False, workspace=z(1 << 20, dt=torch.uint8))):
        with pytest.raises(ValueError):
            mla.mla_nvfp4_fp8_decode(**dict(dec, **kw))
    for kw in (dict(softmax_scale=0.0), dict(softmax_scale=math.nan), dict(workspace=z(64, dt=torch.uint8))):
        with pytest.raises(mla.MLAError):
            mla.mla_nvfp4_fp8_decode(**dict(dec, **kw))
    for bad in (z(4), z(4, 8, dt=torch.float16), z(8, 4).t()):
        with pytest.raises(ValueError):
            mla.mla_nvfp4_fp8_quantize(bad)
    with pytest.raises(mla.MLAError):
        mla.mla_nvfp4_fp8_quantize(z(4, 12))
    a, sa = z(4, 256, dt=torch.uint8).view(F8), z(4, 2, dt=torch.float32)
    w, sw = z(130, 256, dt=torch.uint8).view(F8), z(2, 2, dt=torch.float32)
    for args in ((a, sa, w[:, :240], sw), (a, sa[:, :1], w, sw), (a, sa, w, sw[:1]), (a, sa.t(), w, sw)):
        with pytest.raises(ValueError):
            mla.mla_nvfp4_fp8_gemm(*args)
    with pytest.raises(ValueError):
        mla.mla_nvfp4_fp8_gemm(a, sa, w, sw, out=z(4, 131))
    # nothing to do
    assert mla.mla_nvfp4_fp8_gemm(a[:0], sa[:0], w, sw).shape == (0, 130)
    assert mla.mla_nvfp4_fp8_quantize(z(0, 128))[1].shape == (0, 1)
    assert mla.mla_nvfp4_fp8_decode(**dict(dec, q=z(0, 16, 576), page_table=z(0, 2, dt=i32), seq_lens=z(0, dt=i32))).shape == (0, 16, 512)
    mla.mla_nvfp4_fp8_cache_append(**dict(good, kv_c=z(0, 512), k_pe=z(0, 64)))
    torch.cuda.synchronize()
