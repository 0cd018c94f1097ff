"""The e4m3 decode of a batch with a shared prefix on the GPU against the
float64 oracle, which attends to every sequence by itself.  The kernel's
operands and roundings are those of the decode, so the tolerances are
tests/test_gpu_fp8.py's (check_decode): its derivation bounds each key's weight
relative to the largest of the same piece, and sums of any order."""
import numpy as np
import pytest
import torch

import mla_attention_nvfp4_gb300 as mla
from oracle import fp8, gemm
from tests.fp8_cases import wide_query
from tests.helpers import bf16_half_ulp, f32
from tests.test_gpu_fp8 import DEV, F8, SCALE, angles, check_decode, errw, run_decode
from tests.test_gpu_gemv import rows, weights

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
FAR = 1 << 30  # an entry that is not read


def t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def make(rng, shared, lens, page, scales=(-7, -6)):
    """A batch of total lengths `lens`; (cache, scales, page table, the blocks of each sequence as the oracle reads them).
    Entries and slots that the call must not read are out of range and any bytes."""
    B = len(lens)
    whole, cut = shared // page, shared % page
    width = max(1, -(-max(max(lens), shared) // page)) + 1
    table = np.full((B, width), FAR, np.int32)
    own = []  # (sequence, entry) of pages of its own
    for b, n in enumerate(lens):
        first = whole if n >= shared else 0
        own += [(b, i) for i in range(first, -(-n // page))]
    prefix = whole + (1 if cut and any(n >= shared for n in lens) else 0)
    if any(n >= shared for n in lens):
        own += [(0, i) for i in range(prefix) if (0, i) not in own]
    ids = rng.permutation(len(own) + 2)
    for (b, i), p in zip(own, ids):
        table[b, i] = p
    per = page // 64
    slots = len(ids) * page
    cache = rng.integers(0, 256, (slots, 576), dtype=np.uint8)
    sc = np.exp2(rng.integers(scales[0], scales[1] + 1, slots // 64)).astype(np.float32)
    eff = np.full((B, max(1, -(-max(lens) // 64))), FAR, np.int32)
    for b, n in enumerate(lens):
        for i in range(-(-n // 64)):
            owner = 0 if i * 64 < shared <= n else b
            eff[b, i] = table[owner, i // per] * per + i % per
    for blk, last in {(int(eff[b, i]), min(64, n - 64 * i)) for b, n in enumerate(lens) for i in range(-(-n // 64))}:
        x = rng.standard_normal((last, 576))
        x[:, :512] *= np.where(rng.random((last, 512)) < 0.01, 20, 1)
        cache[blk * 64:blk * 64 + last] = fp8.encode(x * 128)
    return cache, sc, table, eff


def run(q, cache, scales, table, lens, shared, page, scale=SCALE, **kw):
    e = errw()
    out, lse = mla.mla_nvfp4_fp8_decode_shared(
        q.to(DEV), t(cache).view(F8), t(scales), scale, page_table=t(table),
        seq_lens=torch.tensor(list(lens), dtype=torch.int32, device=DEV), shared_len=shared, page_size=page, return_lse=True,
        error_word=e, **kw)
    torch.cuda.synchronize()
    return f32(out), f32(lse), int(e.item())


def queries(rng, B, H):
    return torch.from_numpy(rng.standard_normal((B, H, 576))).bfloat16()


@pytest.mark.parametrize("heads", [1, 5, 16, 31, 32, 33, 64, 65, 128, 130])
@pytest.mark.parametrize("shared", [64, 192, 1024])
def test_shared_heads(heads, shared):
    rng = np.random.default_rng(heads + shared)
    lens = tuple(shared + n for n in (1, 0, 63, 64, 65, 128, 129, 300))
    c = make(rng, shared, lens, 64)
    q = queries(rng, len(lens), heads)
    got = run(q, *c[:3], lens, shared, 64)
    assert got[2] == 0
    check_decode(got, q, c[0], c[1], c[3], lens, 64, what=f"{heads} heads, {shared} shared")


@pytest.mark.parametrize("page", [64, 128, 192, 1024])
@pytest.mark.parametrize("shared,own", [(5056, (1,)), (320, (0, 0)), (64, (64,) * 40), (704, (2, 0, 4097) * 3),
                                        (128, (1,) * 160), (2048, (100,) * 7), (64, tuple(range(0, 400, 3)))])
def test_shared_lengths(page, shared, own):
    rng = np.random.default_rng(page + len(own))
    lens = tuple(shared + n for n in own)
    c = make(rng, shared, lens, page)
    q = queries(rng, len(lens), 12)
    got = run(q, *c[:3], lens, shared, page)
    assert got[2] == 0
    check_decode(got, q, c[0], c[1], c[3], lens, 64, what=f"page {page}, {shared} + {len(own)}")


@pytest.mark.parametrize("heads", [3, 40])
def test_shared_with_shorter_and_empty_sequences(heads):
    # a padded batch: empty rows, rows below the prefix (read through their own pages), row 0 among them
    rng = np.random.default_rng(heads)
    for lens in ((0, 400, 0, 320, 321), (100, 400, 319, 0, 320, 64, 1), (0, 0, 0), (5, 100), (500, 0)):
        c = make(rng, 320, lens, 64)
        q = queries(rng, len(lens), heads)
        got = run(q, *c[:3], lens, 320, 64)
        assert got[2] == 0
        check_decode(got, q, c[0], c[1], c[3], lens, 64, what=f"{lens}")
        empty = np.asarray(lens) == 0
        assert not got[0][empty].any() and np.all(np.isneginf(got[1][empty]))


def test_shared_of_nothing_is_the_decode():
    rng = np.random.default_rng(1)
    lens = (700, 0, 65, 3000)
    c = make(rng, 0, lens, 64)
    q = queries(rng, 4, 16)
    got = run(q, *c[:3], lens, 0, 64)
    assert got[2] == 0
    check_decode(got, q, c[0], c[1], c[3], lens, 64, what="nothing shared")


def test_shared_whole_table_and_long():
    rng = np.random.default_rng(2)
    for shared, own, heads in ((20032, (3, 0, 150, 2000), 16), (20032, (0,) * 11, 128), (40000, (5, 700), 2)):
        lens = tuple(shared + n for n in own)
        c = make(rng, shared, lens, 64)
        q = queries(rng, len(lens), heads)
        got = run(q, *c[:3], lens, shared, 64)
        assert got[2] == 0
        check_decode(got, q, c[0], c[1], c[3], lens, 64, what=f"{shared} shared, {heads} heads")


def test_shared_one_page_table_row_for_all():
    # an expanded row: the batch asks about one text, to different places of it
    rng = np.random.default_rng(3)
    lens = (700, 640, 699, 650)
    c = make(rng, 700 // 64 * 64, (700,), 64)
    table = np.repeat(c[2], 4, 0)
    q = queries(rng, 4, 16)
    e = errw()
    out, lse = mla.mla_nvfp4_fp8_decode_shared(
        q.to(DEV), t(c[0]).view(F8), t(c[1]), SCALE, page_table=t(c[2]).expand(4, -1),
        seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV), shared_len=640, return_lse=True, error_word=e)
    torch.cuda.synchronize()
    assert int(e.item()) == 0
    check_decode((f32(out), f32(lse)), q, c[0], c[1], np.repeat(c[3], 4, 0), lens, 64, what="one row")
    own = run(q, c[0], c[1], table, lens, 640, 64)
    assert np.array_equal(own[0], f32(out)) and np.array_equal(own[1], f32(lse))


@pytest.mark.parametrize("heads", [4, 40])
def test_shared_scores_that_jump(heads):
    # the largest score of each part of a sequence far above the one before, in the prefix or behind it
    rng = np.random.default_rng(heads)
    shared, lens = 1280, (1280 + 700, 1280, 1280 + 1, 1280 + 64)
    for order in (1, -1):
        cache, scales, table, eff = make(rng, shared, lens, 64, scales=(-7, -7))
        steps = np.linspace(0, 1, 31)[::order]
        for i in range(31):
            for b in range(4):
                if eff[b, min(i, eff.shape[1] - 1)] < FAR and i * 64 < lens[b]:
                    blk = int(eff[b, i])
                    cache[blk * 64:blk * 64 + 64, 570] = fp8.encode(np.full(64, 400 * steps[i]))
        q = queries(rng, 4, heads)
        q[:, :, 570] = 600
        got = run(q, cache, scales, table, lens, shared, 64)
        assert got[2] == 0
        check_decode(got, q, cache, scales, eff, lens, 64, what=f"jumps, order {order}")


def test_shared_nan_and_infinity():
    rng = np.random.default_rng(5)
    shared, lens, H = 256, (300, 256, 200, 700), 20
    c = make(rng, shared, lens, 64)
    q = queries(rng, 4, H)
    clean = run(q, *c[:3], lens, shared, 64)
    for value in (float("nan"), float("inf")):
        bad = q.clone()
        bad[1, 3, 5] = value
        out, lse, flags = run(bad, *c[:3], lens, shared, 64)
        assert flags == 0 and np.all(np.isnan(out[1, 3])) and np.isnan(lse[1, 3])
        out[1, 3], lse[1, 3] = clean[0][1, 3], clean[1][1, 3]
        assert np.array_equal(out, clean[0]) and np.array_equal(lse, clean[1])
    # a NaN code in a shared key: every sequence that has the prefix, and no other
    cache = c[0].copy()
    cache[int(c[3][0, 2]) * 64 + 9, 30] = 0xFF
    out, lse, _ = run(q, cache, *c[1:3], lens, shared, 64)
    assert np.all(np.isnan(lse[[0, 1, 3]])) and np.array_equal(out[2], clean[0][2]) and np.array_equal(lse[2], clean[1][2])
    # in an own key: that sequence alone
    cache = c[0].copy()
    cache[int(c[3][3, 6]) * 64 + 9, 30] = 0x7F
    out, lse, _ = run(q, cache, *c[1:3], lens, shared, 64)
    assert np.all(np.isnan(lse[3])) and np.array_equal(out[:3], clean[0][:3])


@pytest.mark.parametrize("heads", [16, 40])
def test_shared_scores_past_the_range(heads):
    # above fp32's range: NaN, wherever the key lies; below it in the whole prefix: no weight; everywhere: NaN
    rng = np.random.default_rng(6)
    shared, lens = 1024, (1500, 1024, 1100)
    cache, scales, table, eff = make(rng, shared, lens, 64)
    scales[:] = 2.0 ** 8
    flat = eff[eff < FAR]
    cache.reshape(-1, 64, 576)[flat, :, 3] = 0
    cache.reshape(-1, 64, 576)[eff[0, :16], :, 3] = 0x7E
    q = torch.zeros(3, heads, 576, dtype=torch.bfloat16)
    q[0, 1, 3] = q[1, 2, 3] = -(2.0 ** 120)
    q[2, 5, 3] = 2.0 ** 120
    out, lse, flags = run(q, cache, scales, table, lens, shared, 64)
    assert flags == 0 and abs(lse[0, 1] - np.log(1500 - 1024)) < 1e-4 and np.all(np.isfinite(out[0]))
    assert np.isnan(lse[1, 2]) and np.all(np.isnan(out[1, 2])) and np.isnan(lse[2, 5]) and np.all(np.isnan(out[2, 5]))
    assert np.all(np.isfinite(np.delete(out[1], 2, 0))) and np.all(np.isfinite(np.delete(out[2], 5, 0)))


def test_shared_bad_entries():
    rng = np.random.default_rng(7)
    shared, lens, H = 256, (300, 256, 200, 700), 20
    c = make(rng, shared, lens, 64)
    q = queries(rng, 4, H)
    for change in ("shared page", "shared page neg", "shared scale", "own page", "length"):
        cache, sc, table, eff = (x.copy() for x in c)
        ln = list(lens)
        if change.startswith("shared page"):
            table[0, 1] = len(cache) // 64 if "neg" not in change else -7
            eff[[0, 1, 3], 1] = table[0, 1]
        elif change == "shared scale":
            sc[table[0, 1]] = np.nan
        elif change == "own page":
            table[3, 8] = eff[3, 8] = len(cache) // 64
        else:
            table = table[:, :11].copy()
            ln[3] = 704
        got = run(q, cache, sc, table, lens, shared, 64)
        assert got[2] == (4 if change == "shared scale" else 0 if change == "length" else 1), change
        check_decode(got, q, cache, sc, eff, lens, 64, what=change)
    got = run(q, c[0], c[1], c[2][:, :10], (300, 256, 200, 641), 256, 64)
    assert got[2] == 1  # 640 of 641 keys
    check_decode(got, q, c[0], c[1], c[3], (300, 256, 200, 640), 64, what="a length past the table")


@pytest.mark.parametrize("heads", [16, 40])
def test_shared_queries_of_wide_range(heads):
    q, k = wide_query(heads, 2.0 ** 12)
    n = len(k)
    cache = np.zeros((320, 576), np.uint8)
    cache[:n] = fp8.encode(k)
    table = np.arange(5, dtype=np.int32)[None]
    got = run(q, cache, np.full(5, 2.0 ** -20, np.float32), table, (n,), 128, 64)
    assert got[2] == 0
    check_decode(got, q, cache, np.full(5, 2.0 ** -20, np.float32), table, (n,), 64, what="wide query")


def test_shared_refusals():
    rng = np.random.default_rng(8)
    lens = (300, 256)
    c = make(rng, 256, lens, 64)
    q = queries(rng, 2, 4)
    for kw in (dict(shared=100), dict(shared=-64), dict(shared=64 * 100)):
        with pytest.raises((ValueError, mla.MLAError)):
            run(q, *c[:3], lens, kw["shared"], 64)
    small = torch.empty(mla.mla_nvfp4_fp8_decode_shared_workspace_size(2, 4) - 1, dtype=torch.uint8, device=DEV)
    with pytest.raises(mla.MLAError, match="WORKSPACE"):
        run(q, *c[:3], lens, 256, 64, workspace=small)
    with pytest.raises(ValueError):
        run(q.float(), *c[:3], lens, 256, 64)
    with pytest.raises(ValueError):
        run(q, *c[:3], lens[:1], 256, 64)


def test_shared_graph_streams_and_repeats():
    rng = np.random.default_rng(9)
    shared, lens, H = 4096, (4096 + 700, 4096, 4096 + 9, 17, 4096 + 64), 16
    c = make(rng, shared, lens, 64)
    q = queries(rng, 5, H).to(DEV)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    args = (q, t(c[0]).view(F8), t(c[1]), SCALE)
    kw = dict(page_table=t(c[2]), seq_lens=ln, shared_len=shared, return_lse=True)
    plain = mla.mla_nvfp4_fp8_decode_shared(*args, **kw)
    size = mla.mla_nvfp4_fp8_decode_shared_workspace_size(5, H)
    dirty = [torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for w, st in zip(dirty, streams):
            with torch.cuda.stream(st):
                got.append(mla.mla_nvfp4_fp8_decode_shared(*args, **kw, workspace=w))
    torch.cuda.synchronize()
    assert all(torch.equal(o, plain[0]) and torch.equal(x, plain[1]) for o, x in got)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = mla.mla_nvfp4_fp8_decode_shared(*args, **kw)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(held[0], plain[0]) and torch.equal(held[1], plain[1])
    now = (4096 + 650, 100, 4096, 0, 4096 + 1)  # a replay reads the lengths anew
    eff = c[3].copy()
    eff[1, :2] = c[2][1, :2]
    cache2, sc2, tab2, eff2 = make(rng, shared, now, 64)
    ln.copy_(torch.tensor(now, dtype=torch.int32))
    kw2 = dict(kw, page_table=t(tab2))
    fresh = mla.mla_nvfp4_fp8_decode_shared(q, t(cache2).view(F8), t(sc2), SCALE, **kw2)
    torch.cuda.synchronize()
    check_decode((f32(fresh[0]), f32(fresh[1])), q.cpu(), cache2, sc2, eff2, now, 64, what="other lengths")


def test_shared_calls_in_a_row_read_what_the_work_ahead_wrote():
    rng = np.random.default_rng(12)
    shared, lens, H = 512, (700, 512, 513, 100), 16
    c = make(rng, shared, lens, 64)
    qs = [queries(rng, 4, H).to(DEV) for _ in range(3)]
    lengths = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (lens, (650, 512, 600, 100), (512, 512, 512, 64))]
    lengths[1][2] = 513
    args, kw = (t(c[0]).view(F8), t(c[1]), SCALE), dict(page_table=t(c[2]), shared_len=shared, return_lse=True)
    ref = []
    for q, ln in zip(qs, lengths):
        ref.append(mla.mla_nvfp4_fp8_decode_shared(q, *args, seq_lens=ln, **kw))
        torch.cuda.synchronize()
    q, ln, got = torch.empty_like(qs[0]), torch.empty_like(lengths[0]), []
    ws = torch.empty(mla.mla_nvfp4_fp8_decode_shared_workspace_size(4, H), dtype=torch.uint8, device=DEV)
    for i in range(90):
        q.copy_(qs[i % 3])
        ln.copy_(lengths[i % 3])
        got.append(mla.mla_nvfp4_fp8_decode_shared(q, *args, seq_lens=ln, workspace=ws, **kw))
    torch.cuda.synchronize()
    for i, (o, x) in enumerate(got):
        assert torch.equal(o, ref[i % 3][0]) and torch.equal(x, ref[i % 3][1]), i


def test_shared_agrees_with_the_decode_on_the_same_sequences():
    rng = np.random.default_rng(10)
    shared, lens, H = 512, (700, 512, 513), 128
    c = make(rng, shared, lens, 64)
    q = queries(rng, 3, H)
    table = c[3].copy()
    a, b = run(q, *c[:3], lens, shared, 64), run_decode(q, c[0], c[1], table, lens, 64)
    oabs = fp8.decode(f32(q), c[0], c[1], SCALE, table, lens, 64)[2]
    # each within half a bf16 step and 2^-8 of sum p |v| of the same value
    assert np.all(np.abs(a[0] - b[0]) <= bf16_half_ulp(a[0]) + bf16_half_ulp(b[0]) + 2.0 ** -6 * oabs)
    assert np.allclose(a[1], b[1], atol=1e-4)


def test_one_decode_step_of_four_bit_projections_around_a_shared_prefix():
    """Hidden states to queries by the heads' 4-bit matrices (W_UK), the new token appended, the shared decode, and its
    output by the heads' W_UV and the output projection: each call's result against the oracle on the call's own inputs."""
    rng = np.random.default_rng(11)
    B, H, shared = 3, 16, 256
    before = (256 + 40, 256, 256 + 7)
    lens = tuple(n + 1 for n in before)
    cache, sc, table, eff = make(rng, shared, lens, 64)
    one = torch.ones(1, device=DEV)
    g = np.float32(0.02)
    gs = torch.tensor([g], device=DEV)

    def gemv(x, w, what):
        got = mla.mla_nvfp4_gemv(x, t(w[0]) if x.dim() == 3 else t(w[0][0]), t(w[1]) if x.dim() == 3 else t(w[1][0]), gs)
        xs = f32(x) if x.dim() == 3 else f32(x)[:, None]
        ref, mag, wsum = gemm.gemv(xs, *w, w[0].shape[1], 2 * w[0].shape[2], g)
        a = f32(got) if x.dim() == 3 else f32(got)[:, None]
        tol = np.maximum(bf16_half_ulp(ref), bf16_half_ulp(a)) + 4.0 * w[0].shape[2] * 2.0 ** -24 * mag
        tol = tol + 2.0 ** -39 * np.abs(xs).max(2)[..., None] * wsum[None] + 1e-36
        assert np.all(np.abs(a - ref) <= tol), what
        return got

    w_q, w_uk = weights(rng, 1, H * 192, 512), weights(rng, H, 512, 128)
    w_uv, w_o = weights(rng, H, 128, 512), weights(rng, 1, 300, H * 128)
    hidden = rows(rng, B, 1, 512)[:, 0].to(DEV)
    full = gemv(hidden, w_q, "queries").view(B, H, 192)
    q = torch.empty((B, H, 576), dtype=torch.bfloat16, device=DEV)
    q[:, :, :512] = gemv(full[:, :, :128], w_uk, "into the latent's space") * 0.02
    q_pe = full[:, :, 128:].contiguous() * 0.02
    kv, pe = (torch.from_numpy(rng.standard_normal((B, d))).bfloat16() for d in (512, 64))
    cs, cu = angles(400), np.arange(B + 1, dtype=np.int32)
    e, dc, ds = errw(), t(cache), t(sc)
    ctx = torch.tensor(before, dtype=torch.int32, device=DEV)
    mla.mla_nvfp4_fp8_cache_append(kv.to(DEV), pe.to(DEV), t(cs), t(cu), ctx, t(table), dc.view(F8), ds, q_pe=q_pe,
                                   q_out=q[:, :, 512:], error_word=e)
    fp8.append(cache, sc, f32(kv), f32(pe), cs, cu, before, np.where(table < FAR, table, 0), 64, True)
    out, lse = mla.mla_nvfp4_fp8_decode_shared(q, dc.view(F8), ds, SCALE, page_table=t(table), seq_lens=ctx + 1,
                                               shared_len=shared, return_lse=True, error_word=e)
    torch.cuda.synchronize()
    assert int(e.item()) == 0
    check_decode((f32(out), f32(lse)), q.cpu(), cache, sc, eff, lens, 64, what="step")
    values = gemv(out, w_uv, "values")
    final = gemv(values.reshape(B, H * 128), w_o, "output")
    assert final.shape == (B, 300) and bool(torch.isfinite(final).all()) and float(one) == 1


@pytest.mark.parametrize("heads", [16, 40, 128])
def test_shared_replays_read_lengths_pages_and_keys_anew(heads):
    """One captured call (its plan, cuts and first lists are made on the device) over batches of other lengths, among them one
    that falls below the prefix, empty ones, and one that shares with nobody; and the first batch again."""
    rng = np.random.default_rng(50 + heads)
    shared = 1024
    batches = [(1024 + 700, 1024, 1024 + 9, 17, 1024 + 64), (1024 + 650, 100, 1024, 0, 1024 + 1), (0, 0, 1024 + 300, 1023, 0),
               (64, 1, 0, 1000, 960), (0,) * 5, (1024 + 3000, 1024 + 3000, 5, 1024 + 1, 1024)]
    made = [make(rng, shared, lens, 64) for lens in batches]
    slots, width = max(c[0].shape[0] for c in made), max(c[2].shape[1] for c in made)
    cache = torch.zeros((slots, 576), dtype=torch.uint8, device=DEV)
    sc = torch.ones(slots // 64, device=DEV)
    table = torch.full((5, width), FAR, dtype=torch.int32, device=DEV)
    ln = torch.zeros(5, dtype=torch.int32, device=DEV)
    qs = [queries(rng, 5, heads) for _ in batches]
    q, e = torch.empty((5, heads, 576), dtype=torch.bfloat16, device=DEV), errw()

    def put(i):
        c = made[i]
        cache[:c[0].shape[0]].copy_(t(c[0]))
        sc[:c[1].shape[0]].copy_(t(c[1]))
        table.fill_(FAR)
        table[:, :c[2].shape[1]].copy_(t(c[2]))
        ln.copy_(torch.tensor(batches[i], dtype=torch.int32))
        q.copy_(qs[i])

    def call():
        return mla.mla_nvfp4_fp8_decode_shared(q, cache.view(F8), sc, SCALE, page_table=table, seq_lens=ln, shared_len=shared,
                                               return_lse=True, error_word=e)

    put(0)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = call()
    for i in list(range(len(batches))) + [0]:
        put(i)
        for x in held:
            x.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        eager = call()
        torch.cuda.synchronize()
        assert int(e.item()) == 0, batches[i]
        assert torch.equal(held[0], eager[0]) and torch.equal(held[1], eager[1]), batches[i]
        check_decode((f32(held[0]), f32(held[1])), qs[i], *made[i][:2], made[i][3], batches[i], 64, what=f"replay of {batches[i]}")
