"""Calls of the 8-bit path's Python functions that their documentation allows
or forbids, beside those of tests/test_gpu_fp8.py."""
import numpy as np
import pytest
import torch

import mla_attention_nvfp4_gb300 as mla
from oracle import fp8
from tests.helpers import f32
from tests.test_gpu_fp8 import F8, SCALE, check_append, check_decode, errw, make_append, make_cache, run_decode, u8

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
DEV = "cuda:0"


def append(c, q=None, q_out=None, **kw):
    d = {k: torch.from_numpy(c[k]).to(DEV) for k in ("cu", "ctx", "cs", "table", "cache", "scales")}
    e = errw()
    got = mla.mla_nvfp4_fp8_cache_append(c["kv"].to(DEV), c["pe"].to(DEV), d["cs"], d["cu"], d["ctx"], d["table"],
                                         d["cache"].view(F8), d["scales"], page_size=c["page"], q_pe=q, q_out=q_out,
                                         error_word=e, **kw)
    torch.cuda.synchronize()
    assert int(e.item()) == 0
    return u8(d["cache"]), d["scales"].cpu().numpy(), None if got is None else f32(got)


@pytest.mark.parametrize("bad", [-1, -(2 ** 31), -(2 ** 31) - 1, 3 - 2 ** 32, 2 ** 31, 2 ** 32 + 3, 2 ** 63 - 1])
def test_append_refuses_max_new_tokens_out_of_range(bad):
    # (3 - 2^32 and 2^32 + 3 have the low 32 bits of 3)
    c = make_append(np.random.default_rng(0), (3,), (0,), 64, 0)
    with pytest.raises((ValueError, mla.MLAError)):
        append(c, max_new_tokens=bad)


@pytest.mark.parametrize("new,ctx", [((5, 70, 1), (60, 3, 128)), ((1,), (7,)), ((1, 1), (0, 64))])
@pytest.mark.parametrize("heads", [1, 4, 33])
@pytest.mark.parametrize("order", ["head-major", "head-major inside wider rows", "head-major out only"])
def test_append_rotates_queries_of_either_order(order, heads, new, ctx):
    c = make_append(np.random.default_rng(heads), new, ctx, 64, heads)
    T, q = sum(new), c["q"].to(DEV)
    by_head = torch.zeros(heads, T, 72 if "wider" in order else 64, dtype=torch.bfloat16, device=DEV)
    view = by_head[:, :, :64].transpose(0, 1)
    if order == "head-major out only":
        got = append(c, q=q, q_out=view)
    else:
        view.copy_(q)
        got = append(c, q=view, q_out=view)
        assert not by_head[:, :, 64:].any()
    check_append(c, got, True, T)


def test_append_refuses_queries_that_overlap():
    c = make_append(np.random.default_rng(1), (3,), (0,), 64, 4)
    q = c["q"].to(DEV)
    flat = torch.zeros(3 * 4 * 64 + 64, dtype=torch.bfloat16, device=DEV)
    for strides in ((64, 64, 1), (128, 64, 1), (64, 128, 1), (0, 64, 1), (256, 0, 1), (256, 56, 1)):
        bad = flat.as_strided((3, 4, 64), strides)
        with pytest.raises(mla.MLAError):
            append(c, q=q, q_out=bad)
        with pytest.raises(mla.MLAError):
            append(c, q=bad, q_out=bad)


@pytest.mark.parametrize("split", [True, False])
def test_decode_reads_one_page_table_for_all_sequences(split):
    # several queries of one cached text: an expanded row
    rng = np.random.default_rng(3)
    n, lens = 700, (700, 1, 513, 700)
    cache, scales, table = make_cache(rng, (n,), 64)
    q = torch.from_numpy(rng.standard_normal((4, 16, 576))).bfloat16()
    e = errw()
    out, lse = mla.mla_nvfp4_fp8_decode(
        q.to(DEV), torch.from_numpy(cache).to(DEV).view(F8), torch.from_numpy(scales).to(DEV), SCALE,
        page_table=torch.from_numpy(table).to(DEV).expand(4, -1), seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
        return_lse=True, split=split, error_word=e)
    torch.cuda.synchronize()
    assert int(e.item()) == 0
    check_decode((f32(out), f32(lse)), q, cache, scales, np.repeat(table, 4, 0), lens, 64, what="one page table")
    own = run_decode(q, cache, scales, np.repeat(table, 4, 0), lens, 64, split=split)
    assert np.array_equal(own[0], f32(out)) and np.array_equal(own[1], f32(lse))
    with pytest.raises(mla.MLAError):  # rows that overlap in part
        mla.mla_nvfp4_fp8_decode(q.to(DEV), torch.from_numpy(cache).to(DEV).view(F8), torch.from_numpy(scales).to(DEV), SCALE,
                                 page_table=torch.zeros(20, dtype=torch.int32, device=DEV).as_strided((4, 5), (3, 1)),
                                 seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("heads", [16, 40])
@pytest.mark.parametrize("n", [300, 20000])
def test_decode_scores_above_the_range_give_nan(n, heads, split):
    # 2^120 times 448 times a block scale of 2^8: the head's results are NaN whether its sequence is cut or not, the
    # others' as ever; with the sign turned the key has no weight
    rng = np.random.default_rng(n)
    cache, scales, table = make_cache(rng, (n,), 64)
    at = table[0][np.arange(n) // 64].astype(np.int64) * 64 + np.arange(n) % 64
    cache[at, 3] = 0
    cache[int(table[0][1]) * 64 + 7, 3] = 0x7E  # key 71
    scales[table[0][1]] = 2.0 ** 8
    q = torch.from_numpy(rng.standard_normal((1, heads, 576)) * 2.0 ** -10).bfloat16()
    q[:, :, 3] = 0
    clean = run_decode(q, cache, scales, table, (n,), 64, split=split)
    for sign in (1, -1):
        big = q.clone()
        big[0, 2] = 0
        big[0, 2, 3] = sign * 2.0 ** 120
        out, lse, flags = run_decode(big, cache, scales, table, (n,), 64, split=split)
        assert flags == 0
        if sign > 0:
            assert np.all(np.isnan(out[0, 2])) and np.isnan(lse[0, 2])
        else:
            assert np.all(np.isfinite(out[0, 2])) and abs(lse[0, 2] - np.log(n - 1)) < 1e-5
        other = np.arange(heads) != 2
        assert np.array_equal(out[:, other], clean[0][:, other]) and np.array_equal(lse[:, other], clean[1][:, other])


@pytest.mark.parametrize("heads", [16, 40])
def test_decode_scores_all_below_the_range_give_nan(heads):
    # (a head without keys gives zeros and -inf; this one has keys)
    cache, scales, table = make_cache(np.random.default_rng(6), (1, 0), 64)
    cache[int(table[0][0]) * 64, 3] = 0x7E
    scales[:] = 2.0 ** 8
    q = torch.zeros(2, heads, 576, dtype=torch.bfloat16)
    q[0, 1, 3] = -(2.0 ** 120)
    for split in (True, False):
        out, lse, flags = run_decode(q, cache, scales, table, (1, 0), 64, split=split)
        assert flags == 0 and np.all(np.isnan(out[0, 1])) and np.isnan(lse[0, 1])
        assert np.all(np.isfinite(np.delete(out[0], 1, 0))) and np.allclose(np.delete(lse[0], 1), 0, atol=1e-6)
        assert np.all(out[1] == 0) and np.all(np.isneginf(lse[1]))


@pytest.mark.parametrize("heads", [16, 40])
def test_decode_scores_below_the_range_in_a_part_of_a_sequence(heads):
    # the first 6000 keys' scores are below fp32's range: they have no weight, though whole pieces of a cut sequence
    # consist of them; with all keys' below it the head is NaN
    rng = np.random.default_rng(7)
    n = 20000
    cache, scales, table = make_cache(rng, (n,), 64)
    at = table[0][np.arange(n) // 64].astype(np.int64) * 64 + np.arange(n) % 64
    cache[at, 3] = np.where(np.arange(n) < 6000, 0x7E, 0)
    scales[table[0][:-(-n // 64)]] = 2.0 ** 8
    q = torch.zeros(1, heads, 576, dtype=torch.bfloat16)
    q[0, 1, 3] = -(2.0 ** 120)
    v = fp8.decode_codes(cache[at, :512]) * 2.0 ** 8
    for split in (True, False):
        out, lse, flags = run_decode(q, cache, scales, table, (n,), 64, split=split)
        assert flags == 0 and np.all(np.isfinite(out)) and abs(lse[0, 1] - np.log(n - 6000)) < 1e-4
        # a mean of n - 6000 values: bf16's rounding and the weights' 2^-8 (of 2^4, exact) of their magnitude
        ref, mag = v[6000:].mean(0), np.abs(v[6000:]).mean(0)
        assert np.all(np.abs(out[0, 1] - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -8 * mag)
        cache2 = cache.copy()
        cache2[at, 3] = 0x7E
        out, lse, flags = run_decode(q, cache2, scales, table, (n,), 64, split=split)
        assert flags == 0 and np.all(np.isnan(out[0, 1])) and np.isnan(lse[0, 1])
        assert np.all(np.isfinite(out[0, 0])) and abs(lse[0, 0] - np.log(n)) < 1e-4


@pytest.mark.parametrize("heads", [16, 40])
@pytest.mark.parametrize("n", [1000, 30000])
@pytest.mark.parametrize("feature", [-448.0, -1.0, 0.0, 448.0])
def test_decode_references_follow_the_first_key_within_the_range(feature, n, heads):
    # the first 320 keys' scores are below fp32's range (2^64 * 448 * 2^60 / 14) and have no weight; the others' are all
    # the same, 0.29 times `feature`: -129 to 129
    rng = np.random.default_rng(8)
    cache, scales, table = make_cache(rng, (n,), 64)
    at = table[0][np.arange(n) // 64].astype(np.int64) * 64 + np.arange(n) % 64
    first = np.arange(n) < 320
    cache[at, 3] = np.where(first, 0x7E, 0)
    cache[at, 4] = np.where(first, 0, fp8.encode(np.array([feature]))[0])
    scales[:] = 2.0 ** -60
    scales[table[0][:5]] = 2.0 ** 60
    q = torch.zeros(1, heads, 576, dtype=torch.bfloat16)
    q[0, 1, 3], q[0, 1, 4] = -(2.0 ** 64), 2.0 ** 62
    v = fp8.decode_codes(cache[at[320:], :512]) * 2.0 ** -60
    ref, mag = v.mean(0), np.abs(v).mean(0)
    for split in (True, False):
        out, lse, flags = run_decode(q, cache, scales, table, (n,), 64, split=split)
        score = 4 * feature * SCALE
        assert flags == 0 and abs(lse[0, 1] - score - np.log(n - 320)) < 1e-4 + 2.0 ** -20 * abs(score)
        # equal weights: bf16's rounding, and the weights' 2^-8 and f16's of their magnitude
        assert np.all(np.abs(out[0, 1] - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * mag), split
