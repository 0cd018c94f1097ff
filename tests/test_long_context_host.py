"""The entry points for long contexts and few rows (shared prefix, key
weights, eviction, append at a position, matrix-vector products) refuse bad
arguments on the host, before any launch (status codes: 1 invalid, 3
alignment, 5 workspace), and empty work is a no-op.  The pointers are never
followed."""
import ctypes

import pytest
import torch

import mla_attention_nvfp4_gb300 as mla

P, ODD = ctypes.c_void_p(256), ctypes.c_void_p(264)
FAR, FAR2 = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)


def _shared(**kw):
    a = dict(q=P, B=2, H=16, cache=P, slots=128, scales=P, pt=P, pt_st=2, pages=2, page=64, lens=P, shared=64, scale=0.1,
             out=P, lse=None, ws=None, ws_bytes=0, err=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return mla.load_library().mla_nvfp4_fp8_decode_shared(*a.values())


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(H=0), dict(slots=-64), dict(slots=0), dict(slots=100), dict(slots=1 << 31), dict(page=0),
    dict(page=32), dict(page=100), dict(pages=0), dict(pt_st=1), dict(q=None), dict(cache=None), dict(scales=None),
    dict(pt=None), dict(lens=None), dict(out=None), dict(scale=0.0), dict(scale=float("nan")), dict(shared=-64),
    dict(shared=63), dict(shared=1), dict(shared=192), dict(pages=2**31, pt_st=2**31), dict(B=2**27, H=16)])
def test_shared_refuses(kw):
    assert _shared(**kw) == 1


def test_shared_alignment_workspace_and_empty():
    for name in ("q", "cache", "out"):
        assert _shared(**{name: ODD}) == 3
    assert _shared(B=0) == 0
    size = mla.mla_nvfp4_fp8_decode_shared_workspace_size
    assert size(0, 16) == 0 and size(2, 0) == 0 and size(2, 16) > 0


def _weights(**kw):
    a = dict(q=P, B=2, H=16, cache=P, slots=128, scales=P, pt=P, pt_st=2, pages=2, page=64, lens=P, scale=0.1, lse=P,
             w=FAR, w_st=128, out=FAR2, out_st=128, row=128, err=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return mla.load_library().mla_nvfp4_fp8_key_weights(*a.values())


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(H=0), dict(slots=-64), dict(slots=0), dict(slots=100), dict(page=32), dict(pages=0), dict(pt_st=1),
    dict(q=None), dict(cache=None), dict(scales=None), dict(pt=None), dict(lens=None), dict(lse=None), dict(out=None),
    dict(scale=0.0), dict(scale=float("inf")), dict(row=-1), dict(w_st=127), dict(out_st=127),
    # weights and out overlap, but are not the same
    dict(out=FAR, out_st=129), dict(out=ctypes.c_void_p((1 << 20) + 4)), dict(out=ctypes.c_void_p((1 << 20) - 512)),
    dict(out=ctypes.c_void_p((1 << 20) + 4 * 255))])
def test_key_weights_refuses(kw):
    assert _weights(**kw) == 1


def test_key_weights_alignment_and_empty():
    assert _weights(q=ODD) == 3 and _weights(cache=ODD) == 3
    assert _weights(B=0) == 0 and _weights(row=0) == 0


def _evict(**kw):
    a = dict(cache=P, slots=256, scales=P, w=FAR, w_st=128, row=128, B=2, pt=P, pt_st=2, pages=2, npt=P, npt_st=1, npages=1,
             page=64, lens=P, keep=40, recent=8, kept=ctypes.c_void_p(512), nlens=ctypes.c_void_p(1024), nw=FAR2, nw_st=40,
             nrow=40, err=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return mla.load_library().mla_nvfp4_fp8_cache_evict(*a.values())


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(slots=-64), dict(slots=0), dict(slots=100), dict(page=32), dict(page=100), dict(pages=0),
    dict(pt_st=1), dict(pt_st=0), dict(npages=0), dict(npt_st=0), dict(npages=2**31, npt_st=2**31), dict(row=-1),
    dict(w_st=127), dict(keep=0), dict(keep=-1), dict(recent=-1), dict(recent=41), dict(keep=2**31 - 1), dict(cache=None),
    dict(scales=None), dict(w=None), dict(pt=None), dict(npt=None), dict(lens=None), dict(kept=None), dict(nlens=None),
    dict(nrow=39), dict(nw_st=39), dict(nw=FAR), dict(nw=ctypes.c_void_p((1 << 20) + 4 * 255)),
    dict(nlens=P), dict(nlens=ctypes.c_void_p(512))])
def test_evict_refuses(kw):
    assert _evict(**kw) == 1


def test_evict_alignment_and_empty():
    assert _evict(cache=ODD) == 3
    assert _evict(B=0) == 0


def _gemv(**kw):
    a = dict(x=P, xm=256, xg=64, M=4, w=P, sf=P, G=4, N=8, K=64, gs=P, out=P, om=32, og=8, err=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return mla.load_library().mla_nvfp4_gemv(*a.values())


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(G=-1), dict(N=-1), dict(K=-32), dict(K=16), dict(K=48), dict(K=0), dict(x=None), dict(w=None),
    dict(sf=None), dict(gs=None), dict(out=None), dict(M=1 << 31), dict(N=1 << 31), dict(K=1 << 31), dict(K=(1 << 30) + 32), dict(N=1 << 30),
    # rows that overlap
    dict(xm=64), dict(xm=248), dict(xg=56), dict(xm=0), dict(xg=0), dict(om=8), dict(om=31), dict(og=7), dict(om=8, og=24),
    dict(xm=64, xg=248)])
def test_gemv_refuses(kw):
    assert _gemv(**kw) == 1


def test_gemv_alignment_and_empty():
    for kw in (dict(x=ODD), dict(w=ODD), dict(sf=ODD), dict(xm=260), dict(xg=68, xm=512), dict(out=ctypes.c_void_p(257)),
               dict(gs=ctypes.c_void_p(258))):
        assert _gemv(**kw) == 3, kw
    assert _gemv(M=0) == 0 and _gemv(G=0) == 0 and _gemv(N=0) == 0


def test_gemv_rows_up_to_the_grid():
    assert _gemv(M=16 * 65535 + 1, xm=1 << 13, om=1 << 13) == 1


def test_append_at_has_the_checks_of_append():
    a = dict(kv_c=P, kv_st=512, k_pe=P, pe_st=64, T=4, cs=P, maxpos=100, il=1, cu=P, ctx=P, pos=P, seqs=2, new=4, pt=P,
             pt_st=2, pages=2, page=64, cache=P, slots=128, scales=P, q=None, qt=0, qh=0, o=None, ot=0, oh=0, H=0,
             err=None, stream=None)
    call = mla.load_library().mla_nvfp4_fp8_cache_append_at
    for kw, st in ((dict(T=-1), 1), (dict(page=96), 1), (dict(ctx=None), 1), (dict(kv_c=ODD), 3), (dict(T=0), 0),
                   (dict(pos=None, T=0), 0), (dict(il=2), 1)):
        assert call(*{**a, **kw}.values()) == st, kw


def test_python_calls_want_cuda_tensors():
    f8 = torch.zeros(64, 576, dtype=torch.float8_e4m3fn)
    sc, i32 = torch.ones(1), torch.zeros(1, dtype=torch.int32)
    q, u8 = torch.zeros(1, 16, 576).bfloat16(), torch.zeros(1, 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        mla.mla_nvfp4_fp8_decode_shared(q, f8, sc, 0.1, page_table=i32[None], seq_lens=i32, shared_len=64)
    with pytest.raises(ValueError, match="CUDA"):
        mla.mla_nvfp4_fp8_key_weights(q, f8, sc, 0.1, torch.zeros(1, 16), page_table=i32[None], seq_lens=i32)
    with pytest.raises(ValueError, match="CUDA"):
        mla.mla_nvfp4_fp8_cache_evict(f8, sc, sc[None], page_table=i32[None], seq_lens=i32, new_page_table=i32[None], keep=1)
    with pytest.raises(ValueError, match="CUDA"):
        mla.mla_nvfp4_gemv(torch.zeros(1, 32).bfloat16(), u8, u8, sc)


def test_launch_accounting_names_them():
    for name in ("fp8_decode_shared", "fp8_key_weights", "fp8_cache_evict", "gemv"):
        assert mla.LAUNCHES_PER_CALL[name] >= 1 and mla.kernel_kind(name) in ("hbm", "tensor", "alu")


@pytest.mark.parametrize("column", [128, 200, 384, -128, -256, -384])
def test_rows_of_one_wider_matrix_are_apart(column):
    # 128 columns of weights, others of out (new_weights) in rows of 512: no refusal (3: the cache's alignment, looked at next)
    at = ctypes.c_void_p((1 << 20) + 4 * column)
    assert _weights(w_st=512, out=at, out_st=512, cache=ODD) == 3
    assert _evict(w_st=512, nw=at, nw_st=512, nrow=128, cache=ODD) == 3


@pytest.mark.parametrize("column", [127, 385, -127, -385, 512, -512, 0.5, 128.5])
def test_rows_of_one_wider_matrix_that_overlap(column):
    at = ctypes.c_void_p((1 << 20) + int(4 * column))
    assert _weights(w_st=512, out=at, out_st=512, cache=ODD) == 1
    assert _evict(w_st=512, nw=at, nw_st=512, nrow=128, cache=ODD) == 1


@pytest.mark.parametrize("kw", [
    # seq_lens 4096.., weights 2^20.., page_table 8192.., new_page_table 8256.., kept 16384.., new_lens 32768.., new_weights 2^21..
    dict(nlens=4100), dict(nlens=4092), dict(nlens=8192 + 12), dict(nlens=8256 + 4), dict(nlens=(1 << 20) + 4 * 255),
    dict(nlens=16384 + 4 * 79), dict(nlens=(1 << 21) + 4 * 79), dict(kept=4092), dict(kept=4096 - 4 * 79), dict(kept=8192 + 8),
    dict(kept=8256 - 4 * 79), dict(kept=(1 << 20) - 4), dict(kept=(1 << 21) - 4), dict(nw=4100), dict(nw=8192 + 12),
    dict(nw=8256 - 4 * 79), dict(nw=16384 - 4 * 79), dict(nw=32768 + 4)])
def test_evict_refuses_results_in_its_arguments(kw):
    base = dict(lens=4096, pt=8192, npt=8256, kept=16384, nlens=32768, nw=1 << 21, cache=264)
    args = lambda d: {k: ctypes.c_void_p(v) for k, v in d.items()}
    assert _evict(**args(base)) == 3  # (the cache's alignment)
    assert _evict(**args({**base, **kw})) == 1


def test_evict_takes_a_record_for_each_sequence():
    # a sequence's table, new table, weights and their result in one record of 512 words; what is contiguous lies elsewhere, or
    # (seq_lens) in a gap
    at = lambda words: ctypes.c_void_p((1 << 20) + 4 * words)
    rec = dict(pt=at(0), pt_st=512, npt=at(2), npt_st=512, w=at(8), w_st=512, nw=at(200), nw_st=512, lens=at(504), cache=ODD,
               kept=ctypes.c_void_p(1 << 24), nlens=ctypes.c_void_p(1 << 25))
    assert _evict(**rec) == 3  # (the cache's alignment)
    assert _evict(**rec | dict(nlens=at(506))) == 3  # in the same gap
    assert _evict(**rec | dict(nlens=at(508), B=4)) == 3
    assert _evict(**rec | dict(kept=at(380))) == 3  # words 380 .. 460
    for kw in (dict(nlens=at(505)), dict(nlens=at(511)), dict(nlens=at(135)), dict(nlens=at(508), B=5), dict(kept=at(430)),
               dict(nw=at(135)), dict(nw=at(475)), dict(nw=at(1), nrow=40), dict(npt=at(210))):
        assert _evict(**rec | kw) == 1, kw
