"""The 8-bit entry points refuse bad arguments on the host, before any launch
(status codes: 1 invalid, 3 alignment, 5 workspace), and empty work is a
no-op.  The pointers are never followed."""
import ctypes
import os
import re

import pytest
import torch

import mla_attention_nvfp4_gb300 as mla

P, ODD = ctypes.c_void_p(256), ctypes.c_void_p(264)


def _append(**kw):
    a = dict(kv_c=P, kv_st=512, k_pe=P, pe_st=64, T=4, cs=P, maxpos=100, il=1, cu=P, ctx=P, seqs=2, new=4, pt=P,
             pt_st=2, pages=2, page=64, cache=P, slots=128, scales=P, q=P, qt=128, qh=64, o=P, ot=128, oh=64, H=2,
             err=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return mla.load_library().mla_nvfp4_fp8_cache_append(*a.values())


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(seqs=-1), dict(new=-1), dict(maxpos=-1), dict(il=2), dict(H=-1), dict(page=0), dict(page=32),
    dict(page=96), dict(slots=100), dict(slots=-64), dict(kv_c=None), dict(k_pe=None), dict(cs=None), dict(cu=None),
    dict(ctx=None), dict(pt=None), dict(cache=None), dict(scales=None), dict(kv_st=504), dict(pe_st=56),
    dict(pages=0), dict(pt_st=1), dict(q=None), dict(o=None), dict(H=0), dict(q=None, o=None), dict(qt=120),
    dict(qh=56), dict(ot=64), dict(oh=32), dict(ot=256), dict(T=1 << 31),
    dict(seqs=2**31 - 1, new=2**30, T=2**30, qt=64, ot=64, H=1)])
def test_append_refuses(kw):
    assert _append(**kw) == 1 or (kw.get("seqs", 0) > 100 and _append(**kw) in (1, 4))


@pytest.mark.parametrize("kw", [
    dict(kv_c=ODD), dict(k_pe=ODD), dict(cs=ODD), dict(cache=ODD), dict(q=ODD), dict(o=ODD), dict(kv_st=516),
    dict(pe_st=68), dict(o=ctypes.c_void_p(512), qt=132), dict(o=ctypes.c_void_p(512), ot=132),
    dict(o=ctypes.c_void_p(512), qh=68, qt=136), dict(o=ctypes.c_void_p(512), oh=68, ot=136)])
def test_append_alignment(kw):
    assert _append(**kw) == 3


@pytest.mark.parametrize("pages", [2**31, 2**62])
def test_page_tables_too_wide_are_refused(pages):
    # (a table's tokens, pages times page size, stay in 64 bits)
    assert _append(pages=pages, pt_st=pages) == 1
    assert _decode(pages=pages, pt_st=pages) == 1


@pytest.mark.parametrize("kw", [dict(T=0), dict(seqs=0), dict(new=0)])
def test_append_nothing_to_do(kw):
    assert _append(**kw) == 0


def _decode(**kw):
    a = dict(q=P, B=2, H=16, cache=P, slots=128, scales=P, pt=P, pt_st=2, pages=2, page=64, lens=P, scale=0.1, out=P,
             lse=None, ws=None, ws_bytes=0, err=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return mla.load_library().mla_nvfp4_fp8_decode(*a.values())


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(H=0), dict(slots=-64), dict(slots=0), dict(slots=100), dict(slots=1 << 31), dict(page=0),
    dict(page=32), dict(page=100), dict(pages=0), dict(pt_st=1), dict(q=None), dict(cache=None), dict(scales=None),
    dict(pt=None), dict(lens=None), dict(out=None), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf"))])
def test_decode_refuses(kw):
    assert _decode(**kw) == 1


def test_decode_alignment_workspace_and_empty():
    for name in ("q", "cache", "out"):
        assert _decode(**{name: ODD}) == 3
    assert _decode(B=0) == 0
    assert mla.mla_nvfp4_fp8_decode_workspace_size(0, 16) == 0
    assert mla.mla_nvfp4_fp8_decode_workspace_size(2, 0) == 0
    assert mla.mla_nvfp4_fp8_decode_workspace_size(2, 16) > 0


def _quantize(**kw):
    a = dict(x=P, st=256, M=4, K=256, codes=P, scales=P, stream=None)
    a.update(kw)
    return mla.load_library().mla_nvfp4_fp8_quantize(*a.values())


def test_quantize_refuses():
    for kw in (dict(M=-1), dict(K=-8), dict(K=12), dict(x=None), dict(codes=None), dict(scales=None), dict(st=248),
               dict(M=1 << 31)):
        assert _quantize(**kw) == 1, kw
    for kw in (dict(x=ODD), dict(st=260), dict(codes=ctypes.c_void_p(260))):
        assert _quantize(**kw) == 3, kw
    assert _quantize(M=0) == 0 and _quantize(K=0) == 0


def _gemm(**kw):
    a = dict(a=P, lda=256, sa=P, M=4, w=P, ldw=256, sw=P, N=8, K=256, out=P, ldc=8, err=None, stream=None)
    a.update(kw)
    return mla.load_library().mla_nvfp4_fp8_gemm(*a.values())


def test_gemm_refuses():
    for kw in (dict(M=-1), dict(N=-1), dict(K=-16), dict(K=24), dict(K=0), dict(a=None), dict(sa=None), dict(w=None),
               dict(sw=None), dict(out=None), dict(lda=240), dict(ldw=240), dict(ldc=7), dict(M=1 << 31),
               dict(N=1 << 31, ldc=1 << 31)):
        assert _gemm(**kw) == 1, kw
    for kw in (dict(a=ODD), dict(w=ODD), dict(lda=264), dict(ldw=264), dict(out=ctypes.c_void_p(257))):
        assert _gemm(**kw) == 3, kw
    assert _gemm(M=0) == 0 and _gemm(N=0) == 0


def test_python_calls_want_cuda_tensors():
    f8 = torch.zeros(64, 576, dtype=torch.float8_e4m3fn)
    sc, i32 = torch.ones(1), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        mla.mla_nvfp4_fp8_cache_append(torch.zeros(1, 512).bfloat16(), torch.zeros(1, 64).bfloat16(),
                                       torch.zeros(4, 64), torch.zeros(2, dtype=torch.int32), i32, i32[None], f8, sc)
    with pytest.raises(ValueError, match="CUDA"):
        mla.mla_nvfp4_fp8_decode(torch.zeros(1, 16, 576).bfloat16(), f8, sc, 0.1, page_table=i32[None], seq_lens=i32)
    with pytest.raises(ValueError, match="CUDA"):
        mla.mla_nvfp4_fp8_quantize(torch.zeros(2, 128).bfloat16())
    with pytest.raises(ValueError, match="CUDA"):
        mla.mla_nvfp4_fp8_gemm(f8, sc[None], f8, sc[None])


def test_python_calls_want_tensors_and_arguments_of_the_right_kind():
    with pytest.raises(TypeError, match="tensor"):
        mla.mla_nvfp4_fp8_quantize([1.0])
    with pytest.raises(TypeError):
        mla.mla_nvfp4_fp8_gemm(None, None, None, None)


def test_no_thread_leaves_a_wait_of_the_append_by_itself():
    # (a lane that returned alone would be missing at the warp's shuffles and the CTA's barriers)
    path = os.path.join(os.path.dirname(mla.__file__), "csrc", "fp8_cache.cu")
    with open(path) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert "mbar_wait_cta(" in code and "drain_copies(" in code
    assert not re.search(r"\bmbar_wait\(", code)


@pytest.mark.parametrize("name,issuers,rings", [("fp8_decode.cu", 2, 2), ("fp8_gemm.cu", 2, 2)])
def test_no_cta_leaves_copies_or_products_in_flight(name, issuers, rings):
    path = os.path.join(os.path.dirname(mla.__file__), "csrc", name)
    with open(path) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert len(re.findall(r"^ +retire_products\(", code, re.M)) == issuers
    # rings are waited for once all roles have ended, when it is known whether one gave up
    ends = [part for part in re.split(r"tmem_dealloc\(", code)[1:]]
    assert sum(len(re.findall(r"drain_copies\(", part.split("__global__")[0])) for part in ends) == rings
    assert len(re.findall(r"drain_copies\(", code)) == rings
