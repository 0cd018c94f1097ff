"""NVFP4 matrix-vector products on the GPU against the float64 oracle.

A product of a bf16 feature, a code and its scale is exact in float32 (8 + 2 +
4 significant bits) and K of them are summed there: off by at most 2 K 2^-24 of
the sum of magnitudes (a factor 2 for sums that round toward zero).  Features
are carried in f16 after a power of two has brought their row's largest to
2^14 or more: exact down to 2^-31 of it, half of f16's smallest step, 2^-25,
below, so off by at most 2^-39 of the largest, times sum |w|.  The output is
rounded to bf16."""
import numpy as np
import pytest
import torch

import mla_attention_nvfp4_gb300 as mla
from oracle import gemm, swizzle
from tests.helpers import bf16_half_ulp, f32

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
DEV = "cuda:0"


def weights(rng, G, N, K, lo=0x28, hi=0x48):
    """Random codes [G, N, K/2] and swizzled scales [G, bytes]; the padding holds any bytes, NaN among them."""
    codes = rng.integers(0, 256, (G, N, K // 2), dtype=np.uint8)
    bufs = []
    for _ in range(G):
        sf = rng.integers(lo, hi, (N, K // 16)).astype(np.uint8)
        buf = rng.integers(0, 256, swizzle.sf_buffer_bytes(N, K // 16), dtype=np.uint8)
        m, k = np.meshgrid(np.arange(N), np.arange(K // 16), indexing="ij")
        buf[swizzle.sf_offset(m, k, K // 16)] = sf
        bufs.append(buf)
    return codes, np.stack(bufs)


def rows(rng, M, G, K):
    x = rng.standard_normal((M, G, K)) * np.where(rng.random((M, G, K)) < 0.01, 30, 1)
    return torch.from_numpy(x).bfloat16()


def check(got, x, codes, sf, gs, what):
    G, N, K = codes.shape[0], codes.shape[1], 2 * codes.shape[2]
    x = f32(x)
    ref, mag, wsum = gemm.gemv(x, codes, sf, N, K, gs)
    tol = np.maximum(bf16_half_ulp(ref), bf16_half_ulp(got)) + 2.0 * K * 2.0 ** -24 * mag
    tol = tol + 2.0 ** -39 * np.abs(x).max(2, initial=0)[..., None] * wsum[None] + 1e-36
    worst = float(np.max(np.abs(got - ref) / tol, initial=0))
    print(f"[gemv] {what}: {worst:.3f} of the tolerance")
    assert np.all(np.isfinite(got)) and worst <= 1, f"{what}: {worst:.2f} times the tolerance"


def to(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def run(x, codes, sf, gs, **kw):
    out = mla.mla_nvfp4_gemv(x, to(codes), to(sf), torch.tensor([gs], device=DEV), **kw)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("M", [1, 2, 3, 7, 8, 9, 16, 17, 40])
@pytest.mark.parametrize("N,K", [(1, 32), (7, 96), (128, 128), (129, 256), (100, 160), (576, 1024), (33, 4128), (16, 16384),
                                 (1000, 2080)])
def test_gemv_matrix(M, N, K):
    rng = np.random.default_rng(M * 7 + N + K)
    gs = np.float32(1 / 3000)
    codes, sf = weights(rng, 1, N, K)
    x = rows(rng, M, 1, K)
    out = run(x[:, 0].to(DEV), codes[0], sf[0], gs)
    assert out.shape == (M, N)
    check(f32(out)[:, None], x, codes, sf, gs, f"{M}x{N}x{K}")


@pytest.mark.parametrize("M", [1, 4, 16, 19])
@pytest.mark.parametrize("G,N,K", [(1, 64, 64), (3, 128, 512), (16, 512, 128), (128, 128, 512), (5, 100, 96), (2, 1, 32)])
def test_gemv_groups(M, G, N, K):
    rng = np.random.default_rng(M + G + N + K)
    gs = np.float32(0.37)
    codes, sf = weights(rng, G, N, K)
    x = rows(rng, M, G, K)
    out = run(x.to(DEV), codes, sf, gs)
    assert out.shape == (M, G, N)
    check(f32(out), x, codes, sf, gs, f"{M}x{G}x{N}x{K}")


def test_gemv_wide_range_of_features_scales_and_codes():
    # features over 2^-30 .. 2^60 of their row, every e4m3 scale but NaN (subnormal and 448), every code
    rng = np.random.default_rng(3)
    M, N, K = 5, 70, 2048
    codes, sf = weights(rng, 1, N, K, 0, 0x7F)
    x = torch.from_numpy(rng.standard_normal((M, 1, K)) * 2.0 ** rng.integers(-30, 60, (M, 1, K))).bfloat16()
    x[3] = 0
    x[4] *= 2.0 ** -100
    out = run(x[:, 0].to(DEV), codes[0], sf[0], np.float32(2.0 ** -20))
    check(f32(out)[:, None], x, codes, sf, np.float32(2.0 ** -20), "wide range")
    assert not f32(out)[3].any()


def test_gemv_one_hot_rows_read_every_weight():
    # row m of x picks feature k = m of every column: the weight itself, rounded to bf16 (7 significant bits: exact)
    rng = np.random.default_rng(4)
    N, K = 37, 160
    codes, sf = weights(rng, 1, N, K)
    x = torch.eye(K).bfloat16()
    out = f32(run(x.to(DEV), codes[0], sf[0], np.float32(1)))
    assert np.array_equal(out.T, swizzle.dequantize_rows(codes[0], sf[0], N, K, 1.0))


def test_gemv_infinities_and_nan_stay_in_their_row_and_column():
    rng = np.random.default_rng(5)
    M, N, K = 4, 40, 512
    codes, sf = weights(rng, 1, N, K)
    codes[0][:, 8] = 0x22  # features 16, 17: code 1.0 in every column ...
    codes[0][5, 8] = 0x20  # ... but column 5, where feature 16 meets a zero
    x = rows(rng, M, 1, K)
    clean = f32(run(x[:, 0].to(DEV), codes[0], sf[0], np.float32(1)))
    x[1, 0, 16] = float("inf")
    x[2, 0, 17] = float("nan")
    got = f32(run(x[:, 0].to(DEV), codes[0], sf[0], np.float32(1)))
    assert np.array_equal(got[[0, 3]], clean[[0, 3]])
    assert np.all(np.isposinf(np.delete(got[1], 5))) and np.isnan(got[1, 5]) and np.all(np.isnan(got[2]))
    # a NaN scale: its column alone
    sf[0][swizzle.sf_offset(7, 3, K // 16)] = 0x7F
    x = rows(rng, M, 1, K)
    got = f32(run(x[:, 0].to(DEV), codes[0], sf[0], np.float32(1)))
    assert np.all(np.isnan(got[:, 7])) and np.all(np.isfinite(np.delete(got, 7, 1)))


def test_gemv_strides_and_outputs():
    rng = np.random.default_rng(6)
    M, G, N, K = 3, 4, 130, 128
    gs = np.float32(1)
    codes, sf = weights(rng, G, N, K)
    x = rows(rng, M, G, K)
    plain = f32(run(x.to(DEV), codes, sf, gs))
    # inside wider rows, group by group, an output at an odd address inside a wider one
    wide = torch.full((M, G, 192), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, :, 64:] = x.to(DEV)
    by_group = x.to(DEV).transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.full((M, G, N + 5), 7.0, dtype=torch.bfloat16, device=DEV)
    r = run(wide[:, :, 64:], codes, sf, gs, out=out[:, :, 3:N + 3])
    assert r.data_ptr() == out[:, :, 3:].data_ptr() and np.array_equal(f32(out[:, :, 3:N + 3]), plain)
    assert bool((out[:, :, :3] == 7).all()) and bool((out[:, :, N + 3:] == 7).all())
    flipped = torch.empty((G, M, N), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    run(by_group, codes, sf, gs, out=flipped)
    assert np.array_equal(f32(flipped), plain)
    # one row for all: an expanded tensor is read, an expanded output refused
    same = run(x[:1, 0].to(DEV).expand(1, K), codes[0], sf[0], gs)
    assert np.array_equal(f32(same), plain[:1, 0])
    with pytest.raises(mla.MLAError):
        run(x.to(DEV), codes, sf, gs, out=torch.empty(N, dtype=torch.bfloat16, device=DEV).expand(M, G, N))
    with pytest.raises(ValueError):
        run(x.to(DEV), codes, sf[:, :-16], gs)
    with pytest.raises(ValueError):
        run(x.to(DEV), codes[:2], sf, gs)


def test_gemv_has_one_global_scale():
    # (one a group is not read as the first for all)
    rng = np.random.default_rng(16)
    codes, sf = weights(rng, 2, 16, 32)
    x = rows(rng, 1, 2, 32).to(DEV)
    for gs in (torch.ones(2, device=DEV), torch.ones(0, device=DEV)):
        with pytest.raises(ValueError, match="gs_w"):
            mla.mla_nvfp4_gemv(x, to(codes), to(sf), gs)


def test_gemv_repeats_itself_in_a_graph_and_on_two_streams():
    rng = np.random.default_rng(7)
    N, K = 7168, 2048
    codes, sf = weights(rng, 1, N, K)
    w, s, gs = to(codes[0]), to(sf[0]), torch.tensor([0.01], device=DEV)
    xs = [rows(rng, m, 1, K)[:, 0].to(DEV) for m in (1, 16)]
    plain = [mla.mla_nvfp4_gemv(x, w, s, gs) for x in xs]
    again = [mla.mla_nvfp4_gemv(x, w, s, gs) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    outs = [torch.empty_like(p) for p in plain]
    for _ in range(20):
        for x, o, st in zip(xs, outs, streams):
            with torch.cuda.stream(st):
                mla.mla_nvfp4_gemv(x, w, s, gs, out=o)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = [mla.mla_nvfp4_gemv(x, w, s, gs) for x in xs]
    xs[0].neg_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for p, a, o, h, sign in zip(plain, again, outs, held, (-1, 1)):
        assert torch.equal(p, a) and torch.equal(p, o) and torch.equal(sign * p, h)


def test_gemv_agrees_with_the_gemm_on_activations_that_nvfp4_holds():
    # x of codes times scales: the same product as mla_nvfp4_gemm's, up to both sums' rounding
    rng = np.random.default_rng(8)
    M, N, K = 16, 256, 1024
    codes, sf = weights(rng, 1, N, K)
    xc, xsf = weights(rng, 1, M, K)
    x = torch.from_numpy(swizzle.dequantize_rows(xc[0], xsf[0], M, K, 1.0).astype(np.float32)).bfloat16()
    one = torch.ones(1, device=DEV)
    a = f32(mla.mla_nvfp4_gemv(x.to(DEV), to(codes[0]), to(sf[0]), one))
    b = f32(mla.mla_nvfp4_gemm(to(xc[0]), to(xsf[0]), to(codes[0]), to(sf[0]), one, one))
    mag = gemm.gemv(f32(x)[:, None], codes, sf, N, K, 1.0)[1][:, 0]
    assert np.all(np.abs(a - b) <= bf16_half_ulp(a) + bf16_half_ulp(b) + 4.0 * K * 2.0 ** -24 * mag)


@pytest.mark.parametrize("M", [1, 3, 6, 16])
def test_gemv_of_the_largest_matrix_sampled(M):
    # 7168 x 16384: the forms that split K over clusters; 60 columns of it against the oracle
    rng = np.random.default_rng(M)
    N, K = 7168, 16384
    gs = np.float32(0.01)
    codes, sf = weights(rng, 1, N, K)
    x = rows(rng, M, 1, K)
    got = f32(run(x[:, 0].to(DEV), codes[0], sf[0], gs))
    cols = np.sort(rng.choice(N, 60, replace=False))
    w = swizzle.unswizzle_scales(sf[0], N, K // 16)[cols]
    check(got[:, cols][:, None], x, codes[:, cols], swizzle.swizzle_scales(w)[None], gs, f"{M} rows of {N}x{K}")


def test_gemv_calls_in_a_row_read_what_the_work_ahead_wrote():
    # every call's x, weights and scale are written by the kernels just before it
    rng = np.random.default_rng(9)
    N, K = 600, 4096
    sets = [(rows(rng, 2, 1, K)[:, 0].to(DEV), *(to(a[0]) for a in weights(rng, 1, N, K)), torch.tensor([0.1 * (i + 1)], device=DEV))
            for i in range(4)]
    ref = []
    for s in sets:
        ref.append(mla.mla_nvfp4_gemv(*s))
        torch.cuda.synchronize()
    held = [torch.empty_like(t) for t in sets[0]]
    got = []
    for i in range(400):
        for h, t in zip(held, sets[i % 4]):
            h.copy_(t)
        got.append(mla.mla_nvfp4_gemv(*held))
    # and a chain of them, each call's result the next one's x
    square = [to(a[0]) for a in weights(rng, 1, 512, 512)]
    one = torch.tensor([2.0 ** -9], device=DEV)
    chain, steps = rows(rng, 4, 1, 512)[:, 0].to(DEV), []
    for _ in range(50):
        steps.append(chain)
        chain = mla.mla_nvfp4_gemv(chain, *square, one)
    torch.cuda.synchronize()
    assert all(torch.equal(g, ref[i % 4]) for i, g in enumerate(got))
    for x, y in zip(steps, steps[1:] + [chain]):
        again = mla.mla_nvfp4_gemv(x, *square, one)
        torch.cuda.synchronize()
        assert torch.equal(again.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("M,few,more,K", [(16, 1024, 1536, 7168), (16, 576, 1536, 7168), (8, 256, 1024, 16384)])
def test_gemv_of_fewer_weights_takes_no_longer(M, few, more, K):
    """The split of K goes by the CTAs that the device holds of the form at hand.  By a count for smaller ones a matrix of
    1024 rows was cut for twice the CTAs that fit, and took twice the time of one of 1536.  (1.4: noise; least of nine.)"""
    rng = np.random.default_rng(60)

    def least(N):
        x = torch.randn(M, K, device=DEV).bfloat16()
        w = [to(a[0]) for a in weights(rng, 1, N, K)]
        gs = torch.ones(1, device=DEV)
        mla.mla_nvfp4_gemv(x, *w, gs)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(20):
                mla.mla_nvfp4_gemv(x, *w, gs)
        times = []
        for _ in range(9):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            g.replay()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    a, b = least(few), least(more)
    assert a <= 1.4 * b, f"{few} rows {a * 50:.1f} us, {more} rows {b * 50:.1f} us"
