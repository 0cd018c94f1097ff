"""The operators of the 8-bit path: what is measured, and their plain forms.

Four operators serve a model whose latent cache and projection weights are
held in e4m3:

  append    new tokens' latent and rotary key, rotated by their position, into
            a paged e4m3 cache with one scale per block of 64 tokens, and the
            new queries' rotary part rotated by the same angles;
  decode    absorbed latent attention over that cache (576-d keys, values the
            first 512 of them, one latent head shared by all query heads);
  quantize  activations to e4m3 with one scale per 128 features of a row;
  gemm      e4m3 x e4m3 product, activations scaled per 128 features, weights
            per block of 128 x 128.

run() computes an operator in elementary torch operations in float32, or with
``own`` set by the library's calls; exact() by the definition in float64.
"""
import math

import torch

own = False

DEV = "cuda"
LATENT, ROPE, KEY, BLOCK = 512, 64, 576, 64
E4M3 = torch.float8_e4m3fn
SOFTMAX_SCALE = 1.0 / math.sqrt(192.0)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one user, one new token: what a call costs at least
        dict(name="append 1x1", op="append", batch=1, new=1, context=999, ragged=False, heads=16, interleaved=True, page=64),
        # a decode step of a full batch, all heads on this GPU, sequences at any place of a block
        dict(name="append 64x1 128h", op="append", batch=64, new=1, context=4096, ragged=True, heads=128, interleaved=True, page=64),
        # a prefill step of ragged prompts, some after a cached context; heads split over 8 GPUs, pages of 128, half-split rotation
        dict(name="append 8x4096 16h", op="append", batch=8, new=4096, context=700, ragged=True, heads=16, interleaved=False, page=128),
        # one short sequence, heads split over 8 GPUs: latency
        dict(name="decode 1x100 16h", op="decode", batch=1, heads=16, lo=100, hi=100, page=64),
        # a full batch of medium contexts, all heads on this GPU
        dict(name="decode 64x4096 128h", op="decode", batch=64, heads=128, lo=4096, hi=4096, page=64),
        # contexts of very different lengths, heads split over 8 GPUs: the cache's bytes bound it
        dict(name="decode 128 mixed 16h", op="decode", batch=128, heads=16, lo=1024, hi=32768, page=64),
        # one long context, work split over its keys
        dict(name="decode 1x65536 128h", op="decode", batch=1, heads=128, lo=65536, hi=65536, page=128),
        # activations of a decode step and of a prefill step
        dict(name="quantize 64x7168", op="quantize", m=64, k=7168),
        dict(name="quantize 8192x16384", op="quantize", m=8192, k=16384),
        # hidden state to latent and rotary key (512 + 64 columns) of one token
        dict(name="gemm 1x576x7168", op="gemm", m=1, n=576, k=7168),
        # output projection of a decode step: the weight's bytes bound it
        dict(name="gemm 64x7168x16384", op="gemm", m=64, n=7168, k=16384),
        # output projection of a prefill step: the tensor cores bound it
        dict(name="gemm 4096x7168x16384", op="gemm", m=4096, n=7168, k=16384),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "quantize", "gemm"])
    if op == "append":
        batch = _log(rng, 1, 128)
        return dict(op=op, batch=batch, new=_log(rng, 1, max(1, min(4096, 32768 // batch))), context=_log(rng, 1, 4096),
                    ragged=rng.random() < 0.7, heads=rng.choice([0, 1, 5, 16, 32]), interleaved=rng.random() < 0.5,
                    page=rng.choice([64, 128]))
    if op == "decode":
        batch, heads = _log(rng, 1, 128), rng.choice([1, 8, 16, 40, 64, 128])
        hi = _log(rng, 1, max(1, min(65536, 262144 // batch)))
        return dict(op=op, batch=batch, heads=heads, lo=rng.choice([hi, max(1, hi // 32), 1]), hi=hi,
                    page=rng.choice([64, 128, 256]))
    if op == "quantize":
        return dict(op=op, m=_log(rng, 1, 8192), k=8 * _log(rng, 1, 2048))
    m = _log(rng, 1, 4096)
    return dict(op=op, m=m, n=_log(rng, 64, 7168), k=16 * _log(rng, 4, 1024))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _spread(n, by):
    """n fractions spread over [0, 1), by the multiples of an irrational number; the first is 1."""
    return [1.0] + [(i * by) % 1.0 for i in range(1, n)]


def _append_sizes(case):
    """New and cached tokens of each sequence: ragged ones from a quarter and a half of the largest up."""
    B, new, ctx = case["batch"], case["new"], case["context"]
    if not case["ragged"]:
        return [new] * B, [ctx] * B
    lo_n, lo_c = max(1, new // 4), ctx // 2
    return ([int(lo_n + (new - lo_n) * u) for u in _spread(B, 0.6180339887)],
            [int(lo_c + (ctx - lo_c) * u) for u in _spread(B, 0.7548776662)])


def _decode_lens(case):
    """Sequence lengths, spread over the logarithm of lo..hi."""
    return [int(case["lo"] * (case["hi"] / case["lo"]) ** u) for u in _spread(case["batch"], 0.6180339887)]


def _latents(g, n):
    """Latent features: normal, one in a hundred 20 times as large."""
    x = _randn(g, n, LATENT)
    return torch.where(torch.rand(x.shape, generator=g, device=DEV) < 0.01, x * 20, x)


def _angles(n):
    """cos | sin of position p at 32 frequencies, from 64-bit angles, in float32."""
    f = 10000.0 ** (-torch.arange(0, ROPE, 2, device=DEV, dtype=torch.float64) / ROPE)
    a = torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _pages(g, lens, page):
    """A permuted page table wide enough for each sequence, and the pages it takes."""
    need = [-(-n // page) for n in lens]
    ids = torch.randperm(max(1, sum(need)), generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((len(lens), max(1, max(need))), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, ids.numel()


def _power_scale(amax):
    """The smallest power of two 2^e, -60 <= e <= 60, with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax)  # amax = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), torch.full_like(e, -60)).clamp(-60, 60)
    return torch.ldexp(torch.ones_like(amax), e)


def _filled_cache(g, blocks):
    """A cache whose blocks all hold tokens, as append would have left them."""
    codes = torch.empty((blocks * BLOCK, KEY), dtype=E4M3, device=DEV)
    scales = torch.empty(blocks, device=DEV)
    for at in range(0, blocks, 4096):
        n = min(4096, blocks - at)
        x = torch.cat([_latents(g, n * BLOCK), _randn(g, n * BLOCK, ROPE)], 1).bfloat16().float().view(n, BLOCK * KEY)
        s = _power_scale(x.abs().amax(1))
        scales[at:at + n] = s
        codes[at * BLOCK:(at + n) * BLOCK] = (x / s[:, None]).view(-1, KEY).to(E4M3)
    return codes, scales


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case)
    if op == "append":
        new, ctx = _append_sizes(case)
        lens = [n + c for n, c in zip(new, ctx)]
        s["table"], pages = _pages(g, lens, case["page"])
        s["cache"], s["scales"] = _filled_cache(g, pages * case["page"] // BLOCK)
        T = sum(new)
        s["cu"] = torch.tensor([0] + new, device=DEV).cumsum(0).int()
        s["context_lens"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        s["kv_c"], s["k_pe"] = _latents(g, T).bfloat16(), _randn(g, T, ROPE).bfloat16()
        s["q_pe"] = _randn(g, T, case["heads"], ROPE).bfloat16() if case["heads"] else None
        s["angles"] = _angles(max(lens))
    elif op == "decode":
        B, H = case["batch"], case["heads"]
        lens = _decode_lens(case)
        s["table"], pages = _pages(g, lens, case["page"])
        s["cache"], s["scales"] = _filled_cache(g, pages * case["page"] // BLOCK)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["q"] = _randn(g, B, H, KEY).bfloat16()
    elif op == "quantize":
        x = _randn(g, case["m"], case["k"])
        s["x"] = torch.where(torch.rand(x.shape, generator=g, device=DEV) < 0.01, x * 20, x).bfloat16()
    else:
        m, n, k = case["m"], case["n"], case["k"]
        kb, nb = -(-k // 128), -(-n // 128)
        a = _randn(g, m, kb * 128)
        a[:, k:] = 0
        a = a.view(m, kb, 128)
        s["a_scales"] = a.abs().amax(2) / 448
        s["a"] = (a / s["a_scales"][:, :, None]).view(m, -1)[:, :k].to(E4M3).contiguous()
        w = torch.zeros(nb * 128, kb * 128, device=DEV)
        w[:n, :k] = _randn(g, n, k) / math.sqrt(k)
        w = w.view(nb, 128, kb, 128)
        s["w_scales"] = w.abs().amax((1, 3)) / 448
        s["w"] = (w / s["w_scales"][:, None, :, None]).view(nb * 128, -1)[:n, :k].to(E4M3).contiguous()
    return s


# ------------------------------------------------------------- plain forms
def _rotate(x, cs, interleaved):
    """Rotates x [..., 64] (float) by the angles cs [..., 64] = cos | sin."""
    c, s = cs[..., :32], cs[..., 32:]
    if interleaved:
        x0, x1 = x[..., 0::2], x[..., 1::2]
        return torch.stack([x0 * c - x1 * s, x1 * c + x0 * s], -1).flatten(-2)
    x0, x1 = x[..., :32], x[..., 32:]
    return torch.cat([x0 * c - x1 * s, x1 * c + x0 * s], -1)


def _plain_append(s):
    T, dev = s["kv_c"].shape[0], s["kv_c"].device
    cu, page, cache, scales = s["cu"].long(), s["page"], s["cache"], s["scales"]
    t = torch.arange(T, device=dev)
    b = (t[:, None] >= cu[None, 1:]).sum(1)
    p = s["context_lens"].long()[b] + t - cu[b]
    cs = s["angles"][p]
    key = torch.cat([s["kv_c"].float(), _rotate(s["k_pe"].float(), cs, s["interleaved"])], 1)
    slot = s["table"].long()[b, p // page] * page + p % page
    blk, off, n = slot // BLOCK, slot % BLOCK, scales.numel()
    # per block: largest new value, first new place, whether a scale changes
    amax = torch.zeros(n, device=dev).scatter_reduce_(0, blk, key.abs().amax(1), "amax")
    first = torch.full((n,), BLOCK, device=dev).scatter_reduce_(0, blk, off, "amin")
    need = _power_scale(amax)
    grown = torch.where(first > 0, torch.maximum(scales, need), need)
    new = torch.where(first < BLOCK, grown, scales)
    # earlier tokens of a block are held in its new scale
    old = cache.view(n, BLOCK, KEY)
    earlier = torch.arange(BLOCK, device=dev)[None] < torch.where(first < BLOCK, first, 0)[:, None]
    ratio = torch.where(earlier, (scales / new)[:, None], 1.0)
    again = (old.float() * ratio[:, :, None]).to(E4M3)
    cache.copy_(again.view(-1, KEY))
    cache[slot] = (key / new[blk][:, None]).clamp(-448, 448).to(E4M3)
    scales.copy_(new)
    if s["q_pe"] is None:
        return cache, scales
    return cache, scales, _rotate(s["q_pe"].float(), cs[:, None], s["interleaved"]).bfloat16()


def _plain_decode(s):
    lens, page, q = s["lens"].long(), s["page"], s["q"].float()
    t = torch.arange(s["hi"], device=q.device)
    there = t[None] < lens[:, None]
    slot = torch.where(there, s["table"].long()[:, t // page] * page + t % page, 0)
    key = s["cache"][slot].float() * s["scales"][slot // BLOCK][..., None]
    score = torch.matmul(q, key.transpose(1, 2)) * SOFTMAX_SCALE
    score = torch.where(there[:, None], score, -math.inf)
    top = score.amax(2, keepdim=True)
    p = (score - top).exp()
    total = p.sum(2, keepdim=True)
    out = torch.matmul(p, key[..., :LATENT]) / total
    return out.bfloat16(), (top + total.log())[..., 0]


def _plain_quantize(s):
    x, k = s["x"].float(), s["x"].shape[1]
    kb = -(-k // 128)
    x = torch.cat([x, x.new_zeros(x.shape[0], kb * 128 - k)], 1).view(-1, kb, 128)
    scale = (x.abs().amax(2) / 448).clamp(min=2.0 ** -126)
    return (x / scale[:, :, None]).clamp(-448, 448).view(-1, kb * 128)[:, :k].to(E4M3), scale


def _plain_gemm(s):
    n, k = s["w"].shape
    a = s["a"].float() * s["a_scales"].repeat_interleave(128, 1)[:, :k]
    w = s["w"].float() * s["w_scales"].repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return torch.matmul(a, w.t()).bfloat16()


def run(s):
    op = s["op"]
    if own:
        import mla_attention_nvfp4_gb300 as mla
        if op == "append":
            got = mla.mla_nvfp4_fp8_cache_append(
                s["kv_c"], s["k_pe"], s["angles"], s["cu"], s["context_lens"], s["table"], s["cache"], s["scales"],
                page_size=s["page"], interleaved=s["interleaved"], q_pe=s["q_pe"], max_new_tokens=s["new"])
            return (s["cache"], s["scales"]) if got is None else (s["cache"], s["scales"], got)
        if op == "decode":
            return mla.mla_nvfp4_fp8_decode(s["q"], s["cache"], s["scales"], SOFTMAX_SCALE, page_table=s["table"],
                                            seq_lens=s["lens"], page_size=s["page"], return_lse=True)
        if op == "quantize":
            return mla.mla_nvfp4_fp8_quantize(s["x"])
        return mla.mla_nvfp4_fp8_gemm(s["a"], s["a_scales"], s["w"], s["w_scales"])
    return {"append": _plain_append, "decode": _plain_decode, "quantize": _plain_quantize, "gemm": _plain_gemm}[op](s)


# -------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "append":
        # a token's row read and its codes written, its angles, its queries read and written; the block scales
        n = sum(_append_sizes(case)[0])
        per = KEY * 2 + KEY + ROPE * 4 + case["heads"] * ROPE * 4
        return {"bytes": n * per + case["batch"] * 16, "flops": n * (case["heads"] + 1) * ROPE * 3}
    if op == "decode":
        keys = sum(_decode_lens(case))
        rows = case["batch"] * case["heads"]
        return {"bytes": keys * (KEY + 4 / BLOCK) + rows * (KEY * 2 + LATENT * 2 + 4), "flops": 2.0 * keys * case["heads"] * (KEY + LATENT)}
    if op == "quantize":
        m, k = case["m"], case["k"]
        return {"bytes": m * (3 * k + 4 * -(-k // 128)), "flops": 3.0 * m * k}
    m, n, k = case["m"], case["n"], case["k"]
    kb = -(-k // 128)
    return {"bytes": m * k + n * k + 4 * kb * (m + -(-n // 128)) + 2 * m * n, "flops": 2.0 * m * n * k}


# ------------------------------------------------------------ in 64 bits
def _e4m3(v):
    """v (float64) to the nearest e4m3 value, ties to the even one, at most 448."""
    a = v.abs()
    e = torch.frexp(a.clamp(min=2.0 ** -40))[1].double() - 1
    step = torch.exp2(e.clamp(min=-6) - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), v)


def _turn(x, angle_row, interleaved):
    """x [n, 64] times the unit numbers cos + i sin of each pair, in float64."""
    z = torch.complex(angle_row[..., :32].double(), angle_row[..., 32:].double())
    if interleaved:
        pair = torch.complex(x[..., 0::2].double(), x[..., 1::2].double()) * z
        return torch.view_as_real(pair).reshape(x.shape)
    pair = torch.complex(x[..., :32].double(), x[..., 32:].double()) * z
    return torch.cat([pair.real, pair.imag], -1)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "append":
        cache, scales = s["cache"].double(), s["scales"].double()
        cu, ctx, table = s["cu"].tolist(), s["context_lens"].tolist(), s["table"].tolist()
        queries = torch.empty(s["q_pe"].shape, dtype=torch.float64, device=DEV) if case["heads"] else None
        for b in range(case["batch"]):
            at, p, end = cu[b], ctx[b], ctx[b] + cu[b + 1] - cu[b]
            rows = s["angles"][p:end]
            key = torch.cat([s["kv_c"][at:cu[b + 1]].double(), _turn(s["k_pe"][at:cu[b + 1]], rows, case["interleaved"])], 1)
            if queries is not None:
                queries[at:cu[b + 1]] = _turn(s["q_pe"][at:cu[b + 1]], rows[:, None], case["interleaved"])
            largest = key.abs().amax(1).tolist()
            while p < end:
                upto = min(end, (p // BLOCK + 1) * BLOCK)
                i = p - ctx[b]
                most = max(largest[i:i + upto - p])
                power = max(-60, min(60, math.ceil(math.log2(most / 448)))) if most > 0 else -60
                slot = table[b][p // case["page"]] * case["page"] + p % case["page"]
                blk, off = slot // BLOCK, slot % BLOCK
                was = float(scales[blk])
                now = 2.0 ** power if off == 0 else max(was, 2.0 ** power)
                if off and now != was:
                    cache[slot - off:slot] = _e4m3(cache[slot - off:slot] * (was / now))
                scales[blk] = now
                cache[slot:slot + upto - p] = _e4m3(key[i:i + upto - p] / now)
                p = upto
        return (cache, scales) if queries is None else (cache, scales, queries)
    if op == "decode":
        out, lse = [], []
        table, page = s["table"].long(), case["page"]
        for b, n in enumerate(s["lens"].tolist()):
            t = torch.arange(n, device=DEV)
            slot = table[b, t // page] * page + t % page
            key = s["cache"][slot].double() * s["scales"][slot // BLOCK].double()[:, None]
            x = (s["q"][b].double() @ key.T) * SOFTMAX_SCALE
            ln = torch.logsumexp(x, 1)
            out.append(torch.exp(x - ln[:, None]) @ key[:, :LATENT])
            lse.append(ln)
        return torch.stack(out), torch.stack(lse)
    if op == "quantize":
        x, k = s["x"].double(), case["k"]
        codes, scales = torch.empty_like(x), torch.empty((case["m"], -(-k // 128)), dtype=torch.float64, device=DEV)
        for j in range(scales.shape[1]):
            part = x[:, 128 * j:128 * (j + 1)]
            scales[:, j] = (part.abs().amax(1) / 448).clamp(min=2.0 ** -126)
            codes[:, 128 * j:128 * (j + 1)] = _e4m3(part / scales[:, j:j + 1])
        return codes, scales
    total = torch.zeros((case["m"], case["n"]), dtype=torch.float64, device=DEV)
    if 2.0 * case["m"] * case["n"] * case["k"] > 4e12:
        return None
    for j in range(s["a_scales"].shape[1]):
        cut = slice(128 * j, 128 * (j + 1))
        by_row = s["w_scales"][:, j].double().repeat_interleave(128)[:case["n"]]
        total += (s["a"][:, cut].double() @ s["w"][:, cut].double().T) * s["a_scales"][:, j].double()[:, None] * by_row
    return total
