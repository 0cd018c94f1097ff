"""Operators of a decode step over long contexts: what is measured, and their
plain forms.

Four operators serve a model whose latent cache is held in e4m3 (codes
[slots, 576] and a power-of-two scale per block of 64 tokens) and whose
projections are held in NVFP4:

  shared   absorbed latent attention of a batch whose sequences begin with the
           same tokens: that prefix is read once for all of them;
  weigh    the attention weight that a decode step's queries give to each cached
           token, summed over the heads and added to what it had;
  evict    of every sequence the tokens of greatest accumulated weight (and the
           most recent ones) moved, in order, to new pages;
  gemv     bf16 rows times an NVFP4 weight matrix (or one matrix a head), its
           codes and scales laid out as the NVFP4 GEMM reads them.

run() computes an operator in elementary torch operations in float32, or with
``own`` set by the library's calls; exact() by the definition in float64.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
LATENT, KEY, BLOCK = 512, 576, 64
E4M3 = torch.float8_e4m3fn
SOFTMAX_SCALE = 1.0 / math.sqrt(192.0)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a few questions about one short text, heads split over 8 GPUs: latency
        dict(name="shared 4x(2048+64) 16h", op="shared", batch=4, heads=16, shared=2048, lo=64, hi=64, page=64),
        # a full batch of dialogues behind one system prompt, heads split over 8 GPUs
        dict(name="shared 64x(16384+mixed) 16h", op="shared", batch=64, heads=16, shared=16384, lo=1, hi=2048, page=64),
        # questions about one long document, all heads on this GPU: the tensor cores bound it
        dict(name="shared 32x(32768+1000) 128h", op="shared", batch=32, heads=128, shared=32768, lo=1000, hi=1000, page=128),
        # one sequence: latency
        dict(name="weigh 1x1000 16h", op="weigh", batch=1, heads=16, lo=1000, hi=1000, page=64),
        # a full batch, all heads on this GPU
        dict(name="weigh 64x4096 128h", op="weigh", batch=64, heads=128, lo=4096, hi=4096, page=64),
        # contexts of very different lengths, heads split over 8 GPUs
        dict(name="weigh 32 mixed 16h", op="weigh", batch=32, heads=16, lo=1024, hi=32768, page=128),
        # one sequence at its limit
        dict(name="evict 1x1000", op="evict", batch=1, lo=1000, hi=1000, keep=256, recent=32, page=64),
        # a batch of long contexts cut to a budget; some are below it
        dict(name="evict 32 mixed", op="evict", batch=32, lo=1024, hi=32768, keep=4000, recent=500, page=64),
        # hidden state to latent and rotary key (512 + 64 columns) of one token
        dict(name="gemv 1x576x7168", op="gemv", m=1, n=576, k=7168, heads=0),
        # output projection of one token: the weight's bytes bound it
        dict(name="gemv 1x7168x16384", op="gemv", m=1, n=7168, k=16384, heads=0),
        # output projection of a small batch
        dict(name="gemv 16x7168x16384", op="gemv", m=16, n=7168, k=16384, heads=0),
        # every head's queries into the latent's space, a few tokens
        dict(name="gemv 4x512x128 128h", op="gemv", m=4, n=512, k=128, heads=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "weigh", "evict", "gemv"])
    page = rng.choice([64, 128, 256])
    if op == "shared":
        heads = rng.choice([1, 8, 16, 40, 128])
        batch = _log(rng, 1, 4096 // heads if heads > 32 else 128)
        hi = _log(rng, 1, 1000)
        return dict(op=op, batch=batch, heads=heads, shared=64 * _log(rng, 1, 512), lo=rng.choice([hi, 1]), hi=hi, page=page)
    if op == "weigh":
        batch, heads = _log(rng, 1, 64), rng.choice([1, 8, 16, 40, 64, 128])
        hi = _log(rng, 1, max(1, min(65536, 262144 // batch)))
        return dict(op=op, batch=batch, heads=heads, lo=rng.choice([hi, max(1, hi // 32), 1]), hi=hi, page=page)
    if op == "evict":
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, min(65536, 262144 // batch)))
        keep = _log(rng, 1, min(8192, 131072 // batch))
        return dict(op=op, batch=batch, lo=rng.choice([hi, max(1, hi // 32)]), hi=hi, keep=keep,
                    recent=rng.choice([0, keep // 8, keep]), page=page)
    if rng.random() < 0.4:
        n, k = rng.choice([(512, 128), (128, 512), (192, 96), (100, 160)])
        return dict(op=op, m=_log(rng, 1, 16), n=n, k=k, heads=rng.choice([8, 16, 40, 128]))
    return dict(op=op, m=_log(rng, 1, 16), n=_log(rng, 64, 7168), k=32 * _log(rng, 4, 512), heads=0)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device=DEV)


def _lens(case):
    """Lengths spread over the logarithm of lo..hi; the first is hi."""
    u = [1.0] + [(i * 0.6180339887) % 1.0 for i in range(1, case["batch"])]
    return [int(case["lo"] * (case["hi"] / case["lo"]) ** x) for x in u]


def _power_scale(amax):
    """The smallest power of two 2^e, -60 <= e <= 60, with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax)  # amax = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), torch.full_like(e, -60)).clamp(-60, 60)
    return torch.ldexp(torch.ones_like(amax), e)


def _filled_cache(g, blocks):
    """A cache whose blocks all hold tokens, as append would have left them: latent features normal, one in a hundred 20
    times as large, blocks of different size."""
    codes = torch.empty((blocks * BLOCK, KEY), dtype=E4M3, device=DEV)
    scales = torch.empty(blocks, device=DEV)
    for at in range(0, blocks, 4096):
        n = min(4096, blocks - at)
        x = _randn(g, n * BLOCK, LATENT)
        x = torch.where(_rand(g, n * BLOCK, LATENT) < 0.01, x * 20, x)
        x = torch.cat([x, _randn(g, n * BLOCK, KEY - LATENT)], 1).bfloat16().float().view(n, BLOCK * KEY)
        s = _power_scale(x.abs().amax(1))
        scales[at:at + n] = s
        codes[at * BLOCK:(at + n) * BLOCK] = (x / s[:, None]).view(-1, KEY).to(E4M3)
    return codes, scales


def _tables(ids, need, first=None):
    """Page tables of `need` pages a sequence, taken in turn from ids, behind the pages `first` of all of them."""
    head = 0 if first is None else first.numel()
    table = torch.zeros((len(need), max(1, head + max(need))), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        if head:
            table[b, :head] = first
        table[b, head:head + n] = ids[at:at + n]
        at += n
    return table


def _pages(lens, page):
    return [-(-n // page) for n in lens]


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case)
    if op == "gemv":
        m, n, k, groups = case["m"], case["n"], case["k"], max(1, case["heads"])
        x = _randn(g, m, groups, k)
        s["x"] = torch.where(_rand(g, m, groups, k) < 0.01, x * 20, x).bfloat16()
        w = _randn(g, groups, n, k) / math.sqrt(k)
        s["gs"] = (w.abs().amax() / 2688).reshape(1)
        w = w.view(groups, n, k // 16, 16)
        sf = (w.abs().amax(3) / 6 / s["gs"]).to(E4M3)
        q = w / (sf.float() * s["gs"])[..., None]
        mag = torch.bucketize(q.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV), out_int32=True)
        code = (mag + 8 * (q < 0)).to(torch.uint8).view(groups, n, k // 2, 2)
        s["codes"] = (code[..., 0] | code[..., 1] << 4).contiguous()
        # 128 x 4 scales a tile, row r of it at 16 (r % 32) + 4 (r / 32)
        nt, kt = -(-n // 128), -(-(k // 16) // 4)
        full = torch.zeros((groups, nt * 128, kt * 4), dtype=torch.uint8, device=DEV)
        full[:, :n, :k // 16] = sf.view(torch.uint8)
        s["sf"] = full.view(groups, nt, 4, 32, kt, 4).permute(0, 1, 4, 3, 2, 5).contiguous().view(groups, -1)
        if not case["heads"]:
            s["x"], s["codes"], s["sf"] = s["x"][:, 0].contiguous(), s["codes"][0], s["sf"][0]
        return s
    page, lens = case["page"], _lens(case)
    if op == "shared":
        # the prefix fills whole blocks; where it ends inside a page, that page is cut there for all
        P, rest = case["shared"] // page, case["shared"] % page
        need = _pages([rest + n for n in lens], page)
        ids = torch.randperm(P + sum(need), generator=g, device=DEV).to(torch.int32)
        s["table"] = _tables(ids[P:], need, ids[:P])
        s["cache"], s["scales"] = _filled_cache(g, ids.numel() * page // BLOCK)
        if rest:  # every sequence's copy of the cut page begins alike
            for b in range(1, case["batch"]):
                for buf, unit in ((s["cache"].view(torch.uint8), 1), (s["scales"], BLOCK)):
                    a, z = int(s["table"][0, P]) * page // unit, int(s["table"][b, P]) * page // unit
                    buf[z:z + rest // unit] = buf[a:a + rest // unit]
        lens = [case["shared"] + n for n in lens]
    else:
        need = _pages(lens, page)
        kept = _pages([min(n, case["keep"]) for n in lens], page) if op == "evict" else [0]
        ids = torch.randperm(sum(need) + sum(kept), generator=g, device=DEV).to(torch.int32)
        s["table"] = _tables(ids, need)
        s["cache"], s["scales"] = _filled_cache(g, ids.numel() * page // BLOCK)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if op == "evict":
        s["new_table"] = _tables(ids[sum(need):], kept)
        w = torch.exp(2 * _randn(g, case["batch"], max(lens)))
        s["weights"] = torch.where(_rand(g, *w.shape) < 0.05, 0.0, w)  # far keys' weights are below float32's range
        return s
    B, H = case["batch"], case["heads"]
    s["q"] = _randn(g, B, H, KEY).bfloat16()
    if op == "weigh":
        s["weights"] = torch.exp(_randn(g, B, max(lens)))
        s["out"] = torch.zeros_like(s["weights"])
        s["lse"] = _scores(s)[0]
    return s


# ------------------------------------------------------------- plain forms
def _gather(s, lo, hi):
    """Keys lo..hi of every sequence [B, hi - lo, 576], and which of them are there."""
    t = torch.arange(lo, hi, device=DEV)
    there = t[None] < s["lens"].long()[:, None]
    page = (t // s["page"]).clamp(max=s["table"].shape[1] - 1)
    slot = torch.where(there, s["table"].long()[:, page] * s["page"] + t % s["page"], 0)
    return s["cache"][slot].float() * s["scales"][slot // BLOCK][..., None], there


def _scores(s):
    """(log of the sum of the exponentials, scores) of every head over its sequence's keys."""
    key, there = _gather(s, 0, int(s["weights"].shape[1]))
    x = torch.matmul(s["q"].float(), key.transpose(1, 2)) * SOFTMAX_SCALE
    x = torch.where(there[:, None], x, -math.inf)
    top = x.amax(2, keepdim=True)
    return (top + (x - top).exp().sum(2, keepdim=True).log())[..., 0], x


def _plain_shared(s):
    B, H, L = s["batch"], s["heads"], s["shared"]
    q = s["q"].float()
    t = torch.arange(L, device=DEV)
    slot = s["table"].long()[0, t // s["page"]] * s["page"] + t % s["page"]
    first = s["cache"][slot].float() * s["scales"][slot // BLOCK][:, None]
    x = (torch.matmul(q.view(B * H, KEY), first.t()) * SOFTMAX_SCALE).view(B, H, L)
    key, there = _gather(s, L, L + s["hi"])
    y = torch.matmul(q, key.transpose(1, 2)) * SOFTMAX_SCALE
    y = torch.where(there[:, None], y, -math.inf)
    top = torch.maximum(x.amax(2, keepdim=True), y.amax(2, keepdim=True))
    x, y = (x - top).exp(), (y - top).exp()
    total = x.sum(2, keepdim=True) + y.sum(2, keepdim=True)
    out = torch.matmul(x.view(B * H, L), first[:, :LATENT]).view(B, H, LATENT) + torch.matmul(y, key[..., :LATENT])
    return (out / total).bfloat16(), (top + total.log())[..., 0]


def _plain_weigh(s):
    x = _scores(s)[1]
    p = (x - s["lse"][..., None]).exp().sum(1)
    there = torch.arange(x.shape[2], device=DEV)[None] < s["lens"].long()[:, None]
    s["out"].copy_(torch.where(there, s["weights"] + p, s["out"]))
    return s["out"]


def _plain_evict(s):
    lens, keep, page = s["lens"].long(), s["keep"], s["page"]
    B, W = s["weights"].shape
    t = torch.arange(W, device=DEV)[None]
    left = lens.clamp(max=keep)
    w = torch.where(t >= (lens - s["recent"])[:, None], math.inf, s["weights"])
    w = torch.where(t < lens[:, None], w, -math.inf)
    order = torch.sort(w, dim=1, descending=True, stable=True).indices
    chosen = torch.zeros((B, W), dtype=torch.bool, device=DEV)
    chosen.scatter_(1, order, t < left[:, None])
    b, src = chosen.nonzero(as_tuple=True)  # in order
    i = (chosen.cumsum(1) - 1)[b, src]
    kept = torch.full((B, keep), -1, dtype=torch.int32, device=DEV)
    kept[b, i] = src.int()
    weights = torch.zeros((B, keep), device=DEV)
    weights[b, i] = s["weights"][b, src]
    # the kept tokens as their new blocks hold them
    slot = s["table"].long()[b, src // page] * page + src % page
    new = s["new_table"].long()[b, i // page] * page + i % page
    value = s["cache"][slot].float() * s["scales"][slot // BLOCK][:, None]
    blocks = s["scales"].numel()
    amax = torch.full((blocks,), -1.0, device=DEV).scatter_reduce_(0, new // BLOCK, value.abs().amax(1), "amax")
    scales = torch.where(amax >= 0, _power_scale(amax), s["scales"])
    s["cache"].view(torch.uint8)[new] = (value / scales[new // BLOCK][:, None]).to(E4M3).view(torch.uint8)
    s["scales"].copy_(scales)
    return kept, left.int(), weights, s["cache"], s["scales"]


def _unpacked(s, dtype):
    """The NVFP4 weights [groups, n, k] without their global scale."""
    groups, n, k = max(1, s["heads"]), s["n"], s["k"]
    codes = s["codes"].view(groups, n, k // 2)
    value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=dtype, device=DEV)
    w = torch.stack([value[(codes & 15).long()], value[(codes >> 4).long()]], -1).view(groups, n, k // 16, 16)
    nt, kt = -(-n // 128), -(-(k // 16) // 4)
    sf = s["sf"].view(groups, nt, kt, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(groups, nt * 128, kt * 4)[:, :n, :k // 16]
    return (w * sf.contiguous().view(E4M3).to(dtype)[..., None]).view(groups, n, k)


def _plain_gemv(s):
    x = s["x"].float().view(s["m"], max(1, s["heads"]), s["k"])
    out = torch.matmul(x.transpose(0, 1), _unpacked(s, torch.float32).transpose(1, 2)).transpose(0, 1) * s["gs"]
    return out.reshape(s["x"].shape[:-1] + (s["n"],)).bfloat16()


def run(s):
    op = s["op"]
    if own:
        import mla_attention_nvfp4_gb300 as mla
        if op == "shared":
            return mla.mla_nvfp4_fp8_decode_shared(
                s["q"], s["cache"], s["scales"], SOFTMAX_SCALE, page_table=s["table"], seq_lens=s["lens"],
                shared_len=s["shared"], page_size=s["page"], return_lse=True)
        if op == "weigh":
            return mla.mla_nvfp4_fp8_key_weights(
                s["q"], s["cache"], s["scales"], SOFTMAX_SCALE, s["lse"], page_table=s["table"], seq_lens=s["lens"],
                page_size=s["page"], weights=s["weights"], out=s["out"])
        if op == "evict":
            kept, lens, weights = mla.mla_nvfp4_fp8_cache_evict(
                s["cache"], s["scales"], s["weights"], page_table=s["table"], seq_lens=s["lens"],
                new_page_table=s["new_table"], keep=s["keep"], recent=s["recent"], page_size=s["page"])
            return kept, lens, weights, s["cache"], s["scales"]
        return mla.mla_nvfp4_gemv(s["x"], s["codes"], s["sf"], s["gs"])
    return {"shared": _plain_shared, "weigh": _plain_weigh, "evict": _plain_evict, "gemv": _plain_gemv}[op](s)


# -------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "gemv":
        m, n, k, groups = case["m"], case["n"], case["k"], max(1, case["heads"])
        return {"bytes": groups * (n * k * (1 / 2 + 1 / 16) + 2 * m * (n + k)), "flops": 2.0 * groups * m * n * k}
    lens = _lens(case)
    if op == "shared":
        B, H, L, keys = case["batch"], case["heads"], case["shared"], sum(lens)
        return {"bytes": (L + keys) * (KEY + 4 / BLOCK) + B * H * (KEY * 2 + LATENT * 2 + 4),
                "flops": 2.0 * H * (B * L + keys) * (KEY + LATENT)}
    if op == "weigh":
        # keys, and the weights read and written; queries and their sums
        keys, rows = sum(lens), case["batch"] * case["heads"]
        return {"bytes": keys * (KEY + 4 / BLOCK + 8) + rows * (KEY * 2 + 4), "flops": 2.0 * keys * case["heads"] * KEY}
    # the weights; the kept rows read and written, with their scales, indices and weights
    left = [min(n, case["keep"]) for n in lens]
    return {"bytes": 4 * sum(lens) + sum(left) * (2 * KEY + 8 / BLOCK) + case["batch"] * (8 * case["keep"] + 4),
            "flops": float(sum(lens))}


# ------------------------------------------------------------ in 64 bits
def _e4m3(v):
    """v (float64) to the nearest e4m3 value, ties to the even one, at most 448."""
    a = v.abs()
    e = torch.frexp(a.clamp(min=2.0 ** -40))[1].double() - 1
    step = torch.exp2(e.clamp(min=-6) - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), v)


def _slots(table, page, t):
    return table[t // page] * page + t % page


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "gemv":
        w = _unpacked_by_tile(s)
        x = s["x"].double().view(case["m"], -1, case["k"])
        out = torch.stack([x[:, i] @ w[i].T for i in range(w.shape[0])], 1) * s["gs"].double()
        return out.view(s["x"].shape[:-1] + (case["n"],))
    lens, page, table = s["lens"].tolist(), case["page"], s["table"].long()
    if op == "evict":
        return _exact_evict(case, s, lens)
    out, lse = [], []
    if op == "weigh":
        total = s["out"].double()
    for b, n in enumerate(lens):
        slot = _slots(table[b], page, torch.arange(n, device=DEV))
        key = s["cache"][slot].double() * s["scales"][slot // BLOCK].double()[:, None]
        x = (s["q"][b].double() @ key.T) * SOFTMAX_SCALE
        if op == "weigh":
            total[b, :n] = s["weights"][b, :n].double() + torch.exp(x - s["lse"][b].double()[:, None]).sum(0)
        else:
            ln = torch.logsumexp(x, 1)
            out.append(torch.exp(x - ln[:, None]) @ key[:, :LATENT])
            lse.append(ln)
    return total if op == "weigh" else (torch.stack(out), torch.stack(lse))


def _unpacked_by_tile(s):
    """The weights in float64, element by element of the packed layout."""
    groups, n, k = max(1, s["heads"]), s["n"], s["k"]
    r, c = torch.arange(n, device=DEV)[:, None], torch.arange(k, device=DEV)[None]
    tiles = -(-(k // 16) // 4)
    at = (r // 128 * tiles + c // 64) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c // 16 % 4
    codes, sf = s["codes"].view(groups, n, k // 2), s["sf"].view(groups, -1)
    out = torch.empty((groups, n, k), dtype=torch.float64, device=DEV)
    for i in range(groups):
        nibble = (codes[i][:, torch.arange(k, device=DEV) // 2].int() >> (4 * (c % 2))) & 15
        e, m = (nibble >> 1 & 3).double(), (nibble & 1).double()
        mag = torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)
        out[i] = torch.where(nibble >= 8, -mag, mag) * sf[i][at].view(E4M3).double()
    return out


def _exact_evict(case, s, lens):
    keep, page = case["keep"], case["page"]
    table, fresh = s["table"].long(), s["new_table"].long()
    cache, scales = s["cache"].double(), s["scales"].double()
    kept = torch.full((case["batch"], keep), -1, dtype=torch.int32, device=DEV)
    weights = torch.zeros((case["batch"], keep), dtype=torch.float64, device=DEV)
    left = []
    for b, n in enumerate(lens):
        w = s["weights"][b, :n].double().cpu().numpy()
        old = max(0, n - case["recent"])
        by_weight = np.lexsort((np.arange(old), -w[:old]))
        m = min(n, keep)
        chosen = np.sort(np.concatenate([by_weight[:m - (n - old)] if m > n - old else by_weight[:0], np.arange(old, n)[:m]]))
        src = torch.from_numpy(chosen).to(DEV)
        kept[b, :m], weights[b, :m] = src.int(), s["weights"][b, src].double()
        left.append(m)
        slot = _slots(table[b], page, src)
        value = s["cache"][slot].double() * s["scales"][slot // BLOCK].double()[:, None]
        for i in range(0, m, BLOCK):
            part = value[i:i + BLOCK]
            most = float(part.abs().amax())
            power = 2.0 ** (max(-60, min(60, math.ceil(math.log2(most / 448)))) if most > 0 else -60)
            at = int(_slots(fresh[b], page, torch.tensor(i, device=DEV)))
            scales[at // BLOCK] = power
            cache[at:at + len(part)] = _e4m3(part / power)
    return kept, torch.tensor(left, dtype=torch.int32, device=DEV), weights, cache, scales
