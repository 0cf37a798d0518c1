"""The 8-bit operators beside the 4-bit ones: what is measured, and their plain forms.

Four operators on E4M3 codes under FP32 block scales:

- ``quant``   bf16 [M, K] -> codes, one scale per 1 x 128 block ("row") or 128 x 128 block ("tile"),
              optionally also of the transposed matrix;
- ``gemm``    D = A B^T of two such tensors;
- ``append``  new tokens' K and V into a paged 8-bit cache, one power-of-two scale per page and head;
- ``attn``    attention of bf16 queries over that cache, for single tokens and for chunks of a prompt.

With ``own`` false, ``run`` computes each from elementary torch operations in 32 bits; with ``own``
true, it makes the library's calls.
"""
import math

import torch

own = False

BLOCK = 128
FP8 = torch.float8_e4m3fn


def listed():
    return [
        # one decoded token's activation row on its way into an 8-bit product: launch latency
        {"name": "quant_row_1x4096", "op": "quant", "M": 1, "K": 4096, "block": "row", "transpose": False},
        # a training step's activations: rows for the forward product, columns for the weight gradient
        {"name": "quant_both_8192x4096", "op": "quant", "M": 8192, "K": 4096, "block": "row", "transpose": True},
        # a weight and its transpose (input gradient), sizes that end inside a block
        {"name": "quant_tile_4097x4344", "op": "quant", "M": 4097, "K": 4344, "block": "tile", "transpose": True},
        # one decoded token through a square projection: reading the weight is all there is
        {"name": "gemm_1x4096x4096", "op": "gemm", "M": 1, "N": 4096, "K": 4096, "b_block": "tile", "out": "bf16"},
        # a decoding batch of odd size
        {"name": "gemm_37x4096x4352", "op": "gemm", "M": 37, "N": 4096, "K": 4352, "b_block": "tile", "out": "bf16"},
        # a prompt or training batch through a square projection (also the input gradient's form)
        {"name": "gemm_8192x4096x4096", "op": "gemm", "M": 8192, "N": 4096, "K": 4096, "b_block": "tile", "out": "bf16"},
        # the weight gradient: both operands have row scales, the sum runs over the tokens, the result is fp32
        {"name": "gemm_wgrad_4096x4096x8190", "op": "gemm", "M": 4096, "N": 4096, "K": 8190, "b_block": "row", "out": "fp32"},
        # a decoding step of 64 sequences: one token each, somewhere inside their last pages
        {"name": "append_64x1", "op": "append", "B": 64, "new": 1, "old": 1000, "Hkv": 8, "D": 128, "page": 64},
        # four prompts of different lengths written at once
        {"name": "append_4x2048", "op": "append", "B": 4, "new": 2048, "old": 0, "Hkv": 8, "D": 128, "page": 64},
        # one short conversation's next token: latency
        {"name": "attn_1x1_500", "op": "attn", "B": 1, "new": 1, "len": 500, "Hkv": 8, "G": 4, "D": 128, "page": 64},
        # a decoding batch with ragged lengths: reading the cache is all there is
        {"name": "attn_32x1_8192", "op": "attn", "B": 32, "new": 1, "len": 8192, "Hkv": 8, "G": 4, "D": 128, "page": 64},
        # chunks of two prompts over what is cached of them
        {"name": "attn_2x1000_4096", "op": "attn", "B": 2, "new": 1000, "len": 4096, "Hkv": 8, "G": 4, "D": 128, "page": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "gemm", "gemm", "append", "attn", "attn"])
    if op == "quant":
        return {"op": op, "M": _log(rng, 1, 8192), "K": _log(rng, 64, 4096), "block": rng.choice(["row", "tile"]),
                "transpose": rng.random() < 0.5}
    if op == "gemm":
        return {"op": op, "M": _log(rng, 1, 8192), "N": 8 * _log(rng, 8, 512), "K": _log(rng, 100, 4096),
                "b_block": rng.choice(["row", "tile"]), "out": rng.choice(["bf16", "fp32"])}
    hkv, d, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    if op == "append":
        new = _log(rng, 1, 2048)
        return {"op": op, "B": max(1, min(64, _log(rng, 1, 64), 8192 // new)), "new": new, "old": rng.choice([0, _log(rng, 1, 2000)]),
                "Hkv": hkv, "D": d, "page": page}
    if rng.random() < 0.7:  # single tokens, or the few of a speculative step
        new, most = rng.choice([1, 1, 1, 2, 4]), 32
        length = _log(rng, 16, 8192)
    else:
        new, most = _log(rng, 16, 1000), 2
        length = max(new, _log(rng, 64, 4096))
    return {"op": op, "B": _log(rng, 1, most), "new": new, "len": length, "Hkv": hkv, "G": rng.choice([1, 2, 4]), "D": d, "page": page}


# ------------------------------------------------------------------ lengths: a property of the case, whatever the seed

def _spread(n, most, least):
    """n lengths between least and most, the longest among them, unevenly spread."""
    return [max(least, most - (most - least) * ((i * 7) % n) // max(1, n) // (1 + i % 2)) for i in range(n)]


def _lengths(c):
    """(new tokens, cached tokens before them) of each sequence."""
    if c["op"] == "append":
        new = _spread(c["B"], c["new"], max(1, c["new"] // 2))
        old = _spread(c["B"], c["old"], c["old"] // 2)
    else:
        new = _spread(c["B"], c["new"], max(1, c["new"] // 2))
        old = [max(0, t - n) for t, n in zip(_spread(c["B"], c["len"], max(1, c["len"] // 4)), new)]
    return new, old


def _pairs(c):
    """Query-key pairs of one head."""
    return sum(n * o + n * (n + 1) // 2 for n, o in zip(*_lengths(c)))


# ------------------------------------------------------------------ inputs

def _activations(g, *shape):
    """bf16 activations: a normal bulk whose last-axis channels have gains of their own, a few of them large."""
    gain = torch.exp(0.5 * torch.randn(shape[-1], generator=g, device="cuda"))
    gain = torch.where(torch.rand(shape[-1], generator=g, device="cuda") < 0.01, gain * 20, gain)
    return (torch.randn(shape, generator=g, device="cuda") * gain).to(torch.bfloat16)


def _e4m3(v):
    return v.clamp(-448.0, 448.0).to(FP8)


def _spans(n):
    return -(-n // BLOCK)


def _row_quant(x):
    """Codes [M, K] and scales [K/128, M] of the 1 x 128 blocks of x."""
    M, K = x.shape
    kb = _spans(K)
    v = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - K)).view(M, kb, BLOCK)
    s = v.abs().amax(-1) / 448.0
    q = torch.where(s.unsqueeze(-1) > 0, v / s.unsqueeze(-1), torch.zeros_like(v))
    return _e4m3(q).view(M, kb * BLOCK)[:, :K], s.t().contiguous()


def _tile_quant(x):
    """Codes [M, K] and scales [K/128, M/128] of the 128 x 128 blocks of x."""
    M, K = x.shape
    mb, kb = _spans(M), _spans(K)
    v = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - K, 0, mb * BLOCK - M)).view(mb, BLOCK, kb, BLOCK)
    s = v.abs().amax((1, 3)) / 448.0
    e = s[:, None, :, None]
    q = torch.where(e > 0, v / e, torch.zeros_like(v))
    return _e4m3(q).view(mb * BLOCK, kb * BLOCK)[:M, :K], s.t().contiguous()


def _padded(codes, scales):
    """The operands as a program holds them: rows of codes 16 bytes apart in step, scale rows 4 floats in step."""
    M, K = codes.shape
    c = torch.zeros((M, -(-K // 16) * 16), dtype=torch.uint8, device=codes.device)
    c[:, :K] = codes.contiguous().view(torch.uint8)
    s = torch.zeros((scales.shape[0], -(-scales.shape[1] // 4) * 4), device=codes.device)
    s[:, :scales.shape[1]] = scales
    return c[:, :K], s[:, :scales.shape[1]]


def _cache(g, pages, hkv, page, d):
    """One side of a cache: codes [pages, hkv, page, d] and their scales, of normal values with channel gains."""
    gain = torch.exp(0.4 * torch.randn((hkv, 1, d), generator=g, device="cuda"))
    codes = torch.empty((pages, hkv, page, d), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages, hkv), device="cuda")
    step = max(1, (1 << 26) // (hkv * page * d))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        v = torch.randn((n, hkv, page, d), generator=g, device="cuda") * gain
        s = torch.exp2(torch.ceil(torch.log2(v.abs().amax((2, 3)) / 448.0)))
        codes[p:p + n] = _e4m3(v / s[:, :, None, None]).view(torch.uint8)
        scales[p:p + n] = s
    return codes, scales


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    if c["op"] == "quant":
        return {"c": c, "x": _activations(g, c["M"], -(-c["K"] // 8) * 8)[:, :c["K"]]}
    if c["op"] == "gemm":
        a = _row_quant(_activations(g, c["M"], c["K"]))
        w = torch.randn((c["N"], c["K"]), generator=g, device="cuda").to(torch.bfloat16)
        b = (_tile_quant if c["b_block"] == "tile" else _row_quant)(w)
        return {"c": c, "a": _padded(*a), "b": _padded(*b)}
    new, old = _lengths(c)
    B, page, hkv, d = c["B"], c["page"], c["Hkv"], c["D"]
    need = [-(-(n + o) // page) for n, o in zip(new, old)]
    pages = sum(need) + 3  # a pool has pages that no sequence here holds
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((B, max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    s = {"c": c, "table": table, "max_new": max(new), "max_len": max(n + o for n, o in zip(new, old))}
    s["k"], s["ks"] = _cache(g, pages, hkv, page, d)
    s["v"], s["vs"] = _cache(g, pages, hkv, page, d)
    cum = [0]
    for n in new:
        cum.append(cum[-1] + n)
    s["cum"] = torch.tensor(cum, dtype=torch.int32, device="cuda")
    s["len"] = torch.tensor([n + o for n, o in zip(new, old)], dtype=torch.int32, device="cuda")
    if c["op"] == "append":
        s["new_k"] = _activations(g, cum[-1], hkv, d)
        s["new_v"] = _activations(g, cum[-1], hkv, d)
    else:
        s["q"] = torch.randn((cum[-1], hkv * c["G"], d), generator=g, device="cuda").to(torch.bfloat16)
        s["ws"] = None
        if own:
            import fp4_micro_block_b200 as fq
            s["ws"] = fq.attention_fp8_workspace(s["q"], s["k"], B, s["max_new"], s["max_len"])
    return s


# ------------------------------------------------------------------ the plain forms

def _plain_gemm(s):
    def values(codes, scales, block):
        n, k = codes.shape
        e = scales.repeat_interleave(BLOCK, 0)[:k]
        if block == "tile":
            e = e.repeat_interleave(BLOCK, 1)[:, :n]
        return codes.contiguous().view(FP8).float() * e.t()

    c = s["c"]
    d = values(*s["a"], "row") @ values(*s["b"], c["b_block"]).t()
    return d if c["out"] == "fp32" else d.to(torch.bfloat16)


def _plain_places(s):
    """(sequence, position) of each new token."""
    t = torch.arange(int(s["q" if "q" in s else "new_k"].shape[0]), device="cuda")
    seq = (torch.searchsorted(s["cum"].long(), t, right=True) - 1)
    pos = s["len"].long()[seq] - s["cum"].long()[seq + 1] + t
    return t, seq, pos


def _power(amax):
    """The smallest power of two s with amax / s <= 448, at least 2^-126; 0 for 0."""
    f, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), torch.where(f <= 0.875, e - 9, e - 8).clamp(min=-126))
    return torch.where(amax > 0, s, torch.zeros_like(s))


def _plain_append_side(x, cache, scale, page_of, off, kept):
    """x [T, h, d] into cache at (page_of, off); kept [pages]: tokens that a page holds already."""
    pages, h, page, d = cache.shape
    amax = torch.zeros((pages, h), device="cuda")
    amax.scatter_reduce_(0, page_of[:, None].expand(-1, h), x.float().abs().amax(-1), "amax")
    touched = torch.zeros(pages, dtype=torch.bool, device="cuda")
    touched[page_of] = True
    old = torch.where((touched & (kept > 0))[:, None], scale, torch.zeros_like(scale))
    now = torch.where(touched[:, None], torch.maximum(old, _power(amax)), scale)
    # what the page holds moves to the new scale
    moved = touched.nonzero()[:, 0]
    ratio = torch.where(now[moved] > 0, old[moved] / now[moved], torch.zeros_like(now[moved]))
    codes = cache[moved].view(FP8).float()
    again = _e4m3(codes * ratio[:, :, None, None]).view(torch.uint8)
    held = torch.arange(page, device="cuda")[None, :] < kept[moved][:, None]
    cache[moved] = torch.where(held[:, None, :, None], again, cache[moved])
    scale.copy_(now)
    e = now[page_of][:, :, None]
    q = torch.where(e > 0, x.float() / e, torch.zeros((), device="cuda"))
    cache[page_of, :, off] = _e4m3(q).view(torch.uint8)


def _plain_append(s):
    page = s["c"]["page"]
    t, seq, pos = _plain_places(s)
    page_of = s["table"].long()[seq, pos // page]
    begin = s["len"].long() - (s["cum"].long()[1:] - s["cum"].long()[:-1])  # tokens before this call
    kept = torch.zeros(s["k"].shape[0], dtype=torch.int64, device="cuda")
    kept[page_of] = (begin[seq] - pos // page * page).clamp(min=0)
    for x, cache, scale in (("new_k", "k", "ks"), ("new_v", "v", "vs")):
        _plain_append_side(s[x], s[cache], s[scale], page_of, pos % page, kept)
    return s["k"].view(FP8), s["ks"], s["v"].view(FP8), s["vs"]


def _plain_attn(s):
    c = s["c"]
    B, h, g, d, page = c["B"], c["Hkv"], c["G"], c["D"], c["page"]
    t, seq, pos = _plain_places(s)
    pages = s["table"].long()

    def gathered(cache, scale):  # [B, h, tokens, d]
        v = cache[pages].view(FP8).float() * scale[pages][..., None, None]
        return v.permute(0, 2, 1, 3, 4).reshape(B, h, -1, d)

    k, v = gathered(s["k"], s["ks"]), gathered(s["v"], s["vs"])
    n = s["max_new"]
    slot = t - s["cum"].long()[seq]
    q = torch.zeros((B, n, h, g, d), device="cuda")
    q[seq, slot] = s["q"].float().view(-1, h, g, d)
    at = torch.full((B, n), -1, dtype=torch.int64, device="cuda")
    at[seq, slot] = pos
    q = q.permute(0, 2, 3, 1, 4).reshape(B, h, g * n, d)
    w = (q @ k.transpose(-1, -2)).view(B, h, g, n, -1) * (1.0 / math.sqrt(d))
    w = w.masked_fill(torch.arange(k.shape[2], device="cuda") > at[:, None, None, :, None], -math.inf)
    top = w.amax(-1, keepdim=True)
    p = torch.exp(w - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, h, g * n, -1) @ v).view(B, h, g, n, d) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total))[..., 0]
    pick = lambda a: a.permute(0, 3, 1, 2, *range(4, a.dim()))[seq, slot]  # noqa: E731
    return pick(o).reshape(-1, h * g, d).to(torch.bfloat16), pick(lse).reshape(-1, h * g)


def _plain_quant(s):
    c, x = s["c"], s["x"]
    q = _row_quant if c["block"] == "row" else _tile_quant
    return (*q(x), *(q(x.t()) if c["transpose"] else ()))


def _own_quant(s, fq):
    c = s["c"]
    block = fq.FP4Q_FP8_ROW if c["block"] == "row" else fq.FP4Q_FP8_TILE
    out = fq.quantize_fp8(s["x"], block, transpose=c["transpose"])
    return tuple(o.view(FP8) if o.dtype == torch.uint8 else o for o in out)


def run(state):
    s, op = state, state["c"]["op"]
    if not own:
        return {"quant": _plain_quant, "gemm": _plain_gemm, "append": _plain_append, "attn": _plain_attn}[op](s)
    import fp4_micro_block_b200 as fq
    if op == "quant":
        return _own_quant(s, fq)
    if op == "gemm":
        c = s["c"]
        return fq.gemm_fp8(*s["a"], *s["b"], fq.FP4Q_FP8_TILE if c["b_block"] == "tile" else fq.FP4Q_FP8_ROW,
                           torch.float32 if c["out"] == "fp32" else torch.bfloat16)
    if op == "append":
        fq.kv_append_fp8(s["new_k"], s["new_v"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["cum"], s["len"], s["max_new"])
        return s["k"].view(FP8), s["ks"], s["v"].view(FP8), s["vs"]
    return fq.attention_fp8(s["q"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["cum"], s["len"],
                            s["max_new"], s["max_len"], causal=True, ws=s["ws"])


def work(case):
    c = case
    if c["op"] == "quant":
        n = c["M"] * c["K"]
        row = c["block"] == "row"
        scales = _spans(c["K"]) * (c["M"] if row else _spans(c["M"]))
        scales_t = _spans(c["M"]) * (c["K"] if row else _spans(c["K"]))
        return {"bytes": 2 * n + n + 4 * scales + ((n + 4 * scales_t) if c["transpose"] else 0), "flops": 2 * n}
    if c["op"] == "gemm":
        m, n, k = c["M"], c["N"], c["K"]
        scales = _spans(k) * (m + (n if c["b_block"] == "row" else _spans(n)))
        return {"bytes": m * k + n * k + 4 * scales + m * n * (4 if c["out"] == "fp32" else 2), "flops": 2 * m * n * k}
    new, old = _lengths(c)
    tokens, hd = sum(new), c["Hkv"] * c["D"]
    if c["op"] == "append":  # the new tokens' K and V read, their codes and their pages' scales written
        pages = sum(-(-(n + o) // c["page"]) - o // c["page"] for n, o in zip(new, old))
        return {"bytes": 2 * tokens * hd * 3 + 2 * 4 * pages * c["Hkv"], "flops": 4 * tokens * hd}
    keys = sum(new) + sum(old)
    return {"bytes": 2 * keys * hd + tokens * hd * c["G"] * 4 + 4 * tokens * c["Hkv"] * c["G"], "flops": 4 * _pairs(c) * hd * c["G"]}


# ------------------------------------------------------------------ the definition in 64 bits

def _round_e4m3(v):
    """Nearest E4M3 value, ties to even, saturating, of float64 values (3 fraction bits, smallest step 2^-9)."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20)))
    e = torch.where(torch.exp2(e) > v.abs().clamp(min=2.0 ** -20), e - 1, e).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_quant(x, block):
    M, K = x.shape
    rows = torch.arange(M, device="cuda") if block == "row" else torch.arange(M, device="cuda") // BLOCK
    v = x.double()
    codes = torch.empty_like(v)
    scales = torch.empty((_spans(K), int(rows[-1]) + 1), dtype=torch.float64, device="cuda")
    for kb in range(_spans(K)):
        part = v[:, kb * BLOCK:(kb + 1) * BLOCK]
        top = torch.zeros(scales.shape[1], dtype=torch.float64, device="cuda").scatter_reduce(0, rows, part.abs().amax(1), "amax")
        scales[kb] = top / 448.0
        e = (top / 448.0).float().double()[rows][:, None]  # a scale is held in 32 bits
        codes[:, kb * BLOCK:(kb + 1) * BLOCK] = torch.where(e > 0, _round_e4m3(part / e.clamp(min=1e-300)), torch.zeros_like(part))
    return codes, scales


def _exact_gemm(s):
    (a, sa), (b, sb) = s["a"], s["b"]
    M, K = a.shape
    d = torch.zeros((M, b.shape[0]), dtype=torch.float64, device="cuda")
    for kb in range(_spans(K)):
        cut = slice(kb * BLOCK, min(K, (kb + 1) * BLOCK))
        part = a[:, cut].contiguous().view(FP8).double() @ b[:, cut].contiguous().view(FP8).double().t()
        col = sb[kb].double() if s["c"]["b_block"] == "row" else sb[kb].double().repeat_interleave(BLOCK)[:b.shape[0]]
        d += part * sa[kb].double()[:, None] * col
    return d


def _exact_append(s):
    c = s["c"]
    new, old = _lengths(c)
    page, at, out = c["page"], 0, []
    for x, cache, scale in (("new_k", "k", "ks"), ("new_v", "v", "vs")):
        values = s[cache].view(FP8).double()
        scales = s[scale].double()
        at = 0
        for i, (n, o) in enumerate(zip(new, old)):
            for p in range(o // page, -(-(n + o) // page)):
                lo, hi = max(o, p * page), min(n + o, (p + 1) * page)
                v = s[x][at + lo - o:at + hi - o].double().transpose(0, 1)  # [h, tokens, d]
                where = int(s["table"][i, p])
                top = v.abs().amax((1, 2))
                frac, power = torch.frexp(top / 448.0)  # in [1/2, 1): a half is a power of two itself
                want = torch.ldexp(torch.ones_like(top), torch.where(frac == 0.5, power - 1, power)).clamp(min=2.0 ** -126)
                want = torch.where(top > 0, want, torch.zeros_like(want))
                kept = lo - p * page
                if kept:
                    want = torch.maximum(want, scales[where])
                    values[where, :, :kept] = _round_e4m3(values[where, :, :kept] * (scales[where] / want)[:, None, None])
                scales[where] = want
                values[where, :, kept:kept + hi - lo] = _round_e4m3(v / want[:, None, None])
            at += n
        out += [values, scales]
    return tuple(out)


def _exact_attn(s):
    c = s["c"]
    new, old = _lengths(c)
    h, g, d = c["Hkv"], c["G"], c["D"]
    o = torch.zeros((sum(new), h * g, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((sum(new), h * g), dtype=torch.float64, device="cuda")
    at = 0
    for i, (n, before) in enumerate(zip(new, old)):
        total = n + before
        pages = s["table"][i, :-(-total // c["page"])].long()
        seen = torch.arange(total, device="cuda")[None, :] <= (before + torch.arange(n, device="cuda"))[:, None]
        for j in range(h):
            k = (s["k"][pages, j].view(FP8).double() * s["ks"][pages, j].double()[:, None, None]).reshape(-1, d)[:total]
            v = (s["v"][pages, j].view(FP8).double() * s["vs"][pages, j].double()[:, None, None]).reshape(-1, d)[:total]
            for q in range(j * g, (j + 1) * g):
                w = s["q"][at:at + n, q].double() @ k.t() / math.sqrt(d)
                w = torch.where(seen, w, torch.full_like(w, -math.inf))
                lse[at:at + n, q] = torch.logsumexp(w, 1)
                o[at:at + n, q] = torch.softmax(w, 1) @ v
        at += n
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "quant":
        out = _exact_quant(s["x"], c["block"])
        return (*out, *(_exact_quant(s["x"].t(), c["block"]) if c["transpose"] else ()))
    return {"gemm": _exact_gemm, "append": _exact_append, "attn": _exact_attn}[c["op"]](s)
