"""Cases, plain forms and 64-bit values of the operators that answer token by token.

Three operators of the decode path of a model whose linears are quantized:

``gemv``    y = x W^T (+ bias) for a few rows of bf16 x that are not quantized, W in NVFP4
            (E2M1 codes, one E4M3 scale per 16 weights in the tensor-core layout, an fp32
            global scale): the package's ``nvfp4_gemv``.
``append``  rotary positions on the new tokens' q and k, then k and v into a paged E4M3
            cache with one power-of-two scale (E8M0) for each block of 16 tokens and head:
            ``fp8kv_append``.
``attend``  attention of the new tokens over that cache: ``fp8kv_attention``.

Where ``own`` is false, ``run`` computes the same with elementary torch operations.
"""
import math
import random

import torch

own = False

BLOCK = 16          # tokens that share one scale of the cache
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a projection of one token: the smallest weight a decode step multiplies by
        dict(name="gemv one token", op="gemv", M=1, N=4096, K=4096, bias=False),
        # seven draft tokens through a layer whose sizes fill no tile
        dict(name="gemv seven rows odd sizes", op="gemv", M=7, N=10376, K=2624, bias=True),
        # a decode batch of 16 through the wide half of an MLP
        dict(name="gemv batch of 16", op="gemv", M=16, N=16384, K=12288, bias=True),
        # one token against a large vocabulary
        dict(name="gemv output head", op="gemv", M=1, N=131072, K=8192, bias=False),
        # one token of one sequence, every dimension of the head rotated
        dict(name="append one token", op="append", B=1, new_lo=1, new_hi=1, past_lo=1003,
             past_hi=1003, Hq=32, Hkv=8, D=128, page=64, rot=128, interleaved=False,
             rope_scale=1.0, theta=10000.0, lens_seed=1),
        # a serving step: one token for each of 192 sequences, some far into their context
        dict(name="append decode batch", op="append", B=192, new_lo=1, new_hi=1, past_lo=0,
             past_hi=500000, Hq=32, Hkv=8, D=128, page=64, rot=128, interleaved=False,
             rope_scale=1.0, theta=500000.0, lens_seed=2),
        # ragged chunks (some sequences bring nothing), one head per key head, a small page
        dict(name="append ragged chunks", op="append", B=9, new_lo=0, new_hi=70, past_lo=0,
             past_hi=3000, Hq=20, Hkv=20, D=80, page=16, rot=32, interleaved=False,
             rope_scale=1.0, theta=10000.0, lens_seed=3),
        # prompts being read in: half of each head rotated in pairs, stretched positions
        dict(name="append prompts", op="append", B=3, new_lo=2900, new_hi=5300, past_lo=0,
             past_hi=40, Hq=32, Hkv=8, D=128, page=64, rot=64, interleaved=True,
             rope_scale=1.2079, theta=1000000.0, lens_seed=4),
        # one token against a short context: latency
        dict(name="attend short", op="attend", B=1, new=1, len_lo=517, len_hi=517, Hq=32, Hkv=8,
             D=128, page=64, window=0, lens_seed=5),
        # four draft tokens for each of 16 sequences, small heads, sliding window, small page
        dict(name="attend draft tokens", op="attend", B=16, new=4, len_lo=3, len_hi=4096, Hq=16,
             Hkv=16, D=64, page=16, window=1024, lens_seed=6),
        # one long context
        dict(name="attend long context", op="attend", B=1, new=1, len_lo=131071, len_hi=131071,
             Hq=64, Hkv=8, D=128, page=64, window=0, lens_seed=7),
        # a serving step over sequences of very different lengths
        dict(name="attend decode batch", op="attend", B=64, new=1, len_lo=64, len_hi=16384, Hq=32,
             Hkv=8, D=128, page=64, window=0, lens_seed=8),
    ]


def _log_int(rng, lo, hi, unit=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / unit)) * unit))


def draw(rng):
    op = rng.choice(("gemv", "append", "attend"))
    if op == "gemv":
        while True:
            N, K = _log_int(rng, 256, 131072, 8), _log_int(rng, 256, 16384, 64)
            if N * K <= 131072 * 8192 // 2:
                break
        return dict(op=op, M=_log_int(rng, 1, 32), N=N, K=K, bias=rng.random() < 0.5)
    Hkv, G = rng.choice((1, 2, 4, 5, 8, 16)), rng.choice((1, 2, 3, 4, 6, 7, 8))
    D, page = rng.choice((64, 80, 96, 128, 128, 128, 192, 256)), rng.choice((16, 32, 48, 64, 128))
    B = _log_int(rng, 1, 160)
    if op == "append":
        hi = max(1, min(_log_int(rng, 1, 6000), 12000 * 5120 // (B * Hkv * (G + 2) * D)))
        return dict(op=op, B=B, new_lo=rng.choice((0, 1, (hi + 1) // 2)), new_hi=hi, past_lo=0,
                    past_hi=_log_int(rng, 1, 1000000), Hq=Hkv * G, Hkv=Hkv, D=D, page=page,
                    rot=rng.choice((16, 32, 64, D // 16 * 16)), interleaved=rng.random() < 0.5,
                    rope_scale=rng.choice((1.0, 1.1386)), theta=rng.choice((1e4, 5e5, 1e6)),
                    lens_seed=rng.randrange(1 << 20))
    top = max(64, min(131072, 131072 * 8 * 128 // (B * Hkv * D)))
    hi = _log_int(rng, 64, top)
    return dict(op=op, B=B, new=rng.choice((1, 1, 1, 2, 3, 5, 8)), len_lo=max(8, hi // rng.choice((1, 4, 64))),
                len_hi=hi, Hq=Hkv * G, Hkv=Hkv, D=D, page=page,
                window=rng.choice((0, 0, 0, 1 + hi // 3)), lens_seed=rng.randrange(1 << 20))


def _lens(c):
    """(new tokens, whole length) of each sequence: part of the case, not of the seed."""
    r = random.Random(c["lens_seed"])
    if c["op"] == "append":
        n = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["B"])]
        if sum(n) == 0:
            n[0] = 1
        past = [int(math.exp(r.uniform(math.log(c["past_lo"] + 1), math.log(c["past_hi"] + 1)))) - 1
                for _ in range(c["B"])]
        past = [min(max(p, c["past_lo"]), c["past_hi"]) for p in past]
        return n, [p + m for p, m in zip(past, n)]
    L = [int(round(math.exp(r.uniform(math.log(c["len_lo"]), math.log(c["len_hi"])))))
         for _ in range(c["B"])]
    return [c["new"]] * c["B"], L


def work(case):
    c = case
    if c["op"] == "gemv":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": N * K // 2 + N * K // 16 + 2 * M * K + 2 * M * N + 2 * N * c["bias"] + 4,
                "flops": 2.0 * M * N * K}
    n, L = _lens(c)
    T, Hq, Hkv, D = sum(n), c["Hq"], c["Hkv"], c["D"]
    meta = 4 * (2 * c["B"] + 1)
    if c["op"] == "append":
        pages = sum((l - 1) // c["page"] - (l - m) // c["page"] + 1 for m, l in zip(n, L) if m)
        blocks = sum((l - 1) // BLOCK - (l - m) // BLOCK + 1 for m, l in zip(n, L) if m)
        return {"bytes": T * D * (4 * Hq + 4 * Hkv + 2 * Hkv) + blocks * Hkv * 2 + 4 * pages
                + meta + 2 * c["rot"],
                "flops": 3.0 * T * c["rot"] * (Hq + Hkv) + 4.0 * T * Hkv * D}
    span = [min(l, c["window"] + m - 1) if c["window"] else l for m, l in zip(n, L)]
    kv = sum(s * Hkv * 2 * D + -(-s // BLOCK) * Hkv * 2 + 4 * -(-s // c["page"]) for s in span)
    return {"bytes": kv + T * Hq * (4 * D + 4) + meta,
            "flops": sum(4.0 * m * Hq * D * s for m, s in zip(n, span))}


# ------------------------------------------------------------------ inputs
def _mma_layout(sf):
    """Scales [N, K/16] in the tensor-core layout: 512-byte tiles of 128 rows x 4 columns."""
    N, nb = sf.shape
    full = torch.zeros(((N + 127) // 128 * 128, nb), dtype=sf.dtype, device=sf.device)
    full[:N] = sf
    t = full.view(-1, 4, 32, nb // 4, 4)            # row tile, row / 32, row % 32, column tile, column
    return t.permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _linear_layout(sf, N, K):
    nb = K // 16
    t = sf.view(-1, nb // 4, 32, 4, 4)
    return t.permute(0, 3, 2, 1, 4).reshape(-1, nb)[:N]


def _quantized_weight(N, K, g, dev):
    """NVFP4 codes, scales and global scale of N(0, 0.02) weights."""
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    sf = torch.empty((N, K // 16), dtype=torch.uint8, device=dev)
    scale = torch.full((1,), 0.02 * 6.5 / (448 * 6), dtype=torch.float32, device=dev)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=dev)
    rows = max(1, (1 << 27) // K)
    for r in range(0, N, rows):
        w = torch.randn((min(rows, N - r), K // 16, 16), device=dev, generator=g) * 0.02
        s = (w.abs().amax(-1, keepdim=True) / (6 * scale)).clamp(max=448).to(torch.float8_e4m3fn)
        sf[r:r + rows] = s.view(torch.uint8).squeeze(-1)
        q = w / (s.float() * scale).clamp(min=1e-30)
        c = torch.bucketize(q.abs(), edges).to(torch.uint8) | (q < 0).to(torch.uint8) << 3
        c = c.view(-1, K // 2, 2)
        codes[r:r + rows] = c[..., 0] | c[..., 1] << 4
    return codes, _mma_layout(sf), scale


def _cache(pages, c, g, dev):
    """A pool of cached values: N(0, 1) with a spread of sizes over channels and blocks."""
    Hkv, D, page = c["Hkv"], c["D"], c["page"]
    codes = torch.empty((pages, Hkv, page, D), dtype=torch.uint8, device=dev)
    scale = torch.empty((pages, Hkv, page // BLOCK), dtype=torch.uint8, device=dev)
    channel = torch.exp(0.5 * torch.randn((Hkv, 1, 1, D), device=dev, generator=g))
    step = max(1, (1 << 27) // (Hkv * D * page))
    for p in range(0, pages, step):
        m = min(step, pages - p)
        x = torch.randn((m, Hkv, page // BLOCK, BLOCK, D), device=dev, generator=g) * channel
        e = torch.ceil(torch.log2(x.abs().amax((-2, -1), keepdim=True) / 448))
        codes[p:p + m] = (x * torch.exp2(-e)).clamp(-448, 448).to(torch.float8_e4m3fn) \
            .view(torch.uint8).view(m, Hkv, page, D)
        scale[p:p + m] = (e + 127).to(torch.uint8).view(m, Hkv, -1)
    return codes, scale


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    randn = lambda *s: torch.randn(s, device=dev, generator=g)  # noqa: E731
    if c["op"] == "gemv":
        x = randn(c["M"], c["K"])
        x = x * torch.where(torch.rand(x.shape, device=dev, generator=g) < 0.005, 20.0, 1.0)
        codes, sf, scale = _quantized_weight(c["N"], c["K"], g, dev)
        bias = (0.1 * randn(c["N"])).bfloat16() if c["bias"] else None
        return dict(c=c, x=x.bfloat16(), codes=codes, sf=sf, scale=scale, bias=bias)
    n, L = _lens(c)
    T, Hq, Hkv, D, page = sum(n), c["Hq"], c["Hkv"], c["D"], c["page"]
    cu = torch.tensor([0] + n, dtype=torch.int32).cumsum(0, dtype=torch.int32).to(dev)
    kv_len = torch.tensor(L, dtype=torch.int32, device=dev)
    most = max(-(-l // page) for l in L)
    table = torch.zeros((c["B"], max(1, most)), dtype=torch.int32)
    order = random.Random(seed)
    if c["op"] == "append":      # only the pages that the new tokens reach are there
        spans = [((l - m) // page, -(-l // page)) if m else (0, 0) for m, l in zip(n, L)]
    else:
        spans = [(0, -(-l // page)) for l in L]
    pages = sum(b - a for a, b in spans) + 3
    ids = list(range(pages))
    order.shuffle(ids)
    at = 0
    for b, (lo, hi) in enumerate(spans):
        table[b, lo:hi] = torch.tensor(ids[at:at + hi - lo], dtype=torch.int32)
        at += hi - lo
    k_cache, k_scale = _cache(pages, c, g, dev)
    v_cache, v_scale = _cache(pages, c, g, dev)
    s = dict(c=c, cu=cu, kv_len=kv_len, table=table.to(dev), k_cache=k_cache, k_scale=k_scale,
             v_cache=v_cache, v_scale=v_scale)
    if c["op"] == "append":      # q, k and v as one projection leaves them: side by side
        qkv = randn(T, Hq + 2 * Hkv, D).mul_(torch.exp(0.5 * randn(1, Hq + 2 * Hkv, D))).bfloat16()
        j = torch.arange(c["rot"] // 2, dtype=torch.float64)
        inv = (c["theta"] ** (-2 * j / c["rot"])).float().to(dev)
        held = {x: s[x].view(torch.float8_e4m3fn if "cache" in x else torch.float8_e8m0fnu)
                for x in ("k_cache", "v_cache", "k_scale", "v_scale")}   # the values they stand for
        return dict(s, held=held, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], inv_freq=inv)
    return dict(s, q=(2 * randn(T, Hq, D)).bfloat16())


# ------------------------------------------------------------------ plain forms
def _plain_gemv(s):
    c = s["c"]
    values = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=s["x"].device)
    codes = s["codes"].int()
    w = values[torch.stack((codes & 15, codes >> 4), -1)].view(c["N"], -1, 16)
    sf = _linear_layout(s["sf"], c["N"], c["K"]).view(torch.float8_e4m3fn).float()
    w = (w * sf.unsqueeze(-1)).view(c["N"], c["K"])
    y = (s["x"].float() @ w.t()) * s["scale"]
    return (y if s["bias"] is None else y + s["bias"].float()).bfloat16()


def _rotate(x, cos, sin, rot, interleaved):
    """x [T, H, D] fp32; cos, sin [T, rot / 2]."""
    cos, sin = cos.unsqueeze(1), sin.unsqueeze(1)
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _store(x, s, cache, scale, unit):
    """x [T, Hkv, D] fp32 into the cache blocks that `unit` names."""
    c = s["c"]
    page_id, slot, token, fresh, kept = unit
    new = torch.where(fresh[..., None, None], x[token.clamp(0, x.shape[0] - 1)], 0.0)  # [U, 16, H, D]
    rows = (page_id[:, None], slot[:, None] * BLOCK + torch.arange(BLOCK, device=x.device))
    view = cache.view(torch.float8_e4m3fn)
    old = view.transpose(1, 2)[rows].float()                                            # [U, 16, H, D]
    has_old = kept.any(-1)
    old_e = torch.where(has_old[:, None], scale[page_id, :, slot].int(), 0)             # [U, H]
    amax = new.abs().amax((1, 3))
    mant, e = torch.frexp(amax)                                                          # mant in [1/2, 1)
    e = torch.where(mant > 0.875, e - 8, e - 9) + 127
    new_e = torch.maximum(torch.where(amax > 0, e, 0).clamp(0, 246), old_e)
    up = torch.exp2((127 - new_e).float())[:, None, :, None]
    down = torch.exp2((old_e - new_e).float())[:, None, :, None]
    value = torch.where(kept[..., None, None], old * down, new * up).clamp(-448, 448)
    keep = fresh | kept
    put = value.to(torch.float8_e4m3fn).view(torch.uint8)[keep]
    cache.transpose(1, 2)[rows[0].expand_as(keep)[keep], rows[1][keep]] = put
    live = fresh.any(-1)
    scale.transpose(1, 2)[page_id[live], slot[live]] = new_e[live].to(torch.uint8)


def _plain_append(s):
    c = s["c"]
    cu, L, dev = s["cu"].long(), s["kv_len"].long(), s["q"].device
    T, B, page = s["q"].shape[0], c["B"], c["page"]
    start = L - (cu[1:] - cu[:-1])
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cu, t, right=True) - 1
    angle = (start[b] + t - cu[b]).double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float() * c["rope_scale"], torch.sin(angle).float() * c["rope_scale"]
    q = _rotate(s["q"].float(), cos, sin, c["rot"], c["interleaved"]).bfloat16()
    k = _rotate(s["k"].float(), cos, sin, c["rot"], c["interleaved"])
    first = cu // BLOCK + 2 * torch.arange(B + 1, device=dev)      # room for each sequence's blocks
    u = torch.arange(T // BLOCK + 2 * B, device=dev)
    b = torch.searchsorted(first, u, right=True) - 1
    block = start[b] // BLOCK + u - first[b]
    pos = block[:, None] * BLOCK + torch.arange(BLOCK, device=dev)
    fresh = (pos >= start[b][:, None]) & (pos < L[b][:, None])
    kept = (pos < start[b][:, None]) & fresh.any(-1, keepdim=True)
    token = cu[b][:, None] + pos - start[b][:, None]
    at = (block * BLOCK // page).clamp(0, s["table"].shape[1] - 1)
    unit = (s["table"][b, at].long(), block * BLOCK % page // BLOCK, token, fresh, kept)
    _store(k, s, s["k_cache"], s["k_scale"], unit)
    _store(s["v"].float(), s, s["v_cache"], s["v_scale"], unit)
    return q


def _plain_attend(s):
    c = s["c"]
    B, n, Hkv, D, page = c["B"], c["new"], c["Hkv"], c["D"], c["page"]
    G, L = c["Hq"] // Hkv, s["kv_len"].long()
    table = s["table"].long()

    def values(cache, scale):                                       # [B, Hkv, tokens, D] fp32
        x = cache.view(torch.float8_e4m3fn)[table].float().view(B, -1, Hkv, page // BLOCK, BLOCK, D)
        x = x * torch.exp2(scale[table].float() - 127)[..., None, None]
        return x.permute(0, 2, 1, 3, 4, 5).reshape(B, Hkv, -1, D)

    q = s["q"].float().view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    score = (q @ values(s["k_cache"], s["k_scale"]).transpose(-1, -2)) * D ** -0.5
    pos = torch.arange(score.shape[-1], device=q.device)
    at = L[:, None] - n + torch.arange(n, device=q.device)          # [B, n]
    seen = pos <= at[..., None]
    if c["window"]:
        seen &= pos > at[..., None] - c["window"]
    seen = seen.repeat_interleave(G, 1)[:, None]                    # [B, 1, n * G, tokens]
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p @ values(s["v_cache"], s["v_scale"])) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).squeeze(-1)
    out = o.view(B, Hkv, n, G, D).permute(0, 2, 1, 3, 4).reshape(B * n, c["Hq"], D).bfloat16()
    return out, lse.view(B, Hkv, n, G).permute(0, 2, 1, 3).reshape(B * n, c["Hq"])


def run(state):
    s, c = state, state["c"]
    if own:
        import block_scaled_precision_act_b200 as bsp
    if c["op"] == "gemv":
        if own:
            return bsp.nvfp4_gemv(s["x"], s["codes"], s["sf"], s["scale"], bias=s["bias"])
        return _plain_gemv(s)
    if c["op"] == "append":
        if own:
            q = bsp.fp8kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"],
                                 s["v_scale"], s["table"], s["cu"], s["kv_len"], q=s["q"],
                                 inv_freq=s["inv_freq"], interleaved=c["interleaved"],
                                 rope_scale=c["rope_scale"])
        else:
            q = _plain_append(s)
        return dict(s["held"], q=q)
    if own:
        return bsp.fp8kv_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                   s["table"], s["cu"], s["kv_len"], window=c["window"],
                                   return_lse=True)
    return _plain_attend(s)


# ------------------------------------------------------------------ 64 bits
def _e4m3_64(x):
    """Nearest E4M3 value, ties to even, of doubles within +-448."""
    _, e = torch.frexp(x.abs())
    step = torch.exp2((e.double() - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _exact_gemv(s):
    c = s["c"]
    N, K = c["N"], c["K"]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")
    rows, x, out = max(1, (1 << 28) // K), s["x"].double(), []
    r = torch.arange(N, device="cuda")
    for a in range(0, N, rows):
        n = r[a:a + rows, None]
        byte = s["codes"][a:a + rows].long()
        w = torch.empty((byte.shape[0], K), dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = table[byte % 16], table[byte // 16]
        kb = torch.arange(K // 16, device="cuda")[None]
        at = ((n // 128) * (K // 64) + kb // 4) * 512 + n % 32 * 16 + n // 32 % 4 * 4 + kb % 4
        w *= s["sf"].view(torch.float8_e4m3fn)[at].double().repeat_interleave(16, 1)
        out.append(x @ w.t())
    y = torch.cat(out, 1) * s["scale"].double()
    return y if s["bias"] is None else y + s["bias"].double()


def _exact_append(s):
    c = s["c"]
    n, L = _lens(c)
    rot, page, at = c["rot"], c["page"], 0
    q_out, table = s["q"].double(), s["table"].tolist()
    caches = {x: (s[x + "_cache"].view(torch.float8_e4m3fn).double(), s[x + "_scale"].double())
              for x in "kv"}
    for b, (m, l) in enumerate(zip(n, L)):
        if m == 0:
            continue
        pos = torch.arange(l - m, l, dtype=torch.float64, device="cuda")
        turn = torch.polar(torch.full((), c["rope_scale"], dtype=torch.float64, device="cuda"),
                           pos[:, None] * s["inv_freq"].double())[:, None]

        def rotated(x):
            x = x.double().clone()
            i = torch.arange(rot // 2, device="cuda")
            i, j = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rot // 2)
            z = torch.complex(x[..., i], x[..., j]) * turn
            x[..., i], x[..., j] = z.real, z.imag
            return x

        q_out[at:at + m] = rotated(s["q"][at:at + m])
        for name, x in (("k", rotated(s["k"][at:at + m])), ("v", s["v"][at:at + m].double())):
            cache, scale = caches[name]
            lo, hi = (l - m) // BLOCK, (l - 1) // BLOCK + 1
            span = torch.zeros(((hi - lo) * BLOCK,) + x.shape[1:], dtype=torch.float64, device="cuda")
            first = l - m - lo * BLOCK
            span[first:first + m] = x
            amax = span.view(hi - lo, BLOCK, c["Hkv"], c["D"]).abs().amax((1, 3))
            part, e = torch.frexp(amax / 448)              # part in [1/2, 1): e = ceil(log2), exactly
            e = torch.where(part > 0.5, e, e - 1).double()
            e = torch.where(amax > 0, e, -127.0).clamp(-127, 119) + 127
            blocks = torch.arange(lo, hi)
            ids = torch.tensor([table[b][k * BLOCK // page] for k in blocks.tolist()], device="cuda")
            slot = (blocks * BLOCK % page // BLOCK).to("cuda")
            if first:
                e[0] = torch.maximum(e[0], scale[ids[0], :, slot[0]])
                old = cache[ids[0], :, slot[0] * BLOCK:slot[0] * BLOCK + first].transpose(0, 1)
                span[:first] = old * torch.exp2(scale[ids[0], :, slot[0]] - 127)[None, :, None]
            code = _e4m3_64((span.view(hi - lo, BLOCK, c["Hkv"], c["D"])
                             * torch.exp2(127 - e)[:, None, :, None]).clamp(-448, 448))
            code = code.view(-1, c["Hkv"], c["D"])[:first + m]
            p = torch.arange(first + m, device="cuda")
            cache[ids[p // BLOCK], :, slot[p // BLOCK] * BLOCK + p % BLOCK] = code
            scale[ids, :, slot] = e
        at += m
    return dict(q=q_out, k_cache=caches["k"][0], v_cache=caches["v"][0],
                k_scale=torch.exp2(caches["k"][1] - 127), v_scale=torch.exp2(caches["v"][1] - 127))


def _exact_attend(s):
    c = s["c"]
    n, L = _lens(c)
    m, Hkv, G, page = c["new"], c["Hkv"], c["Hq"] // c["Hkv"], c["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, l in enumerate(L):
        ids = s["table"][b, :-(-l // page)].long()

        def values(cache, scale):
            x = cache[ids].view(torch.float8_e4m3fn).double()
            x = x * torch.exp2(scale[ids].double() - 127).repeat_interleave(BLOCK, 2)[..., None]
            return x.transpose(0, 1).reshape(Hkv, -1, c["D"])[:, :l]

        k, v = values(s["k_cache"], s["k_scale"]), values(s["v_cache"], s["v_scale"])
        for i in range(m):
            end = l - m + i + 1
            lo = max(0, end - c["window"]) if c["window"] else 0
            if end <= lo:
                continue
            q = s["q"][b * m + i].double().view(Hkv, G, -1)
            z = torch.einsum("hgd,htd->hgt", q, k[:, lo:end]) / math.sqrt(c["D"])
            lse[b * m + i] = torch.logsumexp(z, -1).view(-1)
            out[b * m + i] = torch.einsum("hgt,htd->hgd", torch.softmax(z, -1), v[:, lo:end]) \
                .reshape(-1, c["D"])
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"gemv": _exact_gemv, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)
