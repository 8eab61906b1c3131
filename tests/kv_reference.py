"""64-bit reference of the block-scaled 8-bit cache on the CPU, written from its definition:
E4M3 codes with one power-of-two scale for each block of 16 tokens and head."""
import math
import random

import torch

BLOCK = 16


def e4m3_values():
    """Value of each of the 256 codes (NaN for 0x7F / 0xFF)."""
    v = []
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append((-x if c & 128 else x) if c & 127 != 127 else math.nan)
    return torch.tensor(v, dtype=torch.float64)


E4M3 = e4m3_values()
_MAG = E4M3[:127]


def encode(x):
    """Nearest code of doubles, ties to the even code, saturating; NaN -> 0x7F."""
    a = x.abs().clamp(max=448.0)
    i = torch.bucketize(torch.nan_to_num(a), _MAG).clamp(max=126)
    lo = (i - 1).clamp(min=0)
    dl, dh = a - _MAG[lo], _MAG[i] - a
    c = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, i)
    c = torch.where(torch.isnan(x), 127, c)
    return (c + 128 * torch.signbit(x)).to(torch.uint8)


def scale_exp(amax):
    """ceil(log2(amax / 448)) + 127 within [0, 246]."""
    part, e = torch.frexp(torch.clamp(amax, max=2.0 ** 200) / 448)
    e = torch.where(part > 0.5, e, e - 1) + 127
    return torch.where(amax > 0, e, 0).clamp(0, 246)


class Batch:
    """A ragged batch over a paged cache, all on the CPU."""

    def __init__(self, n, lens, Hq, Hkv, D, page, seed, spare=3, pad_rows=0):
        r = random.Random(seed)
        self.g = torch.Generator().manual_seed(seed)
        self.n, self.lens, self.Hq, self.Hkv, self.D, self.page = n, lens, Hq, Hkv, D, page
        self.B, self.T = len(n), sum(n) + pad_rows
        need = [max(1, -(-l // page)) for l in lens]
        ids = list(range(sum(need) + spare))
        r.shuffle(ids)
        self.pages = len(ids)
        self.table = torch.full((self.B, max(need)), -7, dtype=torch.int32)
        for b, m in enumerate(need):
            self.table[b, :m] = torch.tensor([ids.pop() for _ in range(m)], dtype=torch.int32)
        self.unused = ids
        self.cu = torch.tensor([0] + list(n)).cumsum(0).to(torch.int32)
        self.kv_len = torch.tensor(lens, dtype=torch.int32)
        shape = (self.pages, Hkv, page, D)
        self.k_cache, self.k_scale = self._pool(shape)
        self.v_cache, self.v_scale = self._pool(shape)
        self.q, self.k, self.v = self.randn(self.T, Hq, D), self.randn(self.T, Hkv, D), \
            self.randn(self.T, Hkv, D)

    def randn(self, *s):
        size = torch.exp(0.7 * torch.randn(s[-1], generator=self.g))
        return (torch.randn(s, generator=self.g) * size).bfloat16()

    def _pool(self, shape):
        x = torch.randn(shape, generator=self.g) * 90
        codes = encode(x.double())
        s = torch.randint(116, 122, shape[:2] + (shape[2] // BLOCK,), generator=self.g)
        return codes, s.to(torch.uint8)

    def where(self, b, t):
        """(page, slot) of token t of sequence b."""
        return int(self.table[b, t // self.page]), t % self.page

    def values(self, which, b, length):
        """[Hkv, length, D] doubles of a sequence's cached keys ("k") or values ("v")."""
        codes = self.k_cache if which == "k" else self.v_cache
        scale = self.k_scale if which == "k" else self.v_scale
        ids = self.table[b, :-(-length // self.page)].long()
        x = E4M3[codes[ids].long()] * torch.exp2(scale[ids].double() - 127) \
            .repeat_interleave(BLOCK, 2)[..., None]
        return x.transpose(0, 1).reshape(self.Hkv, -1, self.D)[:, :length]

    def to(self, dev):
        """The arguments that both calls share, on a device."""
        return dict(k_cache=self.k_cache.to(dev), v_cache=self.v_cache.to(dev),
                    k_scale=self.k_scale.to(dev), v_scale=self.v_scale.to(dev),
                    block_table=self.table.to(dev), cu_new=self.cu.to(dev),
                    kv_len=self.kv_len.to(dev))


def rotate(x, pos, inv_freq, interleaved, rope_scale):
    """x [n, H, D] -> doubles, the first 2 * len(inv_freq) elements of each head rotated."""
    x = x.double().clone()
    if inv_freq is None:
        return x
    half = inv_freq.numel()
    a = pos.double()[:, None] * inv_freq.double()
    cos, sin = (rope_scale * torch.cos(a))[:, None], (rope_scale * torch.sin(a))[:, None]
    i = torch.arange(half)
    i, j = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    x1, x2 = x[..., i], x[..., j]
    x[..., i], x[..., j] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    return x


def attention(batch, sm_scale, window):
    """(out, lse, sum p|v|, largest sum |q||k|) of every row, in doubles."""
    T, Hq, D = batch.q.shape
    G = Hq // batch.Hkv
    out = torch.zeros((T, Hq, D), dtype=torch.float64)
    mass = torch.zeros_like(out)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    size = torch.zeros((T, Hq), dtype=torch.float64)
    for b in range(batch.B):
        n, length = batch.n[b], batch.lens[b]
        k, v = batch.values("k", b, max(0, length)), batch.values("v", b, max(0, length))
        for i in range(n):
            row, end = int(batch.cu[b]) + i, length - n + i + 1
            lo = max(0, end - window) if window else 0
            if end <= lo:
                continue
            q = batch.q[row].double().view(batch.Hkv, G, D)
            z = torch.einsum("hgd,htd->hgt", q, k[:, lo:end]) * sm_scale
            p = torch.softmax(z, -1)
            out[row] = torch.einsum("hgt,htd->hgd", p, v[:, lo:end]).reshape(Hq, D)
            mass[row] = torch.einsum("hgt,htd->hgd", p, v[:, lo:end].abs()).reshape(Hq, D)
            lse[row] = torch.logsumexp(z, -1).reshape(Hq)
            size[row] = (torch.einsum("hgd,htd->hgt", q.abs(), k[:, lo:end].abs()).amax(-1)
                         * abs(sm_scale)).reshape(Hq)
    return out, lse, mass, size
