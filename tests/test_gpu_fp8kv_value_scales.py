"""fp8kv_attention where the value blocks of a sequence differ in scale, and the scale bytes that
fp8kv_append does not make, against the 64-bit reference.

Bounds: those of test_gpu_fp8kv_attention.py, and what they leave out, a product p 2^e (weight times the
scale of its block) below f16's normal numbers.  The kernel holds p 2^e to half of f16's smallest step,
2^-25, times 2^(ref - 8), with ref at most 1 above log2 of the row's largest p 2^e: 2^-32 of that largest,
for each token, times the token's code."""
import math

import pytest
import torch

import block_scaled_precision_act_b200 as bsp
from kv_reference import BLOCK, E4M3, Batch, attention
from test_gpu_fp8kv_attention import call

pytestmark = pytest.mark.gpu


def check(b, out, lse, window=0, rows=None, sm=None):
    sm = b.D ** -0.5 if sm is None else sm
    want, wlse, mass, size = attention(b, sm, window)
    least = torch.zeros_like(want)                   # 2^-32 of the row's largest p 2^e, times sum |code|
    G = b.Hq // b.Hkv
    for s in range(b.B):
        L = b.lens[s]
        ids = b.table[s, :-(-L // b.page)].long()
        code = E4M3[b.v_cache[ids].long()].abs().transpose(0, 1).reshape(b.Hkv, -1, b.D)[:, :L]
        unit = torch.exp2(b.v_scale[ids].double() - 127).transpose(0, 1).reshape(b.Hkv, -1) \
            .repeat_interleave(BLOCK, 1)[:, :L]
        k = b.values("k", s, L)
        for i in range(b.n[s]):
            row, end = int(b.cu[s]) + i, L - b.n[s] + i + 1
            lo = max(0, end - window) if window else 0
            if end <= lo:
                continue
            z = torch.einsum("hgd,htd->hgt", b.q[row].double().view(b.Hkv, G, b.D), k[:, lo:end]) * sm
            top = (torch.softmax(z, -1) * unit[:, None, lo:end]).amax(-1)            # [Hkv, G]
            least[row] = (2.0 ** -32 * top[..., None] * code[:, lo:end].sum(1)[:, None]).reshape(b.Hq, b.D)
    L = max(b.lens)
    ds = (b.D / 16 + 20) * 2.0 ** -22 * size
    weight = 2 * (2.0 ** -11 + 2.0 ** -20 + ds)[..., None] + (L / 16 + 32) * 2.0 ** -22 + 2.0 ** -20
    # an output below bf16's normal numbers is off by half of its smallest step, 2^-133
    bound = want.abs() * 2.0 ** -8 + weight * mass + least + 2.0 ** -134
    rows = list(range(int(b.cu[-1]))) if rows is None else rows
    got = out.cpu().double()
    d = (got - want).abs()
    assert (d <= bound)[rows].all(), float((d / bound.clamp(min=1e-300))[rows].max())
    assert ((lse.cpu().double() - wlse).abs() <= ds + 2.0 ** -20 + 2.0 ** -22 * wlse.abs())[rows].all()


def tokens(b, s, lo, hi):
    """(page, slot) of tokens lo .. hi of a sequence."""
    return [b.where(s, t) for t in range(lo, hi)]


def repel(b, s, lo, hi, nats=200.0):
    """Keys of tokens lo .. hi against every row's q: weights of about e^-nats.  All q become ones."""
    b.q = torch.ones_like(b.q)
    for page, slot in tokens(b, s, lo, hi):
        b.k_cache[page, :, slot] = 0xB8              # -1, times the block's scale
        b.k_scale[page, :, slot // BLOCK] = 127 + round(math.log2(nats / b.D ** 0.5))


def raise_values(b, s, lo, hi, by):
    for page, slot in tokens(b, s, lo, hi):
        b.v_scale[page, :, slot // BLOCK] = 120 + by


def level(b, k=118, v=120):
    b.k_scale[:], b.v_scale[:] = k, v


@pytest.mark.parametrize("D,Hq,page", [(64, 4, 16), (128, 16, 64), (192, 16, 32), (256, 4, 16)])
@pytest.mark.parametrize("gap", [4, 10, 12, 16, 20, 24, 28, 32, 34, 40, 60, 100])
@pytest.mark.parametrize("at", [0, 48, 112])
def test_a_large_block_without_weight(D, Hq, page, gap, at):
    """One block of a tile is 2^gap larger than the others, and no row gives it any weight."""
    b = Batch([2], [280], Hq, 2 if Hq == 4 else 1, D, page, seed=gap + at)
    level(b)
    repel(b, 0, at, at + 16)
    raise_values(b, 0, at, at + 16, gap)
    check(b, *call(b))
    assert bsp.bsp_last_device_status() == 0


@pytest.mark.parametrize("nats", [7, 14, 21, 28])
@pytest.mark.parametrize("gap", [10, 20, 30, 40])
def test_a_large_block_of_little_weight(gap, nats):
    """Weights of 2^-10 to 2^-40 on a block 2^gap larger: it counts as much as the others, or more."""
    b = Batch([1, 2], [700, 150], 8, 2, 128, 64, seed=gap + nats)
    level(b)
    for s, lo in ((0, 320), (1, 0)):
        repel(b, s, lo, lo + 16, nats)
        raise_values(b, s, lo, lo + 16, gap)
    check(b, *call(b))


@pytest.mark.parametrize("gap", [20, 34, 60, 110])
@pytest.mark.parametrize("D,Hq", [(64, 2), (128, 8), (256, 4)])
def test_values_that_another_row_of_the_tile_sees(gap, D, Hq):
    """Blocks that only some rows of a tile see: in front of a window, and behind the causal edge."""
    b = Batch([6], [114], Hq, 2, D, 16, seed=gap)    # rows at 108 .. 113
    level(b)
    raise_values(b, 0, 112, 114, gap)                # seen by the last two rows
    check(b, *call(b))
    b = Batch([6], [130], Hq, 2, D, 16, seed=gap + 1)
    level(b)
    raise_values(b, 0, 64, 80, gap)                  # window 50: row at 124 + i sees 75 + i on
    check(b, *call(b, window=50), window=50)
    raise_values(b, 0, 64, 80, 0)
    raise_values(b, 0, 48, 64, gap)                  # window 62: from 63 + i on, the first row sees one
    check(b, *call(b, window=62), window=62)


@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("lens", [[640], [1500], [300, 1900, 129]])
def test_scales_that_rise_and_fall_from_block_to_block(order, lens):
    """Each block 2^3 larger (or smaller) than the one before, over the whole range of bytes."""
    b = Batch([1] * len(lens), lens, 8, 2, 64, 16, seed=sum(lens))
    b.k_scale[:] = 118
    for s, L in enumerate(lens):
        for i in range(-(-L // 16)):
            page, _ = b.where(s, 16 * i)
            b.v_scale[page] = (3 * i * order) % 240
    b.v_cache = (b.v_cache & 0x80) | (b.v_cache & 0x7F) % 56     # at most 1 in size
    check(b, *call(b))


def test_blocks_of_zeros():
    """A block of zeros has scale byte 0; most of the weight may lie on it."""
    b = Batch([2], [300], 8, 2, 128, 32, seed=5)
    level(b)
    repel(b, 0, 0, 128, 90)
    for page, slot in tokens(b, 0, 128, 256):
        b.v_cache[page, :, slot], b.v_scale[page, :, slot // BLOCK] = 0, 0
    check(b, *call(b))


@pytest.mark.parametrize("byte", [0, 1, 246, 247, 250, 254])
def test_every_finite_scale_byte(byte):
    """value = code * 2^(byte - 127) up to byte 254; only codes of at most 1, so that sums stay finite."""
    b = Batch([1, 3], [40, 300], 4, 2, 64, 16, seed=byte)
    b.k_scale[:], b.v_scale[:] = 118, byte
    b.v_cache = (b.v_cache & 0x80) | (b.v_cache & 0x7F) % 56
    check(b, *call(b))
    b = Batch([1, 3], [40, 300], 4, 2, 64, 16, seed=byte + 1)
    b.k_scale[:], b.v_scale[:] = byte, 120
    sm = 2.0 ** (120 - byte)
    if byte > 1:                                     # sm_scale is an fp32 number
        check(b, *call(b, sm_scale=sm), sm=sm)


def test_a_nan_scale_of_values_reaches_the_rows_that_see_it():
    for n, L, window, lo, sees in ((6, 114, 0, 112, [4, 5]), (6, 130, 62, 48, [0]), (2, 700, 0, 256, [0, 1])):
        b = Batch([n], [L], 4, 2, 64, 16, seed=L)
        page, slot = b.where(0, lo)
        b.v_scale[page, 1, slot // BLOCK] = 255
        out, lse = call(b, window=window)
        assert out[sees, 2:].isnan().all()
        assert int(out.isnan().sum()) == len(sees) * 2 * 64
        b.v_scale[page, 1, slot // BLOCK] = 0        # what the reference may not see
        b.v_cache[page, 1] = 0
        rest = [r for r in range(n) if r not in sees]
        if rest:
            check(b, out, lse, window, rest)
        want = attention(b, b.D ** -0.5, window)[1]
        assert torch.allclose(lse.cpu().double(), want, atol=1e-3, rtol=0)


def test_a_nan_scale_of_keys_reaches_the_rows_that_see_it():
    b = Batch([6], [114], 4, 2, 64, 16, seed=9)
    page, slot = b.where(0, 112)
    b.k_scale[page, 0, slot // BLOCK] = 255
    out, lse = call(b)
    assert out[4:, :2].isnan().all() and lse[4:, :2].isnan().all()
    assert int(out.isnan().sum()) == 2 * 2 * 64 and int(lse.isnan().sum()) == 4


@pytest.mark.parametrize("D,Hq", [(64, 4), (128, 16), (256, 4)])
@pytest.mark.parametrize("gap", [6, 12, 18, 22, 24, 26, 28, 30])
def test_elements_that_only_small_blocks_have(D, Hq, gap):
    """A block 2^gap larger has all of the weight that the others have, but its values are zero for every
    other d: there the small blocks make the result, with products of 2^-gap of the row's largest."""
    b = Batch([2], [300], Hq, 2 if Hq == 4 else 1, D, 16, seed=gap)
    level(b)
    raise_values(b, 0, 144, 160, gap)
    for page, slot in tokens(b, 0, 144, 160):
        b.v_cache[page, :, slot, ::2] = 0
    check(b, *call(b))


@pytest.mark.parametrize("D,Hq", [(64, 2), (128, 8), (192, 4)])
@pytest.mark.parametrize("bits", [8, 12, 14, 16, 18, 20, 22, 24, 26, 28])
def test_one_token_against_many(D, Hq, bits):
    """One token has 2^bits times the weight of each of 20000 others, whose values are not zero on
    average: what is cut off of each would add up."""
    L = 20000
    b = Batch([1], [L], Hq, 1, D, 64, seed=bits, spare=0)
    level(b)
    b.q = torch.ones_like(b.q)
    b.k_cache[:] = 0
    page, slot = b.where(0, 12345)
    b.k_cache[page, :, slot] = 0x38                  # 1, times 2^-8 and sm
    sm = bits * math.log(2) * 2.0 ** (127 - 118) / D
    b.v_cache = b.v_cache & 0x7F
    b.v_cache[page, :, slot, ::2] = 0                # for every other d the many make the result
    check(b, *call(b, sm_scale=sm), sm=sm)
