"""The cache operators over head widths, page sizes and groups that the other tests pass over, queries that
are not finite, a context of 131071 tokens, and calls that repeat themselves to the last bit."""
import math

import pytest
import torch

import block_scaled_precision_act_b200 as bsp
from kv_reference import Batch, attention
from test_gpu_fp8kv_append import call as append, check as check_append
from test_gpu_fp8kv_attention import NAMES, call, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [16, 32, 48, 144, 160, 176, 208, 224, 240])
@pytest.mark.parametrize("Hq,Hkv", [(3, 3), (10, 2)])
def test_head_widths(D, Hq, Hkv):
    b = Batch([2, 9, 0, 33], [150, 9, 40, 290], Hq, Hkv, D, 48, seed=D)
    rot = D // 32 * 16
    q, got = append(b, rot, D % 32 == 0)
    check_append(b, q, got, rot, D % 32 == 0)
    check(b, *call(b))
    assert bsp.bsp_last_device_status() == 0


@pytest.mark.parametrize("page", [16, 48, 80, 96, 112, 144, 240, 1040, 4096])
@pytest.mark.parametrize("window", [0, 77])
def test_page_sizes(page, window):
    b = Batch([1, 5, 20], [700, 129, 257], 8, 2, 64, page, seed=page, spare=1)
    q, got = append(b, 64)
    check_append(b, q, got, 64)
    check(b, *call(b, window=window), window=window)


@pytest.mark.parametrize("Hq,Hkv,n", [(64, 1, [1, 3]), (100, 1, [2, 1]), (96, 96, [1, 1]), (21, 7, [17, 1])])
def test_groups(Hq, Hkv, n):
    b = Batch(n, [210, 300], Hq, Hkv, 64, 32, seed=Hq)
    check(b, *call(b))


@pytest.mark.parametrize("D", [64, 256])
def test_queries_that_are_not_finite(D):
    """An infinity or a NaN in a head of a row gives NaN there; every other head and row keeps its value
    within the bounds.  (Not to the last bit: when the references of a tile's rows move, and so the
    numbers that a score is rounded next to, depends on all rows of the tile.  The bounds hold for any.)"""
    b = Batch([3, 1], [45, 300], 8, 2, D, 16, seed=D)
    clean, lse = call(b)
    finite = b.q.clone()
    b.q[1, 2, 5], b.q[1, 6, 0], b.q[3, 7, D - 1] = math.nan, math.inf, -math.inf
    out, lse2 = call(b)
    bad = torch.zeros((4, 8), dtype=torch.bool)
    bad[1, 2], bad[1, 6], bad[3, 7] = True, True, True
    assert out.cpu()[bad].isnan().all() and lse2.cpu()[bad].isnan().all()
    b.q = finite
    out[bad.cuda()], lse2[bad.cuda()] = clean[bad.cuda()], lse[bad.cuda()]
    check(b, out, lse2)


@pytest.mark.parametrize("D,Hq", [(64, 8), (256, 2)])
@pytest.mark.parametrize("power", [0, 8, 12, 16, 18, 20, 22, 24, 26, 30, 100])
def test_a_huge_element_of_q_against_zero_keys(D, Hq, power):
    """The scores come from the other elements, which are held to 2^-25 of the huge one: exact while that
    is below the last bit of all of them."""
    b = Batch([1, 2], [90, 300], Hq, 2, D, 16, seed=power)
    b.q = (torch.randint(128, 256, b.q.shape, generator=b.g) * torch.exp2(
        torch.randint(-9, -6, b.q.shape, generator=b.g))).bfloat16() * torch.sign(b.q)
    b.q[..., 3] = 2.0 ** power
    b.k_cache[..., 3] = 0
    b.v_cache[..., ::2] &= 0x7F
    out, lse = call(b)
    want, wlse, mass, size = attention(b, D ** -0.5, 0)
    # all others are at least 1/4: exact down to 2^-17 of the largest, off by 2^-25 of it below
    off = 0.0 if power <= 15 else 2.0 ** (power - 25)
    k1 = torch.zeros_like(size)                      # largest sum |k| that a row sees
    for s in range(2):
        k = b.values("k", s, b.lens[s]).abs().sum(-1).amax(-1).repeat_interleave(Hq // 2)
        k1[int(b.cu[s]):int(b.cu[s + 1])] = k
    ds = (D / 16 + 20) * 2.0 ** -22 * size + off * k1 * D ** -0.5
    if float(ds.max()) > 0.25:                       # nothing is left of the others
        assert out.isfinite().all()
        return
    assert ((lse.cpu().double() - wlse).abs() <= ds + 2.0 ** -20 + 2.0 ** -22 * wlse.abs()).all()
    weight = torch.expm1(2 * ds)[..., None] + 2 * (2.0 ** -11 + 2.0 ** -20) + (300 / 16 + 32) * 2.0 ** -22
    assert ((out.cpu().double() - want).abs() <= want.abs() * 2.0 ** -8 + weight * mass).all()


def test_a_long_context():
    b = Batch([1], [131071], 8, 1, 128, 64, seed=3)
    check(b, *call(b))


@pytest.mark.parametrize("n,lens,Hq,Hkv,D", [([1] * 40, [100 * i + 1 for i in range(40)], 32, 8, 128),
                                             ([4] * 6, [3000] * 6, 16, 16, 64), ([1], [20000], 16, 2, 256)])
def test_repeated_calls_give_the_same_bits(n, lens, Hq, Hkv, D):
    b = Batch(n, lens, Hq, Hkv, D, 64, seed=1)
    dev = b.to("cuda")
    q, args = b.q.cuda(), [dev[x] for x in NAMES]
    want = bsp.fp8kv_attention(q, *args, return_lse=True)
    for _ in range(50):
        got = bsp.fp8kv_attention(q, *args, return_lse=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("D,Hq,n,window", [(256, 4, 1, 0), (192, 16, 1, 0), (144, 2, 5, 0), (256, 16, 2, 300)])
def test_wide_heads_beside_other_traffic(D, Hq, n, window):
    """Heads of two pieces, whose tiles have two slots: the values of the last tile, whose masked tokens
    hold NaN, are cleared after those of the tile before are used.  Loads are made late by copies on
    another stream; the call gives the same bits each time."""
    lens = [129 + 61 * i for i in range(40)]
    b = Batch([n] * 40, lens, Hq, 2, D, 64, seed=D + n, spare=0)
    for s, L in enumerate(lens):
        for t in range(L, -(-L // 64) * 64):
            page, slot = b.where(s, t)
            b.k_cache[page, :, slot], b.v_cache[page, :, slot] = 0x7F, 0x7F
    dev = b.to("cuda")
    q, args = b.q.cuda(), [dev[x] for x in NAMES]
    want, lse = bsp.fp8kv_attention(q, *args, window=window, return_lse=True)
    check(b, want, lse, window=window)
    side = torch.cuda.Stream()
    big = torch.empty((2, 1 << 28), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(side):
            for _ in range(4):
                big[0].copy_(big[1])
        for _ in range(20):
            got = bsp.fp8kv_attention(q, *args, window=window)
            assert torch.equal(got, want)
    torch.cuda.synchronize()
