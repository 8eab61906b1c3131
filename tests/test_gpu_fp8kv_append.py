"""fp8kv_append on the GPU against the 64-bit reference.

Bounds.  Unrotated values are exact in fp32, so their codes and scales must be equal.  A rotated
value carries the angle's rounding to fp32 (|r| <= pi: 2^-23), sincosf (2 ulp: 2^-22), the
rope_scale product, two products and one sum (4 * 2^-24): within DELTA = 2^-20 of |x1| + |x2|.
q_out adds one bf16 rounding (half a step, 2^-8 of the value).  A code is within half an E4M3
step (2^-4 of the value, or 2^-10 of the scale where subnormal) of x / scale, plus DELTA."""
import math

import pytest
import torch

import block_scaled_precision_act_b200 as bsp
from kv_reference import BLOCK, E4M3, Batch, encode, rotate, scale_exp

pytestmark = pytest.mark.gpu
DELTA = 2.0 ** -20


def inv_freq(rot, theta=10000.0):
    return (theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float() if rot else None


def call(b, rot, interleaved=False, rope_scale=1.0, q=True, **kw):
    dev = b.to("cuda")
    f = inv_freq(rot)
    q_out = bsp.fp8kv_append(b.k.cuda(), b.v.cuda(), dev["k_cache"], dev["v_cache"],
                             dev["k_scale"], dev["v_scale"], dev["block_table"], dev["cu_new"],
                             dev["kv_len"], q=b.q.cuda() if q else None,
                             inv_freq=None if f is None else f.cuda(), interleaved=interleaved,
                             rope_scale=rope_scale, **kw)
    torch.cuda.synchronize()
    return q_out, {k: v.cpu() for k, v in dev.items()}


def check(b, q_out, got, rot, interleaved=False, rope_scale=1.0):
    f = inv_freq(rot)
    touched = {}
    for name, x, before, scale0 in (("k", b.k, b.k_cache, b.k_scale),
                                    ("v", b.v, b.v_cache, b.v_scale)):
        codes, scale = got[name + "_cache"], got[name + "_scale"]
        same_c, same_s = torch.ones(codes.shape, dtype=torch.bool), torch.ones(scale.shape,
                                                                              dtype=torch.bool)
        for s in range(b.B):
            n, L = b.n[s], b.lens[s]
            if n == 0 or L < n:
                continue
            rows, pos = slice(int(b.cu[s]), int(b.cu[s]) + n), torch.arange(L - n, L)
            exact = x[rows].double()
            slack = torch.zeros_like(exact)
            if name == "k" and f is not None:
                exact = rotate(x[rows], pos, f, interleaved, rope_scale)
                slack = DELTA * rope_scale * (torch.ones(1) * x[rows].double().abs()
                                              .amax(-1, keepdim=True) * 2).expand_as(exact)
            for blk in range((L - n) // BLOCK, (L - 1) // BLOCK + 1):
                page, slot = b.where(s, blk * BLOCK)
                at = slot // BLOCK
                lo, hi = max(0, L - n - blk * BLOCK), min(BLOCK, L - blk * BLOCK)
                new = slice(blk * BLOCK + lo - (L - n), blk * BLOCK + hi - (L - n))
                amax = torch.nan_to_num(exact[new].abs(), nan=0.0).amax((0, 2))      # [Hkv]
                least, most = scale_exp(amax * (1 - 2 * DELTA)), scale_exp(amax * (1 + 2 * DELTA))
                if name == "v" or f is None:
                    least = most = scale_exp(amax)
                old = scale0[page, :, at].long() if lo else torch.zeros(b.Hkv, dtype=torch.long)
                e = scale[page, :, at].long()
                assert ((e >= torch.maximum(least, old)) & (e <= torch.maximum(most, old))).all()
                unit = torch.exp2(e.double() - 127)[None, :, None]
                code = codes[page, :, slot + lo:slot + hi].transpose(0, 1)           # [t, H, D]
                want = exact[new] / unit
                if name == "v" or f is None:
                    assert torch.equal(code, encode(want))
                else:
                    d = (E4M3[code.long()] - want.clamp(-448, 448)).abs()
                    half = torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10).double())
                    bad = d > half + slack[new] / unit
                    assert not (bad & ~torch.isnan(want)).any()
                    assert torch.equal(torch.isnan(E4M3[code.long()]), torch.isnan(want))
                if lo:                                                               # older codes
                    kept = E4M3[before[page, :, slot:slot + lo].long()]
                    moved = kept * torch.exp2((old - e).double())[:, None, None]
                    assert torch.equal(codes[page, :, slot:slot + lo], encode(moved))
                same_c[page, :, slot:slot + hi] = False
                same_s[page, :, at] = False
        assert torch.equal(codes[same_c], before[same_c])
        assert torch.equal(scale[same_s], scale0[same_s])
        touched[name] = int((~same_s).sum())
    if q_out is not None:
        q = q_out.cpu().double()
        for s in range(b.B):
            n, L = b.n[s], b.lens[s]
            rows = slice(int(b.cu[s]), int(b.cu[s]) + n)
            if n == 0 or L < n:
                continue
            exact = rotate(b.q[rows], torch.arange(L - n, L), f, interleaved, rope_scale)
            slack = 2 * DELTA * rope_scale * b.q[rows].double().abs().amax(-1, keepdim=True)
            assert ((q[rows] - exact).abs() <= exact.abs() * 2.0 ** -8 + slack).all()
    return touched


SHAPES = [
    # new tokens, lengths, Hq, Hkv, D, page, rot, interleaved, rope_scale
    ([1], [1], 1, 1, 16, 16, 16, False, 1.0),
    ([1], [16], 4, 4, 64, 16, 64, True, 1.0),
    ([1], [17], 8, 1, 128, 64, 128, False, 1.0),
    ([1, 1, 1], [1004, 15, 33], 8, 2, 128, 64, 128, False, 1.0),
    ([0, 5, 0, 31, 1, 0], [7, 5, 0, 100, 49, 16], 6, 3, 80, 48, 32, False, 1.25),
    ([40, 17], [40, 1000], 4, 4, 256, 32, 256, True, 1.0),
    ([33], [65], 2, 2, 96, 128, 0, False, 1.0),
    ([16, 16, 15], [32, 31, 15], 5, 5, 192, 16, 64, True, 1.0),
    ([1] * 70, list(range(1, 71)), 4, 1, 112, 16, 112, False, 0.9),
    ([3] * 300, [3 + 7 * i % 90 for i in range(300)], 2, 1, 64, 32, 32, False, 1.0),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"D{s[4]}-B{len(s[0])}-T{sum(s[0])}")
def test_codes_scales_and_q(shape):
    n, lens, Hq, Hkv, D, page, rot, inter, rs = shape
    b = Batch(n, lens, Hq, Hkv, D, page, seed=sum(lens) + D)
    q_out, got = call(b, rot, inter, rs)
    assert bsp.bsp_last_device_status() == 0
    touched = check(b, q_out, got, rot, inter, rs)
    assert touched["k"] == touched["v"] > 0


def test_far_positions():
    """A position near 2^20 times an fp32 frequency: the angle needs 64 bits.  The table's row
    names only the page that is reached; the rest stays invalid."""
    L, page = 1_000_003, 64
    b = Batch([3], [3], 4, 2, 128, page, seed=5)
    page_id = int(b.table[0, 0])
    table = torch.full((1, L // page + 1), -1, dtype=torch.int32)
    table[0, (L - 3) // page] = page_id
    b.table, b.lens, b.kv_len = table, [L], torch.tensor([L], dtype=torch.int32)
    assert (L - 3) // page == (L - 1) // page
    q_out, got = call(b, 128)
    assert bsp.bsp_last_device_status() == 0
    check(b, q_out, got, 128)


@pytest.mark.parametrize("rise", [0, 1, 5, 40, 300])
def test_raising_a_block_scale_moves_its_codes(rise):
    """Nine tokens are there at scale 2^-7 .. 2^-5; two more need `rise` more bits (or fewer)."""
    b = Batch([2], [11], 2, 2, 64, 16, seed=rise)
    b.v = (b.v.float() * 2.0 ** min(rise, 100)).bfloat16() if rise else b.v * 0
    if rise == 300:                                  # infinities saturate, and raise to the top
        b.v[1, 1, 3], b.v[0, 0, 2] = math.inf, -math.inf
    _, got = call(b, 0, q=False)
    check(b, None, got, 0)
    if rise == 300:
        assert (got["v_scale"][int(b.table[0, 0])] == 246).all()


def test_nan_stays_with_its_element():
    b = Batch([3], [20], 2, 2, 64, 32, seed=9)
    b.v[1, 0, 7], b.k[0, 1, 5] = math.nan, math.nan
    _, got = call(b, 0, q=False)
    check(b, None, got, 0)
    page = int(b.table[0, 0])
    assert int((E4M3[got["v_cache"][page].long()].isnan()).sum()) == 1


def test_rows_behind_the_last_sequence_are_left():
    b = Batch([2, 1], [18, 5], 4, 2, 64, 16, seed=3, pad_rows=5)
    q_out = torch.full((b.T, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    q, got = call(b, 64, q_out=q_out)
    check(b, q, got, 64)
    assert (q_out[3:] == 7.0).all()


def test_packed_projection_and_in_place_q():
    """q, k and v as slices of one projection's output give what contiguous ones give; q_out may
    be q."""
    b = Batch([9, 4], [30, 4], 8, 2, 128, 32, seed=4)
    q1, got1 = call(b, 128)
    qkv = torch.cat((b.q, b.k, b.v), 1).cuda()
    dev = b.to("cuda")
    args = [dev[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale", "block_table", "cu_new",
                             "kv_len")]
    f = inv_freq(128).cuda()
    q2 = bsp.fp8kv_append(qkv[:, 8:10], qkv[:, 10:], *args, q=qkv[:, :8], inv_freq=f)
    assert torch.equal(q1, q2)
    for x in ("k_cache", "v_cache", "k_scale", "v_scale"):
        assert torch.equal(dev[x].cpu(), got1[x])
    q3 = b.q.cuda()
    bsp.fp8kv_append(b.k.cuda(), b.v.cuda(), *args, q=q3, q_out=q3, inv_freq=f)
    assert torch.equal(q1, q3)


def test_appending_again_changes_nothing():
    b = Batch([5, 1], [21, 40], 4, 2, 64, 16, seed=6)
    _, once = call(b, 32)
    b2 = Batch([5, 1], [21, 40], 4, 2, 64, 16, seed=6)
    for x in ("k_cache", "v_cache", "k_scale", "v_scale"):
        setattr(b2, x, once[x])
    _, twice = call(b2, 32)
    for x in ("k_cache", "v_cache", "k_scale", "v_scale"):
        assert torch.equal(once[x], twice[x])


def test_pages_outside_the_pool_are_not_touched():
    b = Batch([4, 4], [20, 20], 2, 2, 64, 16, seed=8)
    good = b.table.clone()
    b.table[0, 1] = b.pages                         # one past the end
    _, got = call(b, 0, q=False)
    assert bsp.bsp_last_device_status() == -1 and bsp.bsp_last_device_status() == 0
    b.table[0, 1] = -1
    _, got2 = call(b, 0, q=False)
    assert bsp.bsp_last_device_status() == -1
    page = int(good[0, 1])
    for g in (got, got2):
        assert torch.equal(g["k_cache"][page], b.k_cache[page])
        other = int(good[1, 1])
        assert not torch.equal(g["k_cache"][other], b.k_cache[other])


def test_malformed_batches_stay_inside():
    """Rows outside [0, T), descending cu_new, lengths below the new tokens or past the table:
    nothing outside the arrays is touched, and the length below its tokens is reported."""
    b = Batch([4, 4], [20, 20], 2, 2, 64, 16, seed=8)
    for cu, lens in (([0, 400, 9], [20, 20]), ([5, 2, -3], [20, 20]), ([0, 4, 8], [3, -9]),
                     ([0, 4, 8], [2 ** 31 - 1, 20])):
        b.cu, b.kv_len = torch.tensor(cu, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32)
        call(b, 64)
        bsp.bsp_last_device_status()
    b.cu, b.kv_len = torch.tensor([0, 4, 8], dtype=torch.int32), torch.tensor([3, 20],
                                                                            dtype=torch.int32)
    _, got = call(b, 0, q=False)
    assert bsp.bsp_last_device_status() == -1
    assert torch.equal(got["k_cache"][int(b.table[0, 0])], b.k_cache[int(b.table[0, 0])])


def test_offsets_past_32_bits():
    page, Hkv, D = 64, 8, 128
    pages = (1 << 32) // (page * Hkv * D) + 5
    k = torch.zeros((pages, Hkv, page, D), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    sc = [torch.zeros((pages, Hkv, page // 16), dtype=torch.uint8, device="cuda") for _ in "kv"]
    b = Batch([3], [19], 8, Hkv, D, page, seed=2)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    bsp.fp8kv_append(b.k.cuda(), b.v.cuda(), k, v, *sc, table, b.cu.cuda(), b.kv_len.cuda())
    torch.cuda.synchronize()
    e = scale_exp(b.v.double().abs().amax((0, 2)))
    assert torch.equal(sc[1][pages - 1, :, 1].cpu().long(), e)
    want = encode(b.v.double() / torch.exp2(e.double() - 127)[None, :, None]).transpose(0, 1)
    assert torch.equal(v[pages - 1, :, 16:19].cpu(), want)
    assert int((v != 0).sum()) == int((want != 0).sum())


def test_other_stream_and_replayed_graph():
    b = Batch([1, 2], [30, 18], 4, 2, 64, 16, seed=12)
    q0, got = call(b, 64)
    dev = b.to("cuda")
    k, v, q, f = b.k.cuda(), b.v.cuda(), b.q.cuda(), inv_freq(64).cuda()
    args = [dev[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale", "block_table", "cu_new",
                             "kv_len")]
    saved = [a.clone() for a in args[:4]]
    q_out = torch.empty_like(q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    bsp.fp8kv_append(k, v, *args, q=q, q_out=q_out, inv_freq=f, stream=side)
    side.synchronize()
    assert torch.equal(q_out, q0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bsp.fp8kv_append(k, v, *args, q=q, q_out=q_out, inv_freq=f)
    for a, s in zip(args[:4], saved):
        a.copy_(s)
    q_out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q_out, q0)
    for x, a in zip(("k_cache", "v_cache", "k_scale", "v_scale"), args):
        assert torch.equal(a.cpu(), got[x])


def test_lengths_past_the_table_store_nothing():
    b = Batch([2, 3], [20, 30], 4, 2, 64, 16, seed=21)
    b.kv_len[0] = b.table.shape[1] * 16 + 1
    _, got = call(b, 64)
    assert bsp.bsp_last_device_status() == -1 and bsp.bsp_last_device_status() == 0
    for page in b.table[0, :2].tolist():
        assert torch.equal(got["k_cache"][page], b.k_cache[page])
        assert torch.equal(got["v_scale"][page], b.v_scale[page])
    last = int(b.table[1, 1])
    assert not torch.equal(got["k_cache"][last], b.k_cache[last])
