"""fp8kv_attention on the GPU against the 64-bit reference.

Bounds.  A score is a sum of D exact products in fp32: chains of at most D / 16 + 16 additions,
each off by at most 2^-22 of sum |q||k| (a tensor core may cut instead of round), times
sm_scale; the scale products add 2^-22 more, and its difference to a maximum of at most that
size another 2^-23: ds = (D / 16 + 20) 2^-22 max_t sum|q||k| sm_scale, the relative error of a
weight before exp's own 2^-20.  A weight is rounded to f16: 2^-11.  The sums over L tokens add
(L / 16 + 32) 2^-22 of sum p|v|, the joins of parts 2^-20, and the output one bf16 rounding, 2^-8."""
import math

import pytest
import torch

import block_scaled_precision_act_b200 as bsp
from kv_reference import Batch, attention

pytestmark = pytest.mark.gpu
NAMES = ("k_cache", "v_cache", "k_scale", "v_scale", "block_table", "cu_new", "kv_len")


def call(b, sm_scale=None, window=0, **kw):
    dev = b.to("cuda")
    out, lse = bsp.fp8kv_attention(b.q.cuda(), *[dev[x] for x in NAMES], sm_scale=sm_scale,
                                   window=window, return_lse=True, **kw)
    torch.cuda.synchronize()
    return out, lse


def check(b, out, lse, sm_scale=None, window=0, rows=None):
    D = b.D
    sm = D ** -0.5 if sm_scale is None else sm_scale
    want, wlse, mass, size = attention(b, sm, window)
    rows = slice(0, int(b.cu[-1])) if rows is None else rows
    L = max(1, max(b.lens))
    ds = (D / 16 + 20) * 2.0 ** -22 * size
    weight = 2 * (2.0 ** -11 + 2.0 ** -20 + ds)[..., None] + (L / 16 + 32) * 2.0 ** -22 + 2.0 ** -20
    bound = want.abs() * 2.0 ** -8 + weight * mass
    got = out.cpu().double()
    assert torch.equal(got[rows].isnan(), want[rows].isnan())
    ok = ((got - want).abs() <= bound) | want.isnan()
    assert ok[rows].all(), float(((got - want).abs() / bound.clamp(min=1e-30))[rows].nan_to_num().max())
    empty = wlse == -math.inf
    gl = lse.cpu().double()
    assert torch.equal(gl[rows] == -math.inf, empty[rows])
    assert (got[rows][empty[rows]] == 0).all()
    d = (gl - wlse).abs() <= ds + 2.0 ** -20 + 2.0 ** -22 * wlse.abs()
    assert (d | empty | wlse.isnan())[rows].all()


SHAPES = [
    # new tokens, lengths, Hq, Hkv, D, page, window
    ([1], [1], 1, 1, 16, 16, 0),
    ([1], [16], 1, 1, 64, 16, 0),
    ([1], [17], 8, 1, 128, 64, 0),
    ([1], [515], 32, 8, 128, 64, 0),
    ([1, 1, 1, 1], [1, 63, 64, 65], 6, 2, 64, 32, 0),
    ([4, 4], [100, 4], 4, 4, 64, 16, 0),
    ([4, 0, 1, 7], [90, 33, 1200, 7], 12, 4, 80, 48, 0),
    ([3, 5], [300, 41], 8, 2, 96, 32, 50),
    ([1, 2], [700, 33], 14, 2, 192, 64, 0),
    ([1, 3], [130, 257], 4, 2, 256, 16, 0),
    ([8], [200], 16, 1, 128, 64, 0),            # 128 rows: eight tiles of one head
    ([2], [150], 34, 2, 32, 16, 17),            # a group of 17 heads
    ([1], [40], 3, 3, 112, 16, 1),              # a window of the row itself
    ([64], [64], 2, 1, 64, 16, 0),              # a whole prompt
    ([1] * 33, [13 * i + 1 for i in range(33)], 8, 2, 128, 16, 0),
    ([1, 1], [3000, 5], 8, 8, 128, 128, 2999),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"D{s[4]}-B{len(s[0])}-L{max(s[1])}-w{s[6]}")
def test_against_64_bits(shape):
    n, lens, Hq, Hkv, D, page, window = shape
    b = Batch(n, lens, Hq, Hkv, D, page, seed=sum(lens) + D)
    out, lse = call(b, window=window)
    assert bsp.bsp_last_device_status() == 0
    check(b, out, lse, window=window)


@pytest.mark.parametrize("sm_scale", [0.0, 1.0, -0.3])
def test_softmax_scales(sm_scale):
    b = Batch([2, 1], [90, 300], 8, 2, 64, 16, seed=1)
    check(b, *call(b, sm_scale=sm_scale), sm_scale=sm_scale)


def test_rows_that_see_nothing():
    """Lengths of zero, and fewer tokens than rows: the first rows see nothing."""
    b = Batch([2, 3, 1], [0, 1, 5], 4, 2, 64, 16, seed=2)
    out, lse = call(b)
    check(b, out, lse)
    assert (out[:4] == 0).all() and (lse[:4] == -math.inf).all()


def test_masked_places_hold_anything():
    """NaN codes, NaN scales and stale bytes behind the end, before a window, and in a
    neighbouring row's token: none reaches a row that does not see it."""
    b = Batch([3, 1], [45, 70], 8, 2, 64, 32, seed=3)
    clean = call(b, window=20)
    for s, L in ((0, 45), (1, 70)):
        for t in list(range(L, -(-L // 32) * 32)) + list(range(0, L - b.n[s] - 19)):
            page, slot = b.where(s, t)
            b.k_cache[page, :, slot], b.v_cache[page, :, slot] = 0x7F, 0xFF
        page, slot = b.where(s, 0)
        b.k_scale[page, :, 0], b.v_scale[page, :, 0] = 255, 255
    for x in b.unused:
        b.k_cache[x], b.v_cache[x], b.k_scale[x], b.v_scale[x] = 0x7F, 0x7F, 255, 255
    dirty = call(b, window=20)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


def test_nan_reaches_exactly_the_rows_that_see_it():
    b = Batch([4], [40], 4, 2, 64, 16, seed=4)
    page, slot = b.where(0, 38)                     # seen by the last two rows
    b.v_cache[page, 1, slot, 5] = 0x7F
    out, lse = call(b)
    check(b, out, lse)
    assert int(out.isnan().sum()) == 2 * 2          # two rows, the two heads of key head 1
    b.v_cache[page, 1, slot, 5] = 0
    b.k_cache[page, 0, slot, 9] = 0xFF
    out, lse = call(b)
    assert out[2:, :2].isnan().all() and not out[:2].isnan().any() and not out[:, 2:].isnan().any()


@pytest.mark.parametrize("spread", [(100, 140), (0, 246)])
def test_scales_of_any_size(spread):
    """V scales that jump between blocks, up to the whole range (values beyond bf16's own are
    kept out by codes of at most 1)."""
    b = Batch([1, 2], [333, 150], 8, 2, 64, 16, seed=5)
    g = torch.Generator().manual_seed(6)
    b.v_scale = torch.randint(spread[0], spread[1] + 1, b.v_scale.shape, generator=g).to(torch.uint8)
    b.v_cache = torch.randint(0, 56, b.v_cache.shape, generator=g).to(torch.uint8)
    check(b, *call(b))


def test_queries_of_any_size():
    b = Batch([1, 1], [100, 100], 4, 2, 64, 16, seed=7)
    b.q[0] = b.q[0] * 2.0 ** -120
    b.q[1, 0], b.q[1, 1] = b.q[1, 0] * 0, b.q[1, 1] * 2.0 ** -60
    b.q[1, 2, ::2] *= 2.0 ** -30
    check(b, *call(b))
    b.q[0] = b.q[0] * 2.0 ** 125                     # times keys of about 2^-1 each
    check(b, *call(b, sm_scale=2.0 ** -5), sm_scale=2.0 ** -5)


def test_rows_behind_the_last_sequence_are_left():
    b = Batch([2, 1], [18, 50], 4, 2, 64, 16, seed=8, pad_rows=6)
    out = torch.full((b.T, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.T, 4), 7.0, device="cuda")
    call(b, out=out, lse=lse)
    check(b, out, lse)
    assert (out[3:] == 7.0).all() and (lse[3:] == 7.0).all()


def test_strided_queries():
    b = Batch([2, 1], [80, 50], 8, 2, 128, 32, seed=9)
    want, _ = call(b)
    dev = b.to("cuda")
    packed = torch.cat((b.q, b.k, b.v), 1).cuda()
    got = bsp.fp8kv_attention(packed[:, :8], *[dev[x] for x in NAMES])
    assert torch.equal(want, got)


def test_pages_outside_the_pool_are_not_read():
    """A page that the pool does not have counts as masked, and is reported."""
    b = Batch([1], [64], 4, 2, 64, 16, seed=10)
    b.table[0, 1] = b.pages
    out, lse = call(b)
    assert bsp.bsp_last_device_status() == -1 and bsp.bsp_last_device_status() == 0
    keep = torch.cat((torch.arange(0, 16), torch.arange(32, 64)))
    b.table[0, 1] = int(b.table[0, 0])
    k, v = b.values("k", 0, 64)[:, keep], b.values("v", 0, 64)[:, keep]
    z = torch.einsum("hgd,htd->hgt", b.q[0].double().view(2, 2, 64), k) / 8
    want = torch.einsum("hgt,htd->hgd", torch.softmax(z, -1), v).reshape(4, 64)
    assert torch.allclose(out[0].cpu().double(), want, rtol=2.0 ** -7, atol=2.0 ** -9 * float(v.abs().max()))


def test_malformed_batches_stay_inside():
    b = Batch([4, 4], [20, 20], 2, 2, 64, 16, seed=11)
    for cu, lens in (([0, 400, 9], [20, 20]), ([5, 2, -3], [20, 20]), ([0, 4, 8], [3, -9]),
                     ([0, 4, 8], [2 ** 31 - 1, 20])):
        b.cu, b.kv_len = torch.tensor(cu, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32)
        call(b)
        bsp.bsp_last_device_status()


def test_offsets_past_32_bits():
    page, Hkv, D = 64, 8, 128
    pages = (1 << 32) // (page * Hkv * D) + 9
    b = Batch([1], [200], 16, Hkv, D, page, seed=13)
    want = call(b)
    dev = b.to("cuda")
    big = {}
    for x in ("k_cache", "v_cache", "k_scale", "v_scale"):
        big[x] = torch.zeros((pages,) + dev[x].shape[1:], dtype=torch.uint8, device="cuda")
        big[x][pages - b.pages:] = dev[x]
    table = dev["block_table"] + (pages - b.pages)
    got = bsp.fp8kv_attention(b.q.cuda(), *big.values(), table, dev["cu_new"], dev["kv_len"],
                              return_lse=True)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_replayed_graph_follows_the_lengths():
    """One captured call, replayed while the sequences grow, against eager calls; two graphs that
    share a workspace, replayed one after the other."""
    b = Batch([1, 1], [900, 1500], 8, 2, 128, 64, seed=14)
    dev = b.to("cuda")
    q = b.q.cuda()
    need = bsp.fp8kv_attention_workspace_bytes(b.T, b.Hq, b.Hkv, b.D)
    ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(q), torch.empty_like(q)]
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    args = [dev[x] for x in NAMES]
    for g, o, w in zip(graphs, outs, (0, 100)):
        with torch.cuda.graph(g):
            bsp.fp8kv_attention(q, *args, out=o, window=w, workspace=ws)
    for lens in ([1, 1], [64, 700], [65, 2], [900, 1500]):
        dev["kv_len"].copy_(torch.tensor(lens, dtype=torch.int32))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, (0, 100)):
            assert torch.equal(o, bsp.fp8kv_attention(q, *args, window=w))


def test_two_streams_at_once_with_their_own_workspaces():
    bs = [Batch([1], [3000 + 500 * i], 16, 4, 128, 64, seed=20 + i) for i in range(2)]
    devs = [[x.to("cuda")[n] for n in NAMES] for x in bs]
    qs = [x.q.cuda() for x in bs]
    want = [bsp.fp8kv_attention(q, *d) for q, d in zip(qs, devs)]
    need = max(bsp.fp8kv_attention_workspace_bytes(x.T, x.Hq, x.Hkv, x.D) for x in bs)
    ws = [torch.empty((need,), dtype=torch.uint8, device="cuda") for _ in bs]
    outs = [torch.zeros_like(w) for w in want]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, q, d, o, w in zip(streams, qs, devs, outs, ws):
            bsp.fp8kv_attention(q, *d, out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("B,every", [(40, 3), (200, 1), (200, 67), (450, 5)])
@pytest.mark.parametrize("wide", [False, True])
def test_padded_batches(B, every, wide):
    """Many sequences, most of them without new tokens (stretches longer than a warp looks at at once),
    and tables that are wider than the lengths need."""
    n = [(1 + i % 2) if i % every == every - 1 else 0 for i in range(B)]
    b = Batch(n, [5 + 37 * i % 600 for i in range(B)], 4, 2, 64, 16, seed=B + every)
    if wide:
        b.table = torch.cat((b.table, torch.full((B, 300), -9, dtype=torch.int32)), 1)
    out, lse = call(b)
    assert bsp.bsp_last_device_status() == 0
    check(b, out, lse)


@pytest.mark.parametrize("n,lens,Hq,Hkv,D,page", [([1], [5000], 16, 8, 128, 4096),
                                                  ([3, 2], [900, 70], 24, 2, 256, 48),
                                                  ([2], [33000], 8, 1, 192, 64),
                                                  ([1] * 3, [640, 639, 1], 8, 8, 128, 64),
                                                  ([1] * 3, [641, 640, 1], 8, 8, 128, 64)])
def test_more_sizes(n, lens, Hq, Hkv, D, page):
    """Large pages, pages that end inside a tile, 16 rows of wide heads, tables at which items are cut
    and at which they are not."""
    b = Batch(n, lens, Hq, Hkv, D, page, seed=sum(lens))
    check(b, *call(b))


def test_shared_pages():
    """Two sequences that have read the same pages, and one page twice in a sequence."""
    b = Batch([1, 1], [150, 190], 8, 2, 64, 32, seed=30)
    b.table[1, :4] = b.table[0, :4]
    b.table[1, 4] = b.table[1, 2]
    check(b, *call(b))


def test_lengths_past_the_table_are_reported():
    b = Batch([1, 1], [64, 40], 4, 2, 64, 16, seed=31)
    want, _ = call(b)
    cap = b.table.shape[1] * 16
    b.kv_len[0] = cap + 3
    out, _ = call(b)
    assert bsp.bsp_last_device_status() == -1 and bsp.bsp_last_device_status() == 0
    assert torch.equal(out, want)                   # cut to the table: 64 tokens


def test_workspace_ends_where_it_says():
    b = Batch([2] * 5, [700 + 300 * i for i in range(5)], 16, 2, 128, 64, seed=32)
    need = bsp.fp8kv_attention_workspace_bytes(b.T, b.Hq, b.Hkv, b.D)
    room = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    out, lse = call(b, workspace=room[:need])
    check(b, out, lse)
    assert (room[need:] == 0xA5).all()


@pytest.mark.parametrize("as_int", [False, True])
def test_own_workspace_on_another_stream(as_int):
    """The memory of a workspace that the call made itself is not given to the current stream's next
    tensor while the call's kernels, far behind on another stream, still use it."""
    b = Batch([1], [9000], 16, 4, 128, 64, seed=33)
    dev = b.to("cuda")
    q, args = b.q.cuda(), [dev[x] for x in NAMES]
    want = bsp.fp8kv_attention(q, *args)
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    need = bsp.fp8kv_attention_workspace_bytes(b.T, b.Hq, b.Hkv, b.D)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    bsp.fp8kv_attention(q, *args, out=out, stream=side.cuda_stream if as_int else side)
    spoil = [torch.zeros((need,), dtype=torch.uint8, device="cuda") for _ in range(4)]
    for _ in range(200):
        for x in spoil:
            x.zero_()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
