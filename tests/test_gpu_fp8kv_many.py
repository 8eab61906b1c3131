"""fp8kv_append with more sequences than the threads of a CTA look at at once."""
import pytest
import torch

import block_scaled_precision_act_b200 as bsp
from kv_reference import BLOCK, Batch, encode, scale_exp
from test_gpu_fp8kv_append import call, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [255, 256, 257, 511, 513, 700])
@pytest.mark.parametrize("kind", ["single", "blocks"])
def test_around_the_threads_of_a_cta(B, kind):
    """Work counted by token and by block, idle sequences in stretches, first and last ones active."""
    if kind == "single":
        n = [0 if 3 <= i % 90 < 40 else 1 + i % 2 for i in range(B)]
    else:
        n = [0 if i % 5 else 40 + i % 7 for i in range(B - 1)] + [19]
    lens = [n[i] + 11 * i % 50 for i in range(B)]
    b = Batch(n, lens, 2, 1, 32, 16, seed=B)
    by_token = b.T < b.T // 16 + 2 * B
    assert by_token == (kind == "single")
    q, got = call(b, 32)
    assert bsp.bsp_last_device_status() == 0
    check(b, q, got, 32)


@pytest.mark.parametrize("B,every,n", [(70000, 1, 1), (1 << 20, 1, 1), (70000, 64, 150), (1 << 20, 4096, 4000),
                                       (66049, 66048, 40), (65537, 3, 1)])
def test_very_many(B, every, n):
    """Sequences i with i % every == 0 bring n tokens each at position 0; each has its own pages."""
    page, D = 16 if n == 1 else 64, 16
    active = torch.arange(0, B, every)
    T, per = n * active.numel(), -(-n // page)
    count = torch.zeros(B + 1, dtype=torch.int64)
    count[active + 1] = n
    cu = count.cumsum(0).to(torch.int32).cuda()
    kv_len = count[1:].to(torch.int32).cuda()
    pages = active.numel() * per
    table = torch.full((B, per), -1, dtype=torch.int32)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(B))
    table[active] = order.view(-1, per).to(torch.int32)
    g = torch.Generator().manual_seed(n)
    v = torch.randn((T, 1, D), generator=g).bfloat16()
    v *= torch.exp2(torch.randint(-9, 9, (T, 1, 1), generator=g)).bfloat16()
    pool = [torch.full((pages, 1, page, D), 0x55, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scales = [torch.full((pages, 1, page // BLOCK), 99, dtype=torch.uint8, device="cuda") for _ in "kv"]
    bsp.fp8kv_append(v.neg().cuda(), v.cuda(), *pool, *scales, table.cuda(), cu, kv_len)
    torch.cuda.synchronize()
    assert bsp.bsp_last_device_status() == 0
    # the sequences' tokens, blocks of 16
    x = torch.zeros((active.numel(), per * page, D), dtype=torch.float64)
    x[:, :n] = v.double().view(-1, n, D)
    amax = x.view(-1, per * page // BLOCK, BLOCK * D).abs().amax(-1)
    e = scale_exp(amax)
    there = torch.arange(per * page // BLOCK) * BLOCK < n
    for pl, sc, sign in ((pool[0], scales[0], -1), (pool[1], scales[1], 1)):
        got_e = sc.cpu()[order, 0].view(-1, per * page // BLOCK).long()
        assert torch.equal(got_e[:, there], e[:, there]) and (got_e[:, ~there] == 99).all()
        got = pl.cpu()[order, 0].view(-1, per * page, D)
        unit = torch.exp2(e.double() - 127).repeat_interleave(BLOCK, 1)[..., None]
        assert torch.equal(got[:, :n], encode(sign * x[:, :n] / unit[:, :n]))
        assert (got[:, n:] == 0x55).all()


@pytest.mark.parametrize("B", [193, 70000, 1 << 20])
def test_attention_over_very_many(B):
    """A few active sequences among B, of one tile each (nothing is cut), against the same ones alone."""
    b = Batch([2, 1, 3, 1], [100, 1, 128, 57], 8, 2, 64, 16, seed=B)
    dev = b.to("cuda")
    want, wlse = bsp.fp8kv_attention(b.q.cuda(), **dev, return_lse=True)
    at = torch.tensor([0, 5, B // 2, B - 1])
    n = torch.zeros(B + 1, dtype=torch.int32)
    n[at + 1] = torch.tensor(b.n, dtype=torch.int32)
    kv_len = torch.full((B,), 9, dtype=torch.int32)
    kv_len[at] = b.kv_len
    table = torch.full((B, b.table.shape[1]), -1, dtype=torch.int32)
    table[at] = b.table
    dev.update(cu_new=n.cumsum(0).to(torch.int32).cuda(), kv_len=kv_len.cuda(), block_table=table.cuda())
    out, lse = bsp.fp8kv_attention(b.q.cuda(), **dev, return_lse=True)
    torch.cuda.synchronize()
    assert bsp.bsp_last_device_status() == 0
    assert torch.equal(out, want) and torch.equal(lse, wlse)
