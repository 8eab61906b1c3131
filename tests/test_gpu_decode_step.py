"""The decode path as it is used: a weight-only QuantLinear makes q, k and v of the new tokens side
by side, PagedKVCache appends and attends, another QuantLinear projects; a prompt is read in first,
then single tokens, in two ragged sequences that share the pool.

Every stage is checked against its 64-bit value on the stage's own inputs (bounds: those of the
stages' own tests), so that a mistake in what one hands to the next shows, and the whole against a
plain attention over the tokens as they were, whose distance is the cache's 4 bits."""
import math

import pytest
import torch

import block_scaled_precision_act_b200 as bsp
from block_scaled_precision_act_b200.nn import PagedKVCache, QuantLinear
from kv_reference import Batch, rotate
from test_gpu_fp8kv_attention import check as check_attention

pytestmark = pytest.mark.gpu

HIDDEN, HQ, HKV, D, PAGE = 512, 8, 2, 64, 32


def linear(N, K, seed, rows):
    g = torch.Generator().manual_seed(seed)
    lin = torch.nn.Linear(K, N, bias=True)
    with torch.no_grad():
        lin.weight.copy_(torch.randn((N, K), generator=g) * K ** -0.5)
        lin.bias.copy_(0.1 * torch.randn((N,), generator=g))
    q = QuantLinear.from_linear(lin.to(torch.bfloat16).cuda(), "nvfp4", input_scale=0.002)
    q.weight_only_rows = rows
    return q


def dequantised(q):
    codes, g = q.weight.cpu().long(), q.weight_scale_2.double().cpu()
    v = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
    v = torch.cat((v, -v))
    w = torch.stack((v[codes & 15], v[codes >> 4]), -1).view(q.out_features, -1)
    s = q.weight_scale.float().double().cpu().repeat_interleave(16, 1)
    return w * s * g


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_prompt_then_single_tokens(graph):
    qkv, proj = linear((HQ + 2 * HKV) * D, HIDDEN, 1, 32), linear(HIDDEN, HQ * D, 2, 32)
    wq, bq = dequantised(qkv), qkv.bias.double().cpu()
    cache = PagedKVCache(16, HKV, D, PAGE, device="cuda")
    table = torch.tensor([[3, 7, 1, 14], [5, 0, 11, 2]], dtype=torch.int32, device="cuda")
    inv = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    g = torch.Generator().manual_seed(3)
    lens, seen = [0, 0], [[], []]                    # keys and values of each sequence as they were

    def layer(x, cu, kv_len):
        y = qkv(x).view(x.shape[0], HQ + 2 * HKV, D)
        q = cache.append(y[:, HQ:HQ + HKV], y[:, HQ + HKV:], table, cu, kv_len, q=y[:, :HQ],
                         inv_freq=inv)
        o, lse = cache.attend(q, table, cu, kv_len, return_lse=True)
        return y, q, o, lse, proj(o.reshape(x.shape[0], HQ * D))

    captured = None
    steps = [(13, 19)] + [(1, 1)] * 14 + [(3, 0)]
    for n in steps:
        T = sum(n)
        lens = [a + b for a, b in zip(lens, n)]
        x = torch.randn((T, HIDDEN), generator=g).bfloat16().cuda()
        cu = torch.tensor([0, n[0], T], dtype=torch.int32, device="cuda")
        kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if graph and n == (1, 1):                    # one captured step, replayed as the lengths grow
            if captured is None:
                bufs = [x.clone(), cu.clone(), kv_len.clone()]
                captured = torch.cuda.CUDAGraph()
                with torch.cuda.graph(captured):
                    res = layer(*bufs)
            for b, v in zip(bufs, (x, cu, kv_len)):
                b.copy_(v)
            captured.replay()
            y, q, o, lse, z = [r.clone() for r in res]
        else:
            y, q, o, lse, z = layer(x, cu, kv_len)
        torch.cuda.synchronize()
        assert bsp.bsp_last_device_status() == 0
        # projection
        want = x.double().cpu() @ wq.t() + bq
        top = x.double().cpu().abs().amax(1, keepdim=True) * wq.abs().sum(1)
        bound = want.abs() * (2.0 ** -8 + 2.0 ** -21) + 2.0 ** -19.58 * top + 2.0 ** -21 * bq.abs()
        bound += (HIDDEN / 64 + 72) * 2.0 ** -22 * (x.double().cpu().abs() @ wq.abs().t() + top)
        yc = y.reshape(T, -1).double().cpu()
        assert ((yc - want).abs() <= bound).all()
        # rotation, and what the cache stands for
        b = Batch(list(n), lens, HQ, HKV, D, PAGE, seed=0)
        b.table, b.cu, b.kv_len, b.q = table.cpu(), cu.cpu(), kv_len.cpu(), q.cpu()
        b.k_cache, b.v_cache = cache.k_cache.cpu(), cache.v_cache.cpu()
        b.k_scale, b.v_scale = cache.k_scale.cpu(), cache.v_scale.cpu()
        yc = y.cpu()
        for s in range(2):
            rows, pos = slice(int(b.cu[s]), int(b.cu[s]) + n[s]), torch.arange(lens[s] - n[s], lens[s])
            if n[s] == 0:
                continue
            qr = rotate(yc[rows, :HQ], pos, inv.cpu(), False, 1.0)
            slack = 2.0 ** -19 * yc[rows, :HQ].double().abs().amax(-1, keepdim=True)
            assert ((q.cpu()[rows].double() - qr).abs() <= qr.abs() * 2.0 ** -8 + slack).all()
            seen[s].append((rotate(yc[rows, HQ:HQ + HKV], pos, inv.cpu(), False, 1.0),
                            yc[rows, HQ + HKV:].double()))
            for which, i in (("k", 0), ("v", 1)):
                held = b.values(which, s, lens[s]).transpose(0, 1)
                was = torch.cat([t[i] for t in seen[s]])
                unit = torch.exp2((b.k_scale if i == 0 else b.v_scale)[b.table[s].long()].double() - 127)
                unit = unit.transpose(0, 1).reshape(HKV, -1).repeat_interleave(16, 1)[:, :lens[s]]
                # each time that a block's scale is raised rounds once more where codes are subnormal
                off = was.abs() * 2.0 ** -4 * 1.01 + unit.t()[..., None] * 2.0 ** -9
                assert ((held - was).abs() <= off).all()
        check_attention(b, o, lse)
        # the output projection
        wp, bp = dequantised(proj), proj.bias.double().cpu()
        oc = o.reshape(T, -1).double().cpu()
        want = oc @ wp.t() + bp
        top = oc.abs().amax(1, keepdim=True) * wp.abs().sum(1)
        bound = want.abs() * (2.0 ** -8 + 2.0 ** -21) + 2.0 ** -19.58 * top + 2.0 ** -21 * bp.abs()
        bound += (HQ * D / 64 + 72) * 2.0 ** -22 * (oc.abs() @ wp.abs().t() + top)
        assert ((z.double().cpu() - want).abs() <= bound).all()
    # the whole: attention of the last step's rows over the tokens as they were, within the codes' 2^-4
    for s in range(2):
        for i in range(steps[-1][s]):
            row, end = int(b.cu[s]) + i, lens[s] - steps[-1][s] + i + 1
            k = torch.cat([t[0] for t in seen[s]])[:end].transpose(0, 1)
            v = torch.cat([t[1] for t in seen[s]])[:end].transpose(0, 1)
            qd = q.cpu()[row].double().view(HKV, HQ // HKV, D)
            score = torch.einsum("hgd,htd->hgt", qd, k) / math.sqrt(D)
            p = torch.softmax(score, -1)
            want = torch.einsum("hgt,htd->hgd", p, v)
            ds = torch.einsum("hgd,htd->hgt", qd.abs(), k.abs()).amax(-1, keepdim=True) / math.sqrt(D) / 16
            mass = torch.einsum("hgt,htd->hgd", p, v.abs())
            got = o.cpu()[row].double().view(HKV, HQ // HKV, D)
            assert ((got - want).abs() <= (torch.exp(2 * ds) * 1.07 - 1) * mass + 0.01 * mass.amax()).all()
