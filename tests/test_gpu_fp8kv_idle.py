"""Sequences of a batch that bring no token: fp8kv_append and fp8kv_attention look at neither their
length nor their row of the table, so both may be stale.

The batches have more than two tokens for each sequence, so that append's work is counted by block
(16 tokens), where an idle sequence has room for a unit of its own; lengths of idle sequences that end
inside a block are what such a unit would have worked on."""
import pytest
import torch

import block_scaled_precision_act_b200 as bsp
from kv_reference import Batch
from test_gpu_fp8kv_append import call, check, inv_freq
from test_gpu_fp8kv_attention import call as attend, check as check_attention

pytestmark = pytest.mark.gpu
POOL = ("k_cache", "v_cache", "k_scale", "v_scale")


def batch(seed, rows=1):
    """Two sequences that append 37 and 20 tokens, and idle ones in front, between and behind."""
    n = [0] * rows + [37] + [0] * rows + [20] + [0] * rows
    lens = [5 + i for i in range(rows)] + [50] + [21 + i for i in range(rows)] + [29] + \
        [100 + i for i in range(rows)]
    assert sum(n) >= sum(n) // 16 + 2 * len(n)
    return Batch(n, lens, 4, 2, 64, 16, seed)


def idle(b):
    return [s for s in range(b.B) if b.n[s] == 0]


def test_an_idle_row_of_no_pages_is_not_reported():
    b = batch(1)
    for s in idle(b):
        b.table[s] = -1
    q, got = call(b, 64)
    assert bsp.bsp_last_device_status() == 0
    check(b, q, got, 64)


@pytest.mark.parametrize("length", [-3, 2 ** 31 - 1, 77])
def test_a_stale_length_of_an_idle_sequence_is_not_reported(length):
    b = batch(2)
    for s in idle(b):
        b.kv_len[s] = length
    q, got = call(b, 64)
    assert bsp.bsp_last_device_status() == 0
    check(b, q, got, 64)


def test_scales_of_an_idle_sequence_stay_as_they_are():
    b = batch(3)
    for s in idle(b):
        pages = b.table[s][b.table[s] >= 0].long()
        b.k_scale[pages], b.v_scale[pages] = 255, 250
    q, got = call(b, 64)
    assert bsp.bsp_last_device_status() == 0
    check(b, q, got, 64)                             # also: every other scale and code is unchanged


@pytest.mark.parametrize("seed", range(8))
def test_idle_rows_that_name_a_page_of_another_sequence(seed):
    """Every block of the idle sequences' rows is one that an active sequence raises the scale of; the
    call is repeated on the same cache many times, and gives the same one each time."""
    b = batch(10 + seed, rows=3)
    b.v, b.k = b.v * 64, b.k * 64                    # above what the blocks hold
    for s in idle(b):                                # the page of the first sequence's block 0, half full
        b.table[s] = b.table[b.n.index(37), 0]
    q, got = call(b, 32)
    assert bsp.bsp_last_device_status() == 0
    check(b, q, got, 32)
    dev, f = b.to("cuda"), inv_freq(32).cuda()
    k, v = b.k.cuda(), b.v.cuda()
    args = [dev[x] for x in POOL + ("block_table", "cu_new", "kv_len")]
    saved = [a.clone() for a in args[:4]]
    for _ in range(200):
        for a, s in zip(args, saved):
            a.copy_(s)
        bsp.fp8kv_append(k, v, *args, inv_freq=f)
        for a, x in zip(args, POOL):
            assert torch.equal(a.cpu(), got[x]), x


def test_attention_with_stale_idle_rows():
    b = batch(4)
    for s in idle(b):
        b.table[s], b.kv_len[s] = -1, 2 ** 31 - 1
    out, lse = attend(b)
    assert bsp.bsp_last_device_status() == 0
    check_attention(b, out, lse)


def test_all_sequences_idle():
    """A padded batch whose rows all lie behind cu_new[B]."""
    b = Batch([0, 0], [5, 40], 4, 2, 64, 16, seed=5, pad_rows=70)
    b.table[:] = -1
    out = torch.full((b.T, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    q, got = call(b, 64, q_out=out)
    assert (q == 7.0).all()
    for x in POOL:
        assert torch.equal(got[x], getattr(b, x)), x
    o, _ = attend(b, out=out)
    assert (o == 7.0).all() and bsp.bsp_last_device_status() == 0
