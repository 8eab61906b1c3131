"""Waits of the decode operators that run out: the loads of a call stop early, every wait is bounded,
the call reports BSP_ERR_TIMEOUT and returns, and the next one is right."""
import pytest
import torch

import block_scaled_precision_act_b200 as bsp

NAMES = ("k_cache", "v_cache", "k_scale", "v_scale", "block_table", "cu_new", "kv_len")


def test_the_hook_gives_back_what_it_held():
    assert bsp.bsp_testing_set_load_stall(3) == -1
    assert bsp.bsp_testing_set_load_stall(0) == 3
    assert bsp.bsp_testing_set_load_stall(-1) == 0
    assert bsp.bsp_testing_set_load_stall(-7) == -1
    assert bsp.bsp_testing_set_load_stall(-1) == -1


@pytest.fixture
def short_waits():
    old = bsp.bsp_set_wait_limit_ms(20)
    yield
    bsp.bsp_testing_set_load_stall(-1)
    bsp.bsp_set_wait_limit_ms(old)


# new tokens, lengths, Hq, Hkv, D, page, window: the four forms of the kernel; one CTA for each item, items
# cut into runs, several items in a run, lengths that end inside a tile and at its end
CASES = [
    ([1], [300], 4, 1, 64, 64, 0),
    ([1, 1], [384, 640], 8, 2, 128, 64, 0),
    ([3], [2000], 8, 1, 128, 32, 0),
    ([1], [300], 4, 1, 256, 64, 0),
    ([4, 2], [700, 129], 16, 2, 192, 16, 90),
    ([1] * 40, [130 + 61 * i for i in range(40)], 8, 8, 64, 16, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"D{c[4]}-B{len(c[0])}-L{max(c[1])}")
@pytest.mark.parametrize("loads", [0, 1, 2, 3, 5])
def test_attention_returns_when_its_loads_stop(case, loads, short_waits):
    from kv_reference import Batch
    n, lens, Hq, Hkv, D, page, window = case
    b = Batch(n, lens, Hq, Hkv, D, page, seed=1)
    dev = b.to("cuda")
    args, q = [dev[x] for x in NAMES], b.q.cuda()
    want = bsp.fp8kv_attention(q, *args, window=window)
    torch.cuda.synchronize()
    assert bsp.bsp_last_device_status() == 0
    bsp.bsp_testing_set_load_stall(loads)
    bsp.fp8kv_attention(q, *args, window=window)
    torch.cuda.synchronize()
    status = bsp.bsp_last_device_status()
    # a run of the smallest weight holds two tiles, four loads; a longer one stops at five too
    assert status == -6 or (loads == 5 and status == 0)
    bsp.bsp_testing_set_load_stall(-1)
    got = bsp.fp8kv_attention(q, *args, window=window)
    torch.cuda.synchronize()
    assert bsp.bsp_last_device_status() == 0 and torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 40968, 2112), (16, 16384, 8192), (32, 2048, 16384), (9, 136, 98368)])
@pytest.mark.parametrize("loads", [0, 1, 2])
def test_gemv_returns_when_its_loads_stop(M, N, K, loads, short_waits):
    """Sizes that go by two launches.  A CTA without a second or third chunk of x does not notice."""
    import synth
    w = synth.bf16_normal((N, K), 0.02, 1).cuda()
    g = bsp.nvfp4_global_scale(w)
    codes, sf = bsp.nvfp4_quantize_act(w, g)
    x = synth.bf16_normal((M, K), 1.0, 2).cuda()
    want = bsp.nvfp4_gemv(x, codes, sf, g)
    torch.cuda.synchronize()
    assert bsp.bsp_last_device_status() == 0
    bsp.bsp_testing_set_load_stall(loads)
    bsp.nvfp4_gemv(x, codes, sf, g)
    torch.cuda.synchronize()
    status = bsp.bsp_last_device_status()
    assert status == -6 or (status == 0 and loads > 0)
    bsp.bsp_testing_set_load_stall(-1)
    got = bsp.nvfp4_gemv(x, codes, sf, g)
    torch.cuda.synchronize()
    assert bsp.bsp_last_device_status() == 0 and torch.equal(got, want)
