"""The decode operators on another stream than the current one: what they allocate is that stream's, so it is
not memory that the current stream's queued work still reads."""
import pytest
import torch

import block_scaled_precision_act_b200 as bsp
import synth
from kv_reference import Batch

pytestmark = pytest.mark.gpu


def gemv():
    N, K, M = 4096, 512, 8
    w = synth.bf16_normal((N, K), 0.02, 1).cuda()
    g = bsp.nvfp4_global_scale(w)
    codes, sf = bsp.nvfp4_quantize_act(w, g)
    x = synth.bf16_normal((M, K), 1.0, 2).cuda()
    return lambda stream: bsp.nvfp4_gemv(x, codes, sf, g, stream=stream), M * N * 2


def cache():
    b = Batch([40], [90], 16, 2, 64, 16, seed=1)
    d = b.to("cuda")
    return b, d, b.q.cuda(), b.k.cuda(), b.v.cuda()


def append():
    b, d, q, k, v = cache()
    f = torch.ones(8, device="cuda")
    return lambda stream: bsp.fp8kv_append(k, v, **d, q=q, inv_freq=f, stream=stream), q.numel() * 2


def attend():
    b, d, q, k, v = cache()
    return lambda stream: bsp.fp8kv_attention(q, **d, stream=stream), q.numel() * 2


@pytest.mark.parametrize("make", [gemv, append, attend])
@pytest.mark.parametrize("as_int", [False, True])
def test_outputs_are_the_streams_own(make, as_int):
    call, nbytes = make()
    side = torch.cuda.Stream()
    handle = side.cuda_stream if as_int else side
    want = call(None)
    torch.cuda.synchronize()
    call(handle)                                     # loads what a first call loads
    torch.cuda.synchronize()
    for _ in range(5):
        tmp = torch.full((nbytes,), 7, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        torch.cuda._sleep(5_000_000)
        kept = tmp.clone()                           # queued, not done
        del tmp                                      # the current stream's pool may give its memory away
        got = call(handle)
        side.synchronize()
        torch.cuda.synchronize()
        assert (kept == 7).all() and torch.equal(got, want)
