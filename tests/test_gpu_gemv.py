"""nvfp4_gemv on the GPU against the 64-bit product of the decoded weight.

Bound.  The bounds' first form was for x as seven E2M1 terms, held to 2^-19.58 of the row's largest
element (`top`); the kernels hold x in f16 to 2^-39 of it, which is inside.  Weights and their scales'
products are exact in f16 and their products with x in fp32.  A sum over K is made by two halves of the
warps, each in a chain of at most K / 32 product instructions (K / 512 + 1 steps of 16), and each adds 16
products to the sum with an error of at most one unit, 2^-23 of sum |x||w|, cut or rounded: K / 64 + 8 times
2^-22 in all, and half of what it is where the halves have half of the sum.  At most K / 1024 + 2 parts
are added after that, 2^-24 each.  (K / 64 + 72) 2^-22 (S + top) covers it.  The factors and the bias add
2^-21 of the result, the output 2^-8."""
import math

import numpy as np
import pytest
import torch

import block_scaled_precision_act_b200 as bsp
import synth
from block_scaled_precision_act_b200.nn import QuantLinear

pytestmark = pytest.mark.gpu
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def weight(N, K, seed, std=0.02):
    w = synth.bf16_normal((N, K), std, seed).cuda()
    g = bsp.nvfp4_global_scale(w)
    codes, sf = bsp.nvfp4_quantize_act(w, g)
    return codes, sf, g


def decode(codes, sf, N, K):
    """[N, K] doubles, without the global scale."""
    c = codes.cpu().long()
    v = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float64)
    w = torch.stack((v[c & 15], v[c >> 4]), -1).view(N, K)
    lin = bsp.nvfp4_sf_convert(sf, N, K, bsp.SF_MMA, bsp.SF_LINEAR).cpu().view(torch.float8_e4m3fn)
    return w * lin.view(N, K // 16).double().repeat_interleave(16, 1)


def check(y, x, codes, sf, g, bias=None):
    N, K = codes.shape[0], 2 * codes.shape[1]
    w, xd = decode(codes, sf, N, K) * g.double().cpu(), x.cpu().double()
    want = xd @ w.t()
    S = xd.abs() @ w.abs().t()
    top = xd.abs().amax(1, keepdim=True) * w.abs().sum(1)
    if bias is not None:
        want = want + bias.cpu().double()
    bound = want.abs() * (2.0 ** -8 + 2.0 ** -21) + 2.0 ** -19.58 * top
    bound += (K / 64 + 72) * 2.0 ** -22 * (S + top)
    bound += 0 if bias is None else bias.cpu().double().abs() * 2.0 ** -21
    d = (y.cpu().double() - want).abs()
    assert (d <= bound).all(), float((d / bound).max())


@pytest.mark.parametrize("M", [1, 2, 3, 5, 8, 9, 16, 17, 24, 31, 32])
@pytest.mark.parametrize("N,K", [(8, 64), (136, 320), (256, 1024)])
def test_rows(M, N, K):
    codes, sf, g = weight(N, K, 3 * N + K)
    x = synth.bf16_normal((M, K), 1.0, M, 0.01, 30.0).cuda()
    bias = synth.bf16_normal((N,), 0.1, 7).cuda() if (M + N) % 3 else None
    check(bsp.nvfp4_gemv(x, codes, sf, g, bias=bias), x, codes, sf, g, bias)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (7, 10376, 2624), (4, 264, 12288), (1, 8, 16384),
                                   (32, 1000, 8256), (13, 128, 64), (1, 65544, 128), (2, 40, 4160)])
def test_sizes(M, N, K):
    codes, sf, g = weight(N, K, N + K)
    x = synth.bf16_normal((M, K), 1.0, M).cuda()
    bias = synth.bf16_normal((N,), 0.1, 7).cuda()
    check(bsp.nvfp4_gemv(x, codes, sf, g, bias=bias), x, codes, sf, g, bias)


def test_every_code_and_scale():
    """All 16 codes under every finite scale byte without a sign (the only ones that a block scale
    has), each block on its own (x is one-hot): the product is exact, so the output is one rounding."""
    N, K = 256, 1024
    i = torch.arange(N * K // 2)
    codes = (i * 7 + i // (K // 2) * 13).to(torch.uint8).view(N, K // 2).cuda()
    lin = ((torch.arange(N * K // 16) * 5 + 1) % 127).to(torch.uint8)
    sf = bsp.nvfp4_sf_convert(lin.cuda(), N, K, bsp.SF_LINEAR, bsp.SF_MMA)
    g = torch.tensor([0.125], device="cuda")
    w = decode(codes, sf, N, K) * 0.125
    for k in range(0, K, 37):
        x = torch.zeros((3, K), dtype=torch.bfloat16, device="cuda")
        x[1, k], x[2, k] = 1.5, -2.0 ** -100
        y = bsp.nvfp4_gemv(x, codes, sf, g).cpu()
        assert (y[0] == 0).all()
        assert torch.equal(y[1], (1.5 * w[:, k]).bfloat16())
        assert torch.equal(y[2], (-2.0 ** -100 * w[:, k]).bfloat16())


def test_activations_of_any_size():
    N, K = 128, 512
    codes, sf, g = weight(N, K, 5)
    x = synth.bf16_normal((6, K), 1.0, 6).cuda()
    x[1] *= 2.0 ** 100
    x[2] *= 2.0 ** -100
    x[3, ::3] *= 2.0 ** 40
    x[4, 256:] *= 2.0 ** -60
    x[5] = 0
    check(bsp.nvfp4_gemv(x, codes, sf, g), x, codes, sf, g)


def test_infinities_and_nan_stay_in_their_row():
    N, K = 64, 256
    codes, sf, g = weight(N, K, 8)
    x = synth.bf16_normal((4, K), 1.0, 9).cuda()
    clean = bsp.nvfp4_gemv(x, codes, sf, g)
    x[1, 17], x[2, 200] = math.nan, math.inf
    y = bsp.nvfp4_gemv(x, codes, sf, g)
    assert torch.equal(y[[0, 3]], clean[[0, 3]])
    assert y[1].isnan().all() and not y[2].isfinite().any()


def test_a_row_does_not_depend_on_its_neighbours():
    N, K = 520, 1088
    codes, sf, g = weight(N, K, 11)
    x = synth.bf16_normal((32, K), 1.0, 12, 0.01, 50.0).cuda()
    y = bsp.nvfp4_gemv(x, codes, sf, g)
    for m in (1, 2, 4, 9, 20):
        check(bsp.nvfp4_gemv(x[:m].contiguous(), codes, sf, g), x[:m], codes, sf, g)
    assert torch.equal(y, bsp.nvfp4_gemv(x, codes, sf, g))


def test_offsets_past_32_bits():
    """A weight of more than 2^32 code bytes: the last rows against the same rows alone."""
    K, N = 65536, (1 << 32) // 32768 + 128
    codes = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    sf = torch.zeros((bsp.nvfp4_sf_bytes(N, K),), dtype=torch.uint8, device="cuda")
    tail = weight(128, K, 21)
    codes[N - 128:] = tail[0]
    sf.view(N // 128, -1)[-1] = tail[1]
    x = synth.bf16_normal((2, K), 1.0, 22).cuda()
    y = bsp.nvfp4_gemv(x, codes, sf, tail[2])
    check(y[:, N - 128:].contiguous(), x, *tail)
    assert (y[:, :N - 128] == 0).all()


def test_other_stream_and_replayed_graph():
    codes, sf, g = weight(1024, 2048, 31)
    x = synth.bf16_normal((3, 2048), 1.0, 32).cuda()
    want = bsp.nvfp4_gemv(x, codes, sf, g)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    bsp.nvfp4_gemv(x, codes, sf, g, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bsp.nvfp4_gemv(x, codes, sf, g, out=out)
    x.neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, -want)


def test_against_the_dequantised_weight():
    """The weight-only product is that of nvfp4_dequantize's weight up to that weight's bf16
    rounding (2^-8 of each product)."""
    N, K = 512, 1024
    codes, sf, g = weight(N, K, 41)
    x = synth.bf16_normal((4, K), 1.0, 42).cuda()
    w = bsp.nvfp4_dequantize(codes, sf, g).double()
    y = bsp.nvfp4_gemv(x, codes, sf, g).double()
    S = x.double().abs() @ w.abs().t()
    assert ((y - x.double() @ w.t()).abs() <= 2.0 ** -8 * (y.abs() + S) * 1.01).all()


@pytest.mark.parametrize("shape", [(64,), (1, 64), (2, 3, 64)])
def test_vector_shapes_through_quant_linear(shape):
    lin = torch.nn.Linear(64, 24).to(torch.bfloat16).cuda()
    q = QuantLinear.from_linear(lin, "nvfp4", input_scale=0.01)
    q.weight_only_rows = 32
    x = torch.randn(shape, device="cuda").bfloat16()
    y = q(x)
    assert y.shape == shape[:-1] + (24,)
    sf = bsp.nvfp4_sf_convert(q.weight_scale.view(torch.uint8).contiguous(), 24, 64, bsp.SF_LINEAR,
                              bsp.SF_MMA)
    want = bsp.nvfp4_gemv(x.reshape(-1, 64), q.weight, sf, q.weight_scale_2, bias=q.bias)
    assert torch.equal(y.reshape(-1, 24), want)
    q.weight_only_rows = 0                          # the default: activations quantized
    q8 = QuantLinear.from_state_dict(q.state_dict())
    assert torch.equal(q(x), q8(x))


@pytest.mark.parametrize("N,K", [(40008, 192), (131072, 256), (16000, 1088), (8200, 2624), (136, 4416),
                                 (2048, 16384)])
@pytest.mark.parametrize("M", [1, 8, 9, 16, 17])
def test_small_weights_in_one_launch_and_two(M, N, K):
    """The K of a tile in one, two, four and eight pieces of even and uneven lengths, and the sizes past
    which the call goes the other way."""
    codes, sf, g = weight(N, K, N + K)
    x = synth.bf16_normal((M, K), 1.0, M, 0.01, 30.0).cuda()
    bias = synth.bf16_normal((N,), 0.1, 7).cuda() if M % 2 else None
    check(bsp.nvfp4_gemv(x, codes, sf, g, bias=bias), x, codes, sf, g, bias)


@pytest.mark.parametrize("N,K", [(136, 4416), (8200, 2624), (40008, 192), (1024, 16640)])
def test_a_row_that_is_not_finite(N, K):
    codes, sf, g = weight(N, K, 51)
    x = synth.bf16_normal((12, K), 1.0, 52).cuda()
    clean = bsp.nvfp4_gemv(x, codes, sf, g)
    for i, v in enumerate([math.inf, -math.inf, math.nan]):
        for j, k in enumerate([0, K // 2, K - 1]):
            x[3 * i + j, k] = v
    y = bsp.nvfp4_gemv(x, codes, sf, g)
    assert y[:9].isnan().all() and torch.equal(y[9:], clean[9:])


@pytest.mark.parametrize("M,N,K", [(32, 4104, 8192), (7, 10376, 2624), (1, 520, 65536)])
def test_workspace_ends_where_it_says(M, N, K):
    codes, sf, g = weight(N, K, 61)
    x = synth.bf16_normal((M, K), 1.0, 62).cuda()
    need = bsp.nvfp4_gemv_workspace_bytes(M, N, K)
    room = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = bsp.nvfp4_gemv(x, codes, sf, g, out=out[:M * N], workspace=room[:need])
    check(y.view(M, N), x, codes, sf, g)
    assert (room[need:] == 0xA5).all() and (out[M * N:] == 7).all()


def test_own_workspace_on_another_stream():
    """The workspace that the call made itself is not given away while its kernels wait."""
    codes, sf, g = weight(2048, 16384, 71)
    x = synth.bf16_normal((9, 16384), 1.0, 72).cuda()
    want = bsp.nvfp4_gemv(x, codes, sf, g)
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    need = bsp.nvfp4_gemv_workspace_bytes(9, 2048, 16384)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    bsp.nvfp4_gemv(x, codes, sf, g, out=out, stream=side)
    spoil = [torch.zeros((need,), dtype=torch.uint8, device="cuda") for _ in range(4)]
    for _ in range(200):
        for y in spoil:
            y.zero_()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_a_weight_written_just_before():
    """The weight, its scales, x and the factor as the kernels in front of the call leave them, with no
    wait in between: what an SM read of them in the call before is not used again."""
    N, K = 4096, 1024
    ws = [weight(N, K, 80 + i) for i in range(2)]
    xs = [synth.bf16_normal((2, K), 1.0, 90 + i).cuda() for i in range(2)]
    want = [bsp.nvfp4_gemv(x, *w) for x, w in zip(xs, ws)]
    now, x = [t.clone() for t in ws[0]], xs[0].clone()
    outs = []
    for i in range(40):
        for a, b in zip(now, ws[i % 2]):
            a.copy_(b)
        x.copy_(xs[i % 2])
        outs.append(bsp.nvfp4_gemv(x, *now))
    for i, y in enumerate(outs):
        assert torch.equal(y, want[i % 2])


@pytest.mark.parametrize("N,K", [(40968, 2112), (600, 50048), (136, 98368), (20008, 6464)])
@pytest.mark.parametrize("M", [1, 7, 9, 16, 23, 32])
def test_large_weights(M, N, K):
    """Tiles that runs begin, end and pass through, steps of K that are not full."""
    codes, sf, g = weight(N, K, N + K)
    x = synth.bf16_normal((M, K), 1.0, M, 0.01, 30.0).cuda()
    bias = synth.bf16_normal((N,), 0.1, 7).cuda() if M % 2 else None
    y = bsp.nvfp4_gemv(x, codes, sf, g, bias=bias)
    check(y, x, codes, sf, g, bias)
    assert torch.equal(y, bsp.nvfp4_gemv(x, codes, sf, g, bias=bias))


def test_large_weight_rows_that_are_not_finite():
    N, K = 38408, 2048
    codes, sf, g = weight(N, K, 53)
    x = synth.bf16_normal((12, K), 1.0, 54).cuda()
    clean = bsp.nvfp4_gemv(x, codes, sf, g)
    for i, v in enumerate([math.inf, -math.inf, math.nan]):
        for j, k in enumerate([0, K // 2, K - 1]):
            x[3 * i + j, k] = v
    y = bsp.nvfp4_gemv(x, codes, sf, g)
    assert y[:9].isnan().all() and torch.equal(y[9:], clean[9:])


@pytest.mark.parametrize("N,K", [(38408, 2048), (136, 98368), (2048, 4096)])
def test_streams_at_once_and_graphs_that_share_a_workspace(N, K):
    M = 9
    ws = [weight(N, K, 55 + i) for i in range(2)]
    xs = [synth.bf16_normal((M, K), 1.0, 56 + i).cuda() for i in range(2)]
    want = [bsp.nvfp4_gemv(x, *w) for x, w in zip(xs, ws)]
    outs = [torch.zeros_like(want[0]) for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, x, w, o in zip(streams, xs, ws, outs):
            bsp.nvfp4_gemv(x, *w, out=o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    need = bsp.nvfp4_gemv_workspace_bytes(M, N, K)
    room = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for gr, x, w, o in zip(graphs, xs, ws, outs):
        with torch.cuda.graph(gr):
            bsp.nvfp4_gemv(x, *w, out=o, workspace=room)
    for i in (0, 1, 0, 1, 1):
        outs[i].zero_()
        graphs[i].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_the_default_stream_by_its_handle():
    codes, sf, g = weight(2048, 16384, 91)
    x = synth.bf16_normal((9, 16384), 1.0, 92).cuda()
    want = bsp.nvfp4_gemv(x, codes, sf, g)
    torch.cuda.synchronize()
    got = bsp.nvfp4_gemv(x, codes, sf, g, stream=0)
    assert torch.equal(got, want)
    assert torch.equal(bsp.nvfp4_gemv(x, codes, sf, g, stream=torch.cuda.default_stream()), want)


def test_quant_linear_past_the_rows_of_the_gemv():
    lin = torch.nn.Linear(128, 64).to(torch.bfloat16).cuda()
    q = QuantLinear.from_linear(lin, "nvfp4", input_scale=0.01)
    x = torch.randn(40, 128, device="cuda").bfloat16()
    want = q(x)
    q.weight_only_rows = 64
    assert torch.equal(q(x), want)
    few = q(x[:32])
    check(few, x[:32], q.weight, q._sf_mma, q.weight_scale_2, q.bias)
