"""nvfp4_gemv where the result is known to the last bit, and the bound of the present kernels.

Exact: x of small whole numbers, scales of 1/2, 1 and 2, a power of two as global scale.  Every product
is a multiple of 1/4 of at most 36 and sums of them stay below 2^24 quarters, so fp32 holds every partial
sum, in whatever order, and the output is one rounding to bf16.  A step of K, or 64 columns of one, that
is left out, taken twice or read from another place shows.

Bound (check): x is held to 2^-39 of the row's largest element (`top`), weights times their scales are
exact in f16 and their products with x in fp32.  A sum over K is made by two halves of the warps, each a
chain of at most K / 512 + 1 steps of 16 product instructions, that is K / 32 + 16, and an instruction is
off by at most 2^-23 of the sum of magnitudes, of which the two halves together have S: (K / 64 + 8) 2^-22 S.
At most 64 parts are added after that, 2^-24 S each.  The factors add 2^-22 of the sum and the bias 2^-24,
the output 2^-8 of the value."""
import pytest
import torch

import block_scaled_precision_act_b200 as bsp
import synth
from test_gpu_gemv import E2M1, decode, weight

pytestmark = pytest.mark.gpu

SIZES = [(8, 64), (128, 128), (264, 832), (4096, 4096), (10376, 2624), (1000, 8256), (2048, 16384),
         (136, 4416), (40008, 192), (40968, 2112), (600, 50048), (136, 98368), (20008, 6464), (8, 16448)]


def whole_weight(N, K, seed):
    """Random codes with scales 1/2, 1 and 2: (codes, scales for the call, decoded [N, K] doubles)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    lin = torch.randint(6, 9, (N, K // 16), device="cuda", generator=g)          # 0x30, 0x38, 0x40
    sf = bsp.nvfp4_sf_convert((lin * 8).to(torch.uint8), N, K, bsp.SF_LINEAR, bsp.SF_MMA)
    v = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float64, device="cuda")
    w = torch.stack((v[(codes & 15).long()], v[(codes >> 4).long()]), -1).view(N, K // 16, 16)
    return codes, sf, (w * torch.exp2(lin.double() - 7)[..., None]).view(N, K)


def run(x, codes, sf, w, bias=None):
    scale = torch.tensor([0.25], device="cuda")
    y = bsp.nvfp4_gemv(x, codes, sf, scale, bias=bias)
    want = (x.double() @ w.t()) * 0.25 + (0 if bias is None else bias.double())
    assert torch.equal(y, want.bfloat16())


@pytest.mark.parametrize("N,K", SIZES)
@pytest.mark.parametrize("M", [1, 3, 8, 9, 16, 17, 25, 32])
def test_whole_numbers(M, N, K):
    codes, sf, w = whole_weight(N, K, N + K + M)
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randint(-3, 4, (M, K), device="cuda", generator=g).bfloat16()
    bias = torch.randint(-9, 10, (N,), device="cuda", generator=g).bfloat16() if M % 2 else None
    run(x, codes, sf, w, bias)


@pytest.mark.parametrize("N,K", SIZES)
def test_few_columns_at_the_edges(N, K):
    """Rows that are zero but for some columns: the last 64, those around each 256-element step's end and
    around the ends of eighths, quarters and 148ths and 296ths of K; a whole step."""
    codes, sf, w = whole_weight(N, K, N + K)
    x = torch.zeros((12, K), dtype=torch.bfloat16, device="cuda")
    x[0, -64:] = 1
    x[1, -1] = 1
    x[2, 0] = 1
    x[3, 255::256], x[3, 256::256] = 1, -2
    x[4, (K - 1) // 256 * 256:] = 1                  # the last step
    x[5, :256] = 1
    for row, parts in ((6, 8), (7, 4), (8, 148), (9, 296)):
        for i in range(1, parts):
            at = K * i // parts // 64 * 64
            x[row, max(0, at - 1)], x[row, min(K - 1, at)] = 2, -3
    x[10, 64 * ((K // 64) // 2):][:64] = 3           # one group of scales in the middle
    x[11, 31::64] = 1
    run(x, codes, sf, w)
    for m in range(x.shape[0]):                      # alone: another piece of K has all of the row's size
        run(x[m:m + 1], codes, sf, w)


def check(y, x, codes, sf, g, bias=None):
    N, K = codes.shape[0], 2 * codes.shape[1]
    w, xd = decode(codes, sf, N, K) * g.double().cpu(), x.cpu().double()
    want, S = xd @ w.t(), xd.abs() @ w.abs().t()
    top = xd.abs().amax(1, keepdim=True)
    b = torch.zeros(N, dtype=torch.float64) if bias is None else bias.cpu().double()
    bound = (want + b).abs() * 2.0 ** -8 + want.abs() * 2.0 ** -22 + b.abs() * 2.0 ** -23
    bound += (K / 64 + 8) * 2.0 ** -22 * S + 64 * 2.0 ** -24 * S + 2.0 ** -39 * top * w.abs().sum(1)
    d = (y.cpu().double() - want - b).abs()
    assert (d <= bound).all(), float((d / bound.clamp(min=1e-300)).max())


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (7, 10376, 2624), (16, 264, 12288), (32, 1000, 8256),
                                   (9, 40968, 2112), (24, 2048, 16384), (3, 136, 98368), (5, 8, 64)])
def test_present_bound(M, N, K):
    codes, sf, g = weight(N, K, N + K)
    x = synth.bf16_normal((M, K), 1.0, M, 0.01, 30.0).cuda()
    bias = synth.bf16_normal((N,), 0.1, 7).cuda()
    check(bsp.nvfp4_gemv(x, codes, sf, g, bias=bias), x, codes, sf, g, bias)


@pytest.mark.parametrize("N,K", [(136, 320), (4096, 4096), (2048, 16384), (40968, 2112)])
@pytest.mark.parametrize("power", [10, 20, 27, 28, 30, 34, 38, 60])
def test_a_huge_element_against_a_zero_weight(N, K, power):
    """x[k] = 2^power where column k of the weight is zero: the other elements make the result."""
    codes, sf, g = weight(N, K, 3 * N + K)
    x = synth.bf16_normal((3, K), 1.0, power).cuda()
    for m, k in enumerate((0, K // 2 + 1, K - 1)):
        x[m, k] = 2.0 ** power
        codes[:, k // 2] &= 0xF0 if k % 2 == 0 else 0x0F
    check(bsp.nvfp4_gemv(x, codes, sf, g), x, codes, sf, g)


def test_elements_of_any_size_are_held():
    """Each row one-hot but for a huge element against a zero column: down to 2^-28 of the largest the
    output is exact, below that it is off by at most 2^-39 of the largest."""
    N, K = 64, 512
    codes, sf, w = whole_weight(N, K, 5)
    codes[:, 0] &= 0xF0
    w[:, 0] = 0
    scale = torch.tensor([0.25], device="cuda")
    for power in range(0, 45):
        x = torch.zeros((2, K), dtype=torch.bfloat16, device="cuda")
        x[:, 0] = 1.0
        x[0, 300], x[1, 37] = 1.6640625 * 2.0 ** -power, -1.3359375 * 2.0 ** -power      # eight bits
        y = bsp.nvfp4_gemv(x, codes, sf, scale).double()
        want = (x.double() @ w.t()) * 0.25
        if power <= 27:                              # the element itself is at least 2^-27 of the largest
            assert torch.equal(y, want.bfloat16().double()), power
        else:
            assert ((y - want).abs() <= want.abs() * 2.0 ** -8 + 2.0 ** -39 * 0.25 * 12).all(), power
