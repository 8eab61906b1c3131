"""The binding's two ways to the decode operators, the compiled short cut and the Python code, give the
same results and refuse the same calls with the same errors."""
import numpy as np
import pytest
import torch

import block_scaled_precision_act_b200 as bsp
import synth
from kv_reference import Batch

pytestmark = pytest.mark.gpu
POOL = ("k_cache", "v_cache", "k_scale", "v_scale", "block_table", "cu_new", "kv_len")


class Unclear:
    """Neither true nor false."""

    def __bool__(self):
        raise ValueError("neither true nor false")

    def __int__(self):
        raise ValueError("neither true nor false")


@pytest.fixture(params=[True, False], ids=["compiled", "python"])
def way(request, monkeypatch):
    bsp.lib()
    assert bsp._fastcall is not None
    if not request.param:
        monkeypatch.setattr(bsp, "_fastcall", None)


def kv(seed=1, Hkv=2):
    b = Batch([3, 1], [40, 70], 8, Hkv, 64, 32, seed=seed)
    return b, b.to("cuda")


def test_arguments_without_a_truth_value(way):
    b, d = kv()
    with pytest.raises(ValueError, match="neither"):
        bsp.fp8kv_append(b.k.cuda(), b.v.cuda(), **d, interleaved=Unclear())
    with pytest.raises(ValueError, match="neither"):
        bsp.fp8kv_attention(b.q.cuda(), **d, return_lse=Unclear())
    with pytest.raises((ValueError, RuntimeError)):
        bsp.fp8kv_attention(b.q.cuda(), **d, return_lse=torch.ones(3))
    with pytest.raises((ValueError, TypeError)):
        bsp.fp8kv_append(b.k.cuda(), b.v.cuda(), **d, interleaved=np.ones(3))


def gemv_operands(M=5, N=136, K=320):
    w = synth.bf16_normal((N, K), 0.02, 1).cuda()
    g = bsp.nvfp4_global_scale(w)
    codes, sf = bsp.nvfp4_quantize_act(w, g)
    return dict(x=synth.bf16_normal((M, K), 1.0, 2).cuda(), w_codes=codes, w_sf=sf, w_scale=g,
                bias=synth.bf16_normal((N,), 0.1, 3).cuda())


def test_the_same_results(monkeypatch):
    bsp.lib()
    assert bsp._fastcall is not None
    b, d = kv()
    f = (10000.0 ** (-torch.arange(0, 64, 2) / 64)).cuda()

    def everything():
        dd = {k: v.clone() for k, v in d.items()}
        g = gemv_operands()
        r = [bsp.nvfp4_gemv(**g), bsp.nvfp4_gemv(**{**g, "bias": None, "out": torch.empty_like(g["x"][:, :136])})]
        r.append(bsp.fp8kv_append(b.k.cuda(), b.v.cuda(), **dd, q=b.q.cuda(), inv_freq=f, rope_scale=1.5,
                                  interleaved=True))
        assert bsp.fp8kv_append(b.k.cuda(), b.v.cuda(), **dd) is None
        r += list(dd.values())
        o, lse = bsp.fp8kv_attention(b.q.cuda(), **dd, return_lse=True)
        given = torch.empty_like(lse)
        r += [o, lse, bsp.fp8kv_attention(b.q.cuda(), **dd, sm_scale=0.3, window=9, lse=given), given]
        out = torch.empty_like(o)
        assert bsp.fp8kv_attention(b.q.cuda(), **dd, out=out) is out
        return r + [out]

    compiled = everything()
    monkeypatch.setattr(bsp, "_fastcall", None)
    python = everything()
    torch.cuda.synchronize()
    assert len(compiled) == len(python)
    for x, y in zip(compiled, python):
        assert x.dtype == y.dtype and x.shape == y.shape and torch.equal(x, y)


def test_the_same_refusals(way):
    g = gemv_operands()
    bad = {"x": [g["x"].float(), g["x"][0], g["x"][:, ::2], g["x"].cpu(), g["x"][:, :288].contiguous()],
           "w_codes": [g["w_codes"].int(), g["w_codes"][:, :-32].contiguous(), g["w_codes"][:-1], None],
           "w_sf": [g["w_sf"].view(-1)[:-1], g["w_sf"].float(), g["w_sf"].cpu()],
           "w_scale": [g["w_scale"].double(), g["w_scale"][:0], g["w_scale"].cpu()],
           "bias": [g["bias"][:-1], g["bias"].float(), g["bias"].cpu(), g["bias"].repeat(2)[::2]],
           "out": [g["x"][:1], torch.empty((5, 136), device="cuda")],
           "workspace": [torch.empty(16, dtype=torch.uint8, device="cuda"),
                         torch.empty(1 << 22, dtype=torch.int8, device="cuda"),
                         torch.empty((1 << 22) + 8, dtype=torch.uint8, device="cuda")[8:]]}
    for name, values in bad.items():
        for v in values:
            with pytest.raises((bsp.BSPError, TypeError)):
                bsp.nvfp4_gemv(**{**g, name: v})
    b, d = kv()
    k, v, q = b.k.cuda(), b.v.cuda(), b.q.cuda()
    for name in POOL:
        # a table without rows is a batch without sequences, which is fine
        for x in (d[name].float(), d[name].cpu(), None, d[name][:0] if name != "block_table" else None):
            with pytest.raises((bsp.BSPError, TypeError)):
                bsp.fp8kv_append(k, v, **{**d, name: x})
            with pytest.raises((bsp.BSPError, TypeError)):
                bsp.fp8kv_attention(q, **{**d, name: x})
    wrong = dict(k=[k.float(), k[:3], k[:, :1], k[..., :32], k.cpu(), k.transpose(0, 1).contiguous().transpose(0, 1)],
                 v=[v[:3], v.float()], q=[q[:3], q[..., :32], q[:, :7], q.cpu(), q.float()],
                 q_out=[q[:2], q.float(), q.repeat(1, 2, 1)[:, ::2]],
                 inv_freq=[torch.ones(33, device="cuda"), torch.ones(20, device="cuda"), torch.ones(8)])
    for name, values in wrong.items():
        for x in values:
            with pytest.raises((bsp.BSPError, TypeError)):
                bsp.fp8kv_append(**{**dict(k=k, v=v, q=q), name: x}, **d)
    for kw in (dict(window=-1), dict(out=q[:2]), dict(lse=torch.empty(3, device="cuda")), dict(lse=q),
               dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((bsp.BSPError, TypeError)):
            bsp.fp8kv_attention(q, **d, **kw)
    for x in wrong["q"][1:]:
        with pytest.raises((bsp.BSPError, TypeError)):
            bsp.fp8kv_attention(x, **d)
    torch.cuda.synchronize()
    assert bsp.bsp_last_device_status() == 0
