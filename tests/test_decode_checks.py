"""Refusals of nvfp4_gemv, fp8kv_append and fp8kv_attention, on the CPU: the C calls' argument
checks (fake addresses, nothing is launched), and the binding's checks of shapes, dtypes and
sizes (tensors of exactly the right sizes are refused only for being on the CPU)."""
import pytest
import torch

import block_scaled_precision_act_b200 as bsp
from block_scaled_precision_act_b200.nn import QuantLinear

OK, INVALID, SHAPE, MISALIGNED = 0, -1, -2, -3
P = 1 << 20
ON_CPU = "not on a CUDA device"


def test_gemv_host_checks():
    g = bsp.lib().nvfp4_gemv
    base = dict(x=P, c=P, s=P, g=P, b=None, o=P, M=1, N=64, K=128, ws=P, wsb=1 << 30)

    def call(**kw):
        a = {**base, **kw}
        return g(a["x"], a["c"], a["s"], a["g"], a["b"], a["o"], a["M"], a["N"], a["K"], a["ws"],
                 a["wsb"], None)

    need = bsp.nvfp4_gemv_workspace_bytes(1, 64, 128)
    assert call(ws=None) == INVALID and call(wsb=need - 1) == INVALID and call(ws=P + 8) == MISALIGNED
    size = bsp.lib().nvfp4_gemv_workspace_bytes
    assert size(33, 64, 128) == SHAPE and size(-1, 64, 128) == INVALID and size(1, 64, 96) == SHAPE
    for name in "xcsgo":
        assert call(**{name: None}) == INVALID
        assert call(**{name: P + (2 if name == "g" else 8)}) == MISALIGNED
    assert call(b=P + 8) == MISALIGNED
    assert call(M=-1) == INVALID and call(N=-8) == INVALID
    assert call(M=33) == SHAPE and call(N=12) == SHAPE and call(K=96) == SHAPE and call(K=0) == SHAPE
    assert call(M=0, x=None, o=None) == OK and call(N=0, c=None) == OK


def test_gemv_binding_checks():
    M, N, K = 3, 40, 128
    ok = dict(x=torch.zeros((M, K), dtype=torch.bfloat16),
              w_codes=torch.zeros((N, K // 2), dtype=torch.uint8),
              w_sf=torch.zeros((bsp.nvfp4_sf_bytes(N, K),), dtype=torch.uint8),
              w_scale=torch.ones(()), bias=torch.zeros((N,), dtype=torch.bfloat16),
              out=torch.zeros((M, N), dtype=torch.bfloat16),
              workspace=torch.zeros((bsp.nvfp4_gemv_workspace_bytes(M, N, K),), dtype=torch.uint8))
    with pytest.raises(bsp.BSPError, match=ON_CPU):
        bsp.nvfp4_gemv(**ok)
    for name, bad in [("w_sf", ok["w_sf"][:-1]), ("bias", ok["bias"][:-8]), ("out", ok["out"][:2])]:
        with pytest.raises(bsp.BSPError, match="needs"):
            bsp.nvfp4_gemv(**{**ok, name: bad})
    for name in ("x", "w_codes", "w_scale", "bias", "out", "workspace"):
        with pytest.raises(TypeError):
            bsp.nvfp4_gemv(**{**ok, name: ok[name].to(torch.float64)})
    with pytest.raises(bsp.BSPError, match="columns"):
        bsp.nvfp4_gemv(**{**ok, "x": torch.zeros((M, K + 64), dtype=torch.bfloat16)})


APPEND = ["q", "qs", "k", "ks", "v", "vs", "f", "rot", "inter", "rs", "qo", "kc", "vc", "ksc", "vsc",
          "pages", "page", "table", "max_pages", "cu", "len", "B", "T", "Hq", "Hkv", "D"]
ATTEND = ["q", "qs", "kc", "vc", "ksc", "vsc", "pages", "page", "table", "max_pages", "cu", "len", "B",
          "T", "Hq", "Hkv", "D", "sm", "window", "o", "lse", "ws", "wsb"]
BASE = dict(q=P, qs=512, k=P, ks=128, v=P, vs=128, f=P, rot=64, inter=0, rs=1.0, qo=P, kc=P, vc=P,
            ksc=P, vsc=P, pages=9, page=32, table=P, max_pages=4, cu=P, len=P, B=2, T=5, Hq=8, Hkv=2,
            D=64, sm=0.1, window=0, o=P, lse=None, ws=P, wsb=1 << 30)


def append(**kw):
    a = {**BASE, **kw}
    return bsp.lib().fp8kv_append(*[a[x] for x in APPEND], None)


def attend(**kw):
    a = {**BASE, **kw}
    return bsp.lib().fp8kv_attention(*[a[x] for x in ATTEND], None)


@pytest.mark.parametrize("call", [append, attend])
def test_cache_host_checks(call):
    for name in ("kc", "vc", "ksc", "vsc", "table", "cu", "len"):
        assert call(**{name: None}) == INVALID, name
    for name in ("kc", "vc", "q"):
        assert call(**{name: P + 8}) == MISALIGNED, name
    for name in ("table", "cu", "len"):
        assert call(**{name: P + 2}) == MISALIGNED, name
    for name in ("B", "T", "pages", "max_pages", "Hq"):
        assert call(**{name: -1}) == INVALID, name
    assert call(Hkv=0) == INVALID and call(D=0) == INVALID and call(page=0) == INVALID
    assert call(pages=0) == INVALID and call(max_pages=0) == INVALID
    assert call(qs=511) == INVALID and call(qs=516) == SHAPE
    assert call(D=72) == SHAPE and call(D=272) == SHAPE and call(page=24) == SHAPE
    assert call(page=8192) == SHAPE and call(Hq=7) == SHAPE and call(B=1 << 21) == SHAPE
    assert call(T=1 << 25) == SHAPE
    assert call(T=0, q=None, kc=None) == OK and call(B=0, q=None, kc=None) == OK


def test_append_host_checks():
    assert append(k=None) == INVALID and append(v=None) == INVALID and append(f=None) == INVALID
    assert append(qo=None) == INVALID and append(inter=2) == INVALID and append(rot=-16) == INVALID
    assert append(ks=120) == INVALID and append(vs=132) == SHAPE
    assert append(rot=24) == SHAPE and append(rot=80) == SHAPE
    for name in ("k", "v", "qo"):
        assert append(**{name: P + 8}) == MISALIGNED
    assert append(f=P + 2) == MISALIGNED


def test_attention_host_checks():
    assert attend(q=None) == INVALID and attend(o=None) == INVALID and attend(window=-1) == INVALID
    assert attend(Hq=0) == INVALID
    assert attend(o=P + 8) == MISALIGNED and attend(lse=P + 2) == MISALIGNED
    need = bsp.fp8kv_attention_workspace_bytes(5, 8, 2, 64)
    assert attend(ws=None) == INVALID and attend(wsb=need - 1) == INVALID
    assert attend(ws=P + 8) == MISALIGNED
    size = bsp.lib().fp8kv_attention_workspace_bytes
    assert size(-1, 8, 2, 64) == INVALID and size(5, 7, 2, 64) == INVALID and size(5, 8, 2, 72) == SHAPE


def kv_tensors():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return dict(k_cache=u8(9, 2, 32, 64), v_cache=u8(9, 2, 32, 64), k_scale=u8(9, 2, 2),
                v_scale=u8(9, 2, 2), block_table=i32(2, 4), cu_new=i32(3), kv_len=i32(2))


def bf16(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def test_cache_binding_checks():
    kv = kv_tensors()
    calls = [lambda t: bsp.fp8kv_append(bf16(5, 2, 64), bf16(5, 2, 64), **t, q=bf16(5, 8, 64),
                                        inv_freq=torch.ones(32)),
             lambda t: bsp.fp8kv_attention(bf16(5, 8, 64), **t,
                                           workspace=torch.zeros(1 << 20, dtype=torch.uint8))]
    for call in calls:
        with pytest.raises(bsp.BSPError, match=ON_CPU):
            call(kv)
        for name in kv:
            with pytest.raises(TypeError):
                call({**kv, name: kv[name].float()})
            with pytest.raises(TypeError):
                call({**kv, name: None})
        for name in ("k_scale", "v_scale", "cu_new", "kv_len"):
            with pytest.raises(bsp.BSPError, match="needs"):
                call({**kv, name: kv[name].view(-1)[:-1]})
        with pytest.raises(bsp.BSPError, match="shape"):
            call({**kv, "v_cache": kv["v_cache"][:8]})
        with pytest.raises(bsp.BSPError, match="page_size"):
            call({**kv, "k_cache": kv["k_cache"][0]})
        with pytest.raises(bsp.BSPError, match="2-D"):
            call({**kv, "block_table": kv["block_table"].view(-1)})


def test_head_binding_checks():
    kv = kv_tensors()
    k = bf16(5, 2, 64)
    for bad in (bf16(4, 2, 64), bf16(5, 2, 32), bf16(5, 128), bf16(5, 3, 64),
                bf16(5, 64, 2).transpose(1, 2), bf16(2, 5, 64).transpose(0, 1)):
        with pytest.raises(bsp.BSPError):
            bsp.fp8kv_append(k, bad, **kv)
    with pytest.raises(bsp.BSPError, match="multiple"):
        bsp.fp8kv_attention(bf16(5, 7, 64), **kv)
    with pytest.raises(TypeError):
        bsp.fp8kv_append(k.float(), k, **kv)
    with pytest.raises(bsp.BSPError, match="needs"):
        bsp.fp8kv_append(k, k, **kv, q=bf16(5, 8, 64), q_out=bf16(4, 8, 64))
    with pytest.raises(bsp.BSPError, match="needs"):
        bsp.fp8kv_attention(bf16(5, 8, 64), **kv, out=bf16(4, 8, 64))
    with pytest.raises(bsp.BSPError, match="needs"):
        bsp.fp8kv_attention(bf16(5, 8, 64), **kv, lse=torch.zeros(5, 7))


def test_quant_linear_weight_only_rows():
    m = QuantLinear(64, 16, "nvfp4")
    assert m.weight_only_rows == 0 and "weight_only_rows" not in m.state_dict()
    assert QuantLinear(64, 16, "nvfp4", weight_only_rows=4).weight_only_rows == 4
    with pytest.raises(ValueError):
        QuantLinear(64, 16, "nvfp4", weight_only_rows=33)
    with pytest.raises(ValueError):
        QuantLinear(64, 16, "fp8r", weight_only_rows=4)


def test_paged_kv_cache_module():
    from block_scaled_precision_act_b200.nn import PagedKVCache
    c = PagedKVCache(5, 2, 64, page_size=32)
    assert c.k_cache.shape == c.v_cache.shape == (5, 2, 32, 64) and c.k_scale.shape == (5, 2, 2)
    assert not c.state_dict() and "page_size=32" in repr(c)
    for bad in (dict(head_dim=72), dict(head_dim=272), dict(page_size=24), dict(num_pages=0),
                dict(num_heads=0), dict(page_size=8192)):
        with pytest.raises(ValueError):
            PagedKVCache(**{**dict(num_pages=5, num_heads=2, head_dim=64), **bad})
    with pytest.raises(bsp.BSPError, match=ON_CPU):
        c.append(bf16(1, 2, 64), bf16(1, 2, 64), *[torch.zeros(s, dtype=torch.int32)
                                                  for s in ((1, 1), (2,), (1,))])


@pytest.mark.parametrize("call", [append, attend])
def test_tables_past_2_to_30_tokens(call):
    assert call(max_pages=(1 << 25) + 1) == SHAPE           # pages of 32
    assert call(max_pages=1 << 40) == SHAPE
