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
