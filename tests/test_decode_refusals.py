"""Refusals of the decode operators' binding, on the CPU."""
import pytest
import torch

import block_scaled_precision_act_b200 as bsp


def test_a_cache_without_heads_is_refused():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    kv = (u8(9, 0, 32, 64), u8(9, 0, 32, 64), u8(9, 0, 2), u8(9, 0, 2), i32(2, 4), i32(3), i32(2))
    for heads in (0, 8):
        with pytest.raises(bsp.BSPError):
            bsp.fp8kv_attention(torch.zeros((5, heads, 64), dtype=torch.bfloat16), *kv)
