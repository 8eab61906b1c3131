"""Batches that hold what they must not, with every array inside a larger one: nothing outside the arrays,
no unused page and no block that the batch does not append to changes, and the status is the documented one.

Rows outside [0, T) are cut off and a descending pair of cu_new is no rows.  Of a sequence with new tokens
whose length does not fit, fp8kv_append stores nothing and fp8kv_attention reads what the table holds."""
import pytest
import torch

import block_scaled_precision_act_b200 as bsp
from kv_reference import Batch
from test_gpu_fp8kv_append import check as check_append, inv_freq
from test_gpu_fp8kv_attention import check as check_attention
from test_gpu_guard import Guarded

pytestmark = pytest.mark.gpu
POOL = ("k_cache", "v_cache", "k_scale", "v_scale")
META = ("block_table", "cu_new", "kv_len")

# cu_new, kv_len; what they come to: rows and length of each sequence; status of append and of attention
BATCHES = [
    ([0, 400, 9], [20, 20], [(0, 8, 20), (8, 0, 20)], 0, 0),
    ([5, 2, -3], [20, 20], [(5, 0, 20), (2, 0, 20)], 0, 0),
    ([-7, 3, 3], [20, 20], [(0, 3, 20), (3, 0, 20)], 0, 0),
    ([0, 4, 8], [3, -9], [(0, 4, 3), (4, 4, 0)], -1, -1),
    ([0, 4, 8], [2 ** 31 - 1, 20], [(0, 4, 32), (4, 4, 20)], -1, -1),
    ([0, 4, 8], [33, 32], [(0, 4, 32), (4, 4, 32)], -1, -1),
    ([0, 4, 8], [20, -2 ** 31], [(0, 4, 20), (4, 4, 0)], -1, -1),
]


class Arrays:
    """A batch's arrays inside guard bands."""

    def __init__(self, b):
        self.g, self.t = {}, {}
        dev = b.to("cuda")
        for x in POOL + META:
            self.add(x, dev[x])
        for x in "qkv":
            self.add(x, getattr(b, x).cuda())
        self.add("q_out", torch.full_like(b.q, 7.0).cuda())
        self.add("out", torch.full_like(b.q, 7.0).cuda())
        self.add("lse", torch.full(b.q.shape[:2], 7.0, device="cuda"))
        need = bsp.fp8kv_attention_workspace_bytes(b.T, b.Hq, b.Hkv, b.D)
        self.add("workspace", torch.zeros(need, dtype=torch.uint8, device="cuda"))

    def add(self, name, value):
        self.g[name] = Guarded(value.numel() * value.element_size())
        self.t[name] = self.g[name].view(value.dtype, value.shape)
        self.t[name].copy_(value)

    def intact(self):
        return [x for x, g in self.g.items() if not g.intact()]


def batch(cu, lens, means, D, Hq):
    b = Batch([4, 4], [20, 20], Hq, 2, D, 16, seed=8)
    b.cu, b.kv_len = torch.tensor(cu, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32)
    return b


def effective(b, means):
    """What the batch comes to, for the reference: rows of a sequence that has none are not looked at."""
    b.cu = torch.tensor([m[0] for m in means] + [means[-1][0] + means[-1][1]], dtype=torch.int32)
    b.n, b.lens = [m[1] for m in means], [m[2] for m in means]


@pytest.mark.parametrize("case", BATCHES, ids=lambda c: f"{c[0]}-{c[1]}")
@pytest.mark.parametrize("D,Hq", [(64, 2), (128, 8), (256, 4)])
def test_append(case, D, Hq):
    cu, lens, means, status, _ = case
    b = batch(cu, lens, means, D, Hq)
    a = Arrays(b)
    t = a.t
    bsp.fp8kv_append(t["k"], t["v"], *[t[x] for x in POOL + META], q=t["q"], q_out=t["q_out"],
                     inv_freq=inv_freq(D).cuda())
    torch.cuda.synchronize()
    assert bsp.bsp_last_device_status() == status and bsp.bsp_last_device_status() == 0
    assert a.intact() == []
    # a sequence of a bad length: neither stored nor, in q_out, rotated
    cap = b.table.shape[1] * 16
    bad = [not m[1] <= L <= cap for m, L in zip(means, lens)]
    effective(b, [(r, 0 if x else n, L) for (r, n, L), x in zip(means, bad)])
    got = {x: t[x].cpu() for x in POOL}
    touched = torch.zeros(b.T, dtype=torch.bool)
    for r, n, x in zip(b.cu.tolist(), b.n, bad):
        touched[r:r + n] = True
    assert (t["q_out"].cpu()[~touched] == 7.0).all()
    check_append(b, t["q_out"], got, D)


@pytest.mark.parametrize("case", BATCHES, ids=lambda c: f"{c[0]}-{c[1]}")
@pytest.mark.parametrize("D,Hq", [(64, 2), (128, 8), (256, 4)])
def test_attention(case, D, Hq):
    cu, lens, means, _, status = case
    b = batch(cu, lens, means, D, Hq)
    a = Arrays(b)
    t = a.t
    bsp.fp8kv_attention(t["q"], *[t[x] for x in POOL + META], out=t["out"], lse=t["lse"],
                        workspace=t["workspace"])
    torch.cuda.synchronize()
    assert bsp.bsp_last_device_status() == status and bsp.bsp_last_device_status() == 0
    assert a.intact() == []
    for x in POOL:
        assert torch.equal(t[x].cpu(), getattr(b, x)), x
    effective(b, means)
    rows = [r + i for r, n, _ in means for i in range(n)]
    rest = [r for r in range(b.T) if r not in rows]
    assert (t["out"].cpu()[rest] == 7.0).all() and (t["lse"].cpu()[rest] == 7.0).all()
    check_attention(b, t["out"], t["lse"], rows=rows)
