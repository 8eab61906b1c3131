"""fp8kv_append to blocks whose scale byte it would not have made (above 246)."""
import pytest

import block_scaled_precision_act_b200 as bsp
from kv_reference import Batch
from test_gpu_fp8kv_append import call, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("byte", [245, 246, 247, 250, 253, 254, 255])
@pytest.mark.parametrize("n,L", [([3], [20]), ([20, 1], [25, 8]), ([1], [16])])
def test_a_block_keeps_the_larger_byte(byte, n, L):
    """The earlier tokens' values stay: neither their codes nor their scale change."""
    b = Batch(n, L, 4, 2, 64, 16, seed=byte)
    b.k_scale[:], b.v_scale[:] = byte, byte
    b.v[0, 0, 3] = 2.0 ** 118                        # a code other than 0 beside it
    q, got = call(b, 32)
    check(b, q, got, 32)
    assert bsp.bsp_last_device_status() == 0
