"""8-bit-float layers without a GPU: sizes that the products' 32-bit counts do
not hold."""
import ctypes

import numpy as np
import pytest


def _handle(N, K):
    """The host-side fields of a handle (n_experts, N, K, tiles, blocks, device, SMs), which the refusals read."""
    raw = np.zeros(256, np.int64)
    raw.view(np.int32)[:7] = [1, N, K, -(-N // 128), -(-K // 128), 0, 148]
    return raw


@pytest.mark.parametrize("M", [2**31 - 1, 2**31 - 2, 2**31 - 16, 2**31 - 200, 2**31 - 255])
@pytest.mark.parametrize("grouped", [False, True])
def test_rows_next_to_2_31_are_refused(M, grouped):
    """Rounding M up to a block of 16 .. 256 rows would leave 32 bits."""
    import vq_compressed_linear_b200 as m
    raw = _handle(1, 16)
    buf = np.zeros(64, np.float64)
    p = ctypes.c_void_p((buf.ctypes.data + 15) // 16 * 16)
    h = ctypes.c_void_p(raw.ctypes.data)
    if grouped:
        rc = m.lib.hxq_fp8_forward_grouped(h, p, p, p, None, p, 0, M, None)
    else:
        rc = m.lib.hxq_fp8_forward(h, p, p, None, p, 0, M, None)
    assert rc == m.HXQ_EINVAL


@pytest.mark.parametrize("bad", [dict(h=False), dict(stage=-2), dict(limit=0), dict(limit=2000001), dict(M=-1),
                                 dict(x=False)], ids=str)
def test_withheld_hook_refuses(bad):
    import vq_compressed_linear_b200 as m
    a = {**dict(h=True, stage=1, limit=1000, M=4, x=True), **bad}
    raw = _handle(1, 16)
    buf = np.zeros(64, np.float64)
    p = ctypes.c_void_p((buf.ctypes.data + 15) // 16 * 16)
    h = ctypes.c_void_p(raw.ctypes.data) if a["h"] else None
    assert m.lib.hxq_test_fp8_forward_withheld(h, p if a["x"] else None, p, None, p, a["M"], a["stage"], a["limit"],
                                               None) == m.HXQ_EINVAL
