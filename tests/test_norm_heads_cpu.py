"""How many heads the gated norm's C entry points take, without a GPU."""
import ctypes

import pytest

from test_delta_abi_cpu import ESHAPE, OK, gated, lib  # noqa: F401

I2 = ctypes.c_int64 * 2


@pytest.mark.parametrize("heads", [1 << 20, (1 << 20) + 1, 1 << 22])
def test_heads_without_a_weight_each(lib, heads):  # noqa: F811
    n = lib.sscan_gated_norm_bwd_workspace_bytes(1, heads, 4)
    assert n > 0 and (n <= 1 << 20 or heads <= 1 << 20)
    for per_head in (0, 1):
        p, r = gated(rows=1, heads=heads, size=4, per_head=per_head, x_stride=I2(0, 4), z_stride=I2(0, 4))
        want = ESHAPE if per_head and heads > 1 << 20 else OK
        assert lib.sscan_validate_gated_norm(ctypes.byref(p), r["out"]) == want
        assert lib.sscan_validate_gated_norm_bwd(ctypes.byref(p), r["dout"], r["dx"], r["dz"], r["dw"], r["ws"], n) == want
