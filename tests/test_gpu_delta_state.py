"""States of the gated delta rule: what a non-finite one reaches, states that are slices of
a pool."""
import pytest
import torch

import delta_ref
from delta_ref import close
from selective_state_space_sscan_amd import sscan
from test_gpu_delta import DEV, inputs, on, state
from test_gpu_delta_bwd import NAMES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("L,m", [(9, 4), (100, 70), (1300, 650), (1300, 0)])
def test_a_non_finite_state_stays_inside_the_rows_length(L, m, bad, dtype):
    """Tokens past a row's length answer 0 and have no gradient, whatever its state; the
    state's other value columns are as if it were finite."""
    ins = inputs(2, L, 1, 2, 64, 64, dtype, seed=5, g_scale=0.05)
    h0 = state(2, 2, 64, 64)
    h0[0, 1, 3, 17] = bad
    n = torch.tensor([m, L], dtype=torch.int32)
    out, last = sscan.delta_fwd(*on(*ins), *on(h0, n))
    assert not out[0, m:].any()
    clean = state(2, 2, 64, 64)
    clean[0, 1, :, 17] = 0.0
    ref, ref_last = delta_ref.delta(*ins, clean, n)
    others = [c for c in range(64) if c != 17]
    close(out[..., others], ref[..., others], "out")
    close(last[..., others], ref_last[..., others], "h_last")
    if m:
        assert not torch.isfinite(out[0, :m, 1, 17]).any()
    dout = torch.randn(2, L, 2, 64, generator=torch.Generator().manual_seed(1)).to(dtype)
    r = sscan.delta_bwd(*on(*ins, dout), h0=h0.to(DEV), lengths=n.to(DEV))
    for name in NAMES[:5]:
        assert not r[name][0, m:].any(), name
        assert torch.isfinite(r[name][1]).all(), name
