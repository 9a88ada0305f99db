"""Arguments of the mixer's operators that are no tensors are refused as such, by name."""
import pytest
import torch

from selective_state_space_sscan_amd import sscan
from test_gpu_delta import DEV, inputs, on, state

pytestmark = pytest.mark.gpu

BAD = [None, [1.0], 3.0, torch.zeros(2).numpy()]


def refused(call, kw, names, bad):
    call(**kw)
    for name in names:
        with pytest.raises((TypeError, ValueError), match=rf"\b{name}\b"):
            call(**dict(kw, **{name: bad}))


@pytest.mark.parametrize("bad", BAD)
def test_delta(bad):
    names = ("q", "k", "v", "g", "beta")
    ins = dict(zip(names, on(*inputs(1, 20, 1, 2, 64, 64, torch.float32))))
    refused(sscan.delta_fwd, ins, names, bad)
    refused(sscan.delta_bwd, dict(ins, dout=torch.zeros(1, 20, 2, 64, device=DEV)), names + ("dout",) * (bad is not None), bad)
    one = {n: x[:, 0].contiguous() for n, x in ins.items()}
    refused(sscan.delta_step, dict(one, state=state(1, 2, 64, 64).to(DEV)), names + ("state",), bad)
    if bad is not None:
        refused(sscan.delta_fwd, ins, ("h0", "lengths", "out", "h_last"), bad)


@pytest.mark.parametrize("bad", BAD)
def test_norms(bad):
    x, w = torch.randn(3, 64, device=DEV), torch.ones(64, device=DEV)
    optional = bad is None
    refused(sscan.gated_norm, dict(x=x, z=x, weight=w), ("x", "z") if optional else ("x", "z", "weight", "out"), bad)
    refused(sscan.gated_norm_bwd, dict(x=x, z=x, dout=x, weight=w), ("x", "z") if optional else ("x", "z", "dout", "weight"), bad)
    refused(sscan.add_norm, dict(x=x, residual=x, weight=w),
            ("x",) if optional else ("x", "residual", "weight", "scale", "post_weight", "out", "residual_out"), bad)
    refused(sscan.add_norm_bwd, dict(x=x, residual_out=x, dout=x, weight=w),
            ("x",) if optional else ("x", "dout", "weight", "scale", "post_weight"), bad)
