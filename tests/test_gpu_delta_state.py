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


def pool(n, hv, dk, dv):
    """States one after the other: of 33 x 50 floats, every other one is off a 16-byte boundary."""
    return 0.5 * torch.randn(n, 1, hv, dk, dv, generator=torch.Generator().manual_seed(3))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L", [7, 100, 1300])
def test_states_sliced_from_a_pool(L, dtype):
    ins = inputs(1, L, 1, 1, 33, 50, dtype, seed=L, g_scale=0.05)
    states = pool(3, 1, 33, 50)
    ref, ref_last = delta_ref.delta(*ins, states[1])
    at = states.to(DEV)
    assert at[1].data_ptr() % 16
    out, last = sscan.delta_fwd(*on(*ins), h0=at[1])
    close(out, ref, "out")
    close(last, ref_last, "h_last")
    out2, same = sscan.delta_fwd(*on(*ins), h0=at[1], h_last=at[1])
    assert torch.equal(out2, out) and torch.equal(at[1], last) and same.data_ptr() == at[1].data_ptr()
    assert torch.equal(at[0].cpu(), states[0]) and torch.equal(at[2].cpu(), states[2])
    dout = torch.ones(1, L, 1, 50, dtype=dtype, device=DEV)
    back = states.to(DEV)
    a, b = (sscan.delta_bwd(*on(*ins), dout, h0=s, dh_last=s) for s in (back[1], back[1].clone()))
    for name in NAMES:
        assert torch.equal(a[name], b[name]), name


def test_tokens_from_a_pool():
    states = pool(3, 1, 33, 50)
    at = states.to(DEV)
    ins = inputs(1, 1, 1, 1, 33, 50, torch.float32, seed=4)
    ref, ref_s = delta_ref.delta(*ins, states[1])
    version = at._version
    out = sscan.delta_step(at[1], *[x[:, 0] for x in on(*ins)])
    close(out, ref[:, 0], "out")
    close(at[1], ref_s, "state")
    assert torch.equal(at[0].cpu(), states[0]) and torch.equal(at[2].cpu(), states[2]) and at._version > version
    with pytest.raises(ValueError, match="overlap"):
        sscan.delta_step(at[1], *[x[:, 0] for x in on(*ins)], out=at[1].view(-1)[:50].view(1, 1, 50))


def test_gradients_through_states_put_together():
    """The gradient of one of two states joined by torch.cat is a slice of the whole's."""
    rows = [[x.requires_grad_(True) for x in on(*inputs(1, 70, 1, 1, 33, 50, torch.float32, seed=s))] for s in (1, 2)]
    weight = torch.randn(2, 1, 33, 50, device=DEV)
    lasts = [sscan.gated_delta(*ins)[1] for ins in rows]
    got = torch.autograd.grad((torch.cat(lasts) * weight).sum(), [x for ins in rows for x in ins[1:]])
    want = []
    for ins, w in zip(rows, weight):
        want += torch.autograd.grad((sscan.gated_delta(*ins)[1] * w).sum(), ins[1:])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
