"""What autograd has to know of the mixer's operators: which tensors are written in place, and
that the gradients have none of their own."""
import pytest
import torch

from selective_state_space_sscan_amd import sscan
from test_gpu_delta import DEV, inputs, on, state

pytestmark = pytest.mark.gpu


def some(L=20):
    return on(*inputs(1, L, 1, 2, 64, 64, torch.float32, seed=1))


def test_a_saved_state_that_is_stepped_is_noticed():
    ins, s = some(), state(1, 2, 64, 64).to(DEV)
    v = ins[2].requires_grad_(True)
    out, _ = sscan.gated_delta(*ins, h0=s)
    with torch.no_grad():
        sscan.delta_step(s, *[x[:, 0] for x in ins])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(out.sum(), [v])


@pytest.mark.parametrize("L", [5, 100])
def test_a_saved_state_handed_on_in_place_is_noticed(L):
    ins, s = some(L), state(1, 2, 64, 64).to(DEV)
    v = ins[2].requires_grad_(True)
    out, _ = sscan.gated_delta(*ins, h0=s)
    with torch.no_grad():
        sscan.delta_fwd(*ins, h0=s, h_last=s)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(out.sum(), [v])


def test_every_tensor_given_to_write_to_counts():
    ins, s = some(), state(1, 2, 64, 64).to(DEV)
    one = [x[:, 0].contiguous() for x in ins]
    x, w = torch.randn(3, 2, 64, device=DEV), torch.ones(64, device=DEV)
    o4, o3, y, total = (torch.empty(n, device=DEV) for n in ((1, 20, 2, 64), (1, 2, 64), (3, 2, 64), (3, 2, 64)))
    res = x.clone()
    for call, written in (
            (lambda: sscan.delta_fwd(*ins, out=o4), [o4]), (lambda: sscan.delta_fwd(*ins, h_last=s), [s]),
            (lambda: sscan.delta_step(s, *one, out=o3), [s, o3]), (lambda: sscan.gated_norm(x, x, w, out=y), [y]),
            (lambda: sscan.add_norm(x, res, w, out=y, residual_out=res), [y, res]),
            (lambda: sscan.add_norm(x, res, w, residual_out=total), [total])):
        before = [t._version for t in written]
        kept = [t._version for t in (*ins, x, w)]
        call()
        assert all(t._version > v for t, v in zip(written, before))
        assert [t._version for t in (*ins, x, w)] == kept


def test_states_of_inference_mode():
    with torch.inference_mode():
        s = state(1, 2, 64, 64).to(DEV)
    t = s.clone()
    one = [x[:, 0].contiguous() for x in some()]
    assert torch.equal(sscan.delta_step(s, *one), sscan.delta_step(t, *one)) and torch.equal(s, t)


def test_second_derivatives_are_refused():
    ins = [x.requires_grad_(True) for x in some()]
    x, z = (torch.randn(5, 64, device=DEV, requires_grad=True) for _ in range(2))
    w = torch.ones(64, device=DEV, requires_grad=True)
    for f, at in ((lambda: sscan.gated_delta(*ins)[0], ins[0]), (lambda: sscan.gated_rms_norm(x, z, w), x),
                  (lambda: sscan.add_rms_norm(x, z, w)[0], x)):
        for loss in (lambda: f().square().sum(), lambda: f().sum()):
            (want,) = torch.autograd.grad(loss(), [at])
            (g,) = torch.autograd.grad(loss(), [at], create_graph=True)
            assert torch.equal(g, want)
            with pytest.raises(RuntimeError, match="no second derivatives"):
                torch.autograd.grad(g.sum() + at.square().sum(), [at])
