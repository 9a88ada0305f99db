"""Gradients of the gated delta rule against differentiation of the float64 token
recurrence, and against differences of the kernels' own forward."""
import pytest
import torch

import delta_ref
from delta_ref import close
from selective_state_space_sscan_amd import sscan
from test_gpu_delta import DEV, inputs, on, state

pytestmark = pytest.mark.gpu


def reference(ins, dout, h0=None, dh=None, **kw):
    leaves = [x.double().requires_grad_(True) for x in ins]
    b, L, hk, dk = ins[0].shape
    hv, dv = ins[2].shape[2:]
    s0 = (torch.zeros(b, hv, dk, dv) if h0 is None else h0).double().requires_grad_(True)
    out, last = delta_ref.delta(*leaves, s0, **kw)
    loss = (out * dout.double()).sum() + (0 if dh is None else (last * dh.double()).sum())
    if not loss.requires_grad:
        return [torch.zeros_like(x) for x in leaves + [s0]]
    got = torch.autograd.grad(loss, leaves + [s0], allow_unused=True)
    return [torch.zeros_like(x) if g is None else g for x, g in zip(leaves + [s0], got)]


NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dh0")


def check(ins, h0=None, dh=None, lengths=None, garbage=False, **kw):
    print("delta_bwd", [tuple(x.shape) for x in ins], ins[0].dtype, kw, flush=True)
    v = ins[2]
    dout = torch.randn(v.shape, generator=torch.Generator().manual_seed(99)).to(v.dtype)
    refs = reference(ins, dout, h0, dh, lengths=lengths, **kw)
    if garbage:
        for i, m in enumerate(lengths):
            for x in list(ins) + [dout]:
                x[i, max(int(m), 0):] = float("nan")
    r = sscan.delta_bwd(*on(*ins, dout), h0=on(h0)[0], dh_last=on(dh)[0], lengths=on(lengths)[0], **kw)
    torch.cuda.synchronize()
    for name, ref in zip(NAMES, refs):
        close(r[name], ref, name)
    return r


SHAPES = [  # b, L, hk, hv, dk, dv
    (1, 1, 1, 1, 1, 1), (2, 3, 1, 2, 16, 8), (1, 8, 2, 2, 128, 128), (1, 63, 1, 3, 33, 50), (1, 64, 1, 2, 64, 64),
    (1, 65, 1, 1, 128, 256), (2, 130, 2, 2, 48, 72), (1, 200, 1, 2, 128, 100), (3, 70, 1, 1, 7, 17),
    (1, 300, 2, 4, 96, 128),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradients(shape, dtype):
    b, L, hk, hv, dk, dv = shape
    check(inputs(*shape, dtype, seed=L), state(b, hv, dk, dv), state(b, hv, dk, dv, seed=8))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L", [5, 100])
def test_gradients_qk_norm(L, dtype):
    check(inputs(2, L, 2, 4, 64, 40, dtype, seed=3, unit=False), qk_norm=True, scale=0.7)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_lengths(dtype):
    n = torch.tensor([0, 64, 150, 65, -2, 500], dtype=torch.int32)
    r = check(inputs(6, 150, 1, 2, 64, 64, dtype, seed=5), state(6, 2, 64, 64), state(6, 2, 64, 64, seed=8), n,
              garbage=True)
    for i, m in enumerate(n.clamp(0, 150)):
        for name in NAMES[:5]:
            assert not r[name][i, int(m):].any(), name


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", [(64, 48), (128, 130)])
def test_gradients_of_long_rows_walked_in_segments(dk, dv, dtype):
    n = torch.tensor([1200, 640, 3], dtype=torch.int32)
    check(inputs(3, 1200, 1, 1, dk, dv, dtype, seed=21, g_scale=0.02), state(3, 1, dk, dv),
          state(3, 1, dk, dv, seed=8), n)


def test_gradients_resets_zero_beta_and_zero_keys():
    ins = list(inputs(1, 140, 1, 2, 64, 64, torch.float32, seed=4, unit=False))
    ins[4][0, 10:20] = 0.0
    ins[1][0, 30:40] = 0.0
    ins[0][0, 35:45] = 0.0
    ins[3][0, 50, 0] = -200.0
    ins[3][0, 60:90, 1] = -30.0
    check(ins, state(1, 2, 64, 64), qk_norm=True)


def test_gradients_correlated_keys():
    gen = torch.Generator().manual_seed(2)
    ins = list(inputs(1, 128, 1, 1, 64, 32, torch.float32, seed=2, g_scale=0.01))
    k = torch.randn(1, 1, 1, 64, generator=gen) + 0.3 * torch.randn(1, 128, 1, 64, generator=gen)
    ins[1] = k / k.norm(dim=-1, keepdim=True)
    check(ins)


def test_strided_inputs_and_repeatability():
    b, L, hk, hv, dk, dv = 2, 90, 2, 4, 64, 48
    ins = inputs(b, L, hk, hv, dk, dv, torch.bfloat16, seed=8)
    dout = torch.randn(b, L, hv, dv).bfloat16().to(DEV)
    want = sscan.delta_bwd(*on(*ins), dout)
    views = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in on(*ins)]
    got, again = sscan.delta_bwd(*views, dout), sscan.delta_bwd(*views, dout)
    for n in NAMES:
        assert torch.equal(got[n], again[n]) and torch.equal(got[n], want[n]), n


def test_differences_of_the_forward():
    """Directional differences of the kernels' forward: with steps of 1e-2 in float32 the
    difference quotient is good to about 1e-3 (second-order truncation and rounding)."""
    ins = on(*inputs(1, 100, 1, 2, 64, 64, torch.float32, seed=6))
    h0 = state(1, 2, 64, 64).to(DEV)
    gen = torch.Generator().manual_seed(1)
    dout = torch.randn(1, 100, 2, 64, generator=gen).to(DEV)
    dh = torch.randn(1, 2, 64, 64, generator=gen).to(DEV)
    r = sscan.delta_bwd(*ins, dout, h0=h0, dh_last=dh)

    def loss(xs):
        out, last = sscan.delta_fwd(*xs[:5], h0=xs[5].contiguous())
        return float((out.double() * dout).sum() + (last.double() * dh).sum())

    xs = ins + [h0]
    for k, name in enumerate(NAMES):
        d = torch.randn(xs[k].shape, generator=gen).to(DEV)
        d = d / d.norm()
        up, down = ([x + s * d if j == k else x for j, x in enumerate(xs)] for s in (1e-2, -1e-2))
        diff = (loss(up) - loss(down)) / 2e-2
        want = float((r[name].double() * d).sum())
        assert abs(diff - want) <= 2e-3 * (abs(want) + float(r[name].norm()) / d.numel() ** 0.5), (name, diff, want)


def test_autograd_through_pieces():
    """A sequence trained in two pieces, the state handed on, equals the whole."""
    ins = [x.requires_grad_(True) for x in on(*inputs(2, 120, 1, 2, 64, 64, torch.float32, seed=10))]
    h0 = state(2, 2, 64, 64).to(DEV).requires_grad_(True)
    dout = torch.randn(2, 120, 2, 64, device=DEV)
    out, last = sscan.gated_delta(*ins, h0=h0)
    whole = torch.autograd.grad((out * dout).sum() + last.square().sum(), ins + [h0])
    o1, s = sscan.gated_delta(*[x[:, :50] for x in ins], h0=h0)
    o2, s = sscan.gated_delta(*[x[:, 50:] for x in ins], h0=s)
    parts = torch.autograd.grad((torch.cat([o1, o2], 1) * dout).sum() + s.square().sum(), ins + [h0])
    for n, a, b in zip(NAMES, parts, whole):
        close(a, b.cpu().double(), n)
    (only,) = torch.autograd.grad(sscan.gated_delta(*ins)[1].sum(), [ins[2]])
    assert torch.isfinite(only).all()


def test_empty_and_refusals():
    ins = inputs(2, 0, 1, 1, 64, 64, torch.float32)
    dh = state(2, 1, 64, 64)
    r = sscan.delta_bwd(*on(*ins), torch.zeros(2, 0, 1, 64, device=DEV), dh_last=dh.to(DEV))
    assert torch.equal(r["dh0"].cpu(), dh) and r["dq"].shape == (2, 0, 1, 64)
    q, k, v, g, beta = on(*inputs(1, 70, 1, 2, 64, 64, torch.float32))
    with pytest.raises(ValueError):
        sscan.delta_bwd(q, k, v, g, beta, torch.zeros(1, 70, 1, 64, device=DEV))
    with pytest.raises(TypeError):
        sscan.delta_bwd(q, k, v, g, beta, torch.zeros(1, 70, 2, 64, device=DEV).bfloat16())
    with pytest.raises(sscan.SScanError):
        sscan.delta_bwd(q, k, v, g, beta, torch.zeros(1, 70, 2, 64, device=DEV),
                        workspace=torch.empty(1024, dtype=torch.uint8, device=DEV))


def test_graph_replays():
    ins = on(*inputs(1, 100, 1, 2, 64, 64, torch.bfloat16, seed=12))
    dout = torch.randn(1, 100, 2, 64, device=DEV).bfloat16()
    n = sscan.delta_workspace_bytes(1, 100, 1, 2, 64, 64, backward=True)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    sscan.delta_bwd(*ins, dout, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = sscan.delta_bwd(*ins, dout, workspace=ws)
    for seed in (13, 14, 15):
        for x, y in zip(ins, inputs(1, 100, 1, 2, 64, 64, torch.bfloat16, seed=seed)):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        want = sscan.delta_bwd(*ins, dout)
        torch.cuda.synchronize()
        for name in NAMES:
            assert torch.equal(r[name], want[name]), name
