"""The plain forms of tests/rec_ref.py: their gradients against differentiation by torch and
against central differences, their bounds against a float32 evaluation of the same loops."""
import itertools

import pytest
import torch

import rec_ref


def draw(b, l, d, seed=0, dtype=torch.float64):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64).to(dtype)
    lam = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * torch.rand(d, generator=gen, dtype=torch.float64)) / 8)).to(dtype)
    return dict(x=r(b, l, d), g=r(b, l, d), i=r(b, l, d), z=r(b, l, d), lam=lam, h0=r(b, d), dout=r(b, l, d), dh_last=r(b, d))


def loss(t, lengths, reverse, gated):
    """Token by token, in torch operations: the sum whose gradients are wanted."""
    b, l, _ = t["x"].shape
    total = 0
    for row, n in enumerate([l] * b if lengths is None else lengths):
        h = t["h0"][row]
        for tok in (range(n - 1, -1, -1) if reverse else range(n)):
            x, g, i, z = (t[k][row, tok] for k in ("x", "g", "i", "z"))
            if gated:
                a = torch.exp(-8 * torch.nn.functional.softplus(t["lam"]) * torch.sigmoid(g))
                w = torch.sqrt(1 - a * a)
            else:
                a, w = torch.exp(g), 1
            h = a * h + w * torch.sigmoid(i) * x
            total = total + (h * z * torch.sigmoid(z) * t["dout"][row, tok]).sum()
        total = total + (h * t["dh_last"][row]).sum()
    return total


@pytest.mark.parametrize("gated,reverse,ragged", itertools.product([True, False], repeat=3))
def test_gradients(gated, reverse, ragged):
    t = draw(3, 7, 4, seed=1)
    lengths = [0, 4, 7] if ragged else None
    if not gated:
        t["g"] = -t["g"].abs()
    names = ["x", "g", "i", "z", "h0"] + (["lam"] if gated else [])
    leaves = {k: v.clone().requires_grad_(k in names) for k, v in t.items()}
    want = dict(zip(names, torch.autograd.grad(loss(leaves, lengths, reverse, gated), [leaves[k] for k in names])))
    got = rec_ref.rec_bwd(t["x"], t["g"], t["dout"], t["i"], t["lam"] if gated else None, t["z"], t["h0"], t["dh_last"],
                          lengths, 8.0, reverse)
    for k in names:
        assert torch.allclose(got["d" + k][0], want[k], rtol=1e-10, atol=1e-12), k
    # and central differences, off by their step's square and the rounding of the sum over it
    gen = torch.Generator().manual_seed(9)
    for k in names:
        step = torch.randn(t[k].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        up, down = (loss(dict(t, **{k: t[k] + s * h * step}), lengths, reverse, gated) for s in (1, -1))
        assert abs(float((up - down) / (2 * h)) - float((got["d" + k][0] * step).sum())) < 1e-6


@pytest.mark.parametrize("gated,reverse", itertools.product([True, False], repeat=2))
def test_bounds_hold_for_float32_loops(gated, reverse):
    t = draw(2, 300, 16, seed=2, dtype=torch.float32)
    if not gated:
        t["g"] = -t["g"].abs() * 0.05
    lam = t["lam"] if gated else None
    leaves = {k: v.clone().requires_grad_(True) for k, v in t.items()}
    want = rec_ref.rec_bwd(t["x"], t["g"], t["dout"], t["i"], lam, t["z"], t["h0"], t["dh_last"], None, 8.0, reverse)
    if not gated:
        got = torch.autograd.grad(loss(leaves, None, reverse, False), [leaves[k] for k in ("x", "g", "i", "z", "h0")])
        for k, v in zip(("dx", "dg", "di", "dz", "dh0"), got):
            rec_ref.within(v, want[k], k)
    fwd = rec_ref.rec(t["x"], t["g"], t["i"], lam, t["z"], t["h0"], None, 8.0, reverse)
    h, outs = t["h0"], {}
    for tok in (range(299, -1, -1) if reverse else range(300)):
        x, g, i, z = (t[k][:, tok] for k in ("x", "g", "i", "z"))
        if gated:
            loss_ = -torch.expm1(-8 * torch.nn.functional.softplus(t["lam"]) * torch.sigmoid(g))
            a, w = 1 - loss_, torch.sqrt(loss_ * (2 - loss_))
        else:
            a, w = torch.exp(g), 1
        h = a * h + w * torch.sigmoid(i) * x
        outs[tok] = h * z * torch.sigmoid(z)
    rec_ref.within(torch.stack([outs[k] for k in range(300)], 1), fwd["out"], "out")
    rec_ref.within(h, fwd["h_last"], "h_last")


def test_layer_norm_gradients():
    gen = torch.Generator().manual_seed(3)
    x, d, dt = (torch.randn(5, 37, generator=gen, dtype=torch.float64) for _ in range(3))
    w, c = torch.randn(37, generator=gen, dtype=torch.float64), torch.randn(37, generator=gen, dtype=torch.float64)
    leaves = [v.clone().requires_grad_(True) for v in (x, w, c)]
    y = torch.nn.functional.layer_norm(leaves[0], (37,), leaves[1], leaves[2], 1e-5)
    want = torch.autograd.grad((y * d).sum() + (leaves[0] * dt).sum(), leaves)
    got = rec_ref.layer_norm(x, w, c, 1e-5, d, dt)
    assert torch.allclose(got["out"][0], y)
    for k, v in zip(("dx", "dweight", "dbias"), want):
        assert torch.allclose(got[k][0], v, rtol=1e-10, atol=1e-12), k


def test_eight_bits():
    x = torch.randn(3, 130, generator=torch.Generator().manual_seed(4))
    x[0, :64] = 0
    x[1, 70] = float("inf")
    x[2, 129] = 1e-38
    x[2, 128] = 0
    q, scale, value = rec_ref.eight(x)
    assert not q[0, :64].any() and scale[0, 0] == 0 and torch.isnan(value[1, 64:128]).all() and scale[2, 2] == 0
    fine = torch.isfinite(value) & (value != 0)
    step = scale.repeat_interleave(64, -1)[:, :130].double()
    assert ((value - x).abs()[fine] <= 0.5 * step[fine] * (1 + 1e-6)).all()
