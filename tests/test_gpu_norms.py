"""The gated norm and the residual norm, both directions, against float64."""
import pytest
import torch

import delta_ref
from delta_ref import close
from selective_state_space_sscan_amd import sscan

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
EPS = 1e-6


def rand(*shape, seed=0, dtype=torch.float32, scale=1.0):
    return (scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).to(dtype)


def on(*xs):
    return [None if x is None else x.to(DEV) for x in xs]


def grads(f, ins, douts):
    ins = [None if x is None else x.double().requires_grad_(True) for x in ins]
    outs = f(*ins)
    outs = outs if isinstance(outs, tuple) else (outs,)
    live = [x for x in ins if x is not None]
    got = iter(torch.autograd.grad(outs, live, [d.double() for d in douts]))
    return [None if x is None else next(got) for x in ins]


GATED = [(1, 1, 1), (3, 2, 8), (5, 3, 33), (70, 4, 128), (9, 1, 200), (4, 2, 257), (33, 1, 768), (6, 1, 1536),
         (3, 1, 2500), (2, 1, 5000), (3, 1, 8192), (600, 16, 64)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("weight", ["none", "shared", "per_head"])
@pytest.mark.parametrize("n,h,size", GATED)
def test_gated_norm(n, h, size, weight, gate_first, dtype):
    print("gated", n, h, size, weight, gate_first, dtype, flush=True)
    x, z, dout = (rand(n, h, size, seed=s, dtype=dtype) for s in (1, 2, 3))
    w = {"none": None, "shared": 1 + rand(size, seed=4, scale=0.2), "per_head": 1 + rand(h, size, seed=4, scale=0.2)}[weight]
    y = sscan.gated_norm(*on(x, z, w), eps=EPS, gate_first=gate_first)
    close(y, delta_ref.gated_norm(x, z, w, EPS, gate_first), "y")
    r = sscan.gated_norm_bwd(*on(x, z, dout, w), eps=EPS, gate_first=gate_first)
    gx, gz, gw = grads(lambda x, z, w: delta_ref.gated_norm(x, z, w, EPS, gate_first), (x, z, w), [dout])
    zd, dn = z.double(), dout.double() * (1 if w is None else w.double())
    gate = zd * torch.sigmoid(zd)
    m, dm = (x.double() * gate, dn) if gate_first else (x.double(), dn * gate)
    terms = delta_ref.norm_terms(m, dm, EPS)
    close(r["dx"], gx, "dx", terms)
    close(r["dz"], gz, "dz", terms)
    assert (r["dweight"] is None) == (w is None)
    if w is not None:
        close(r["dweight"], gw, "dweight")


ADD = [(1, 1), (4, 8), (7, 50), (130, 128), (5, 333), (33, 768), (4, 1536), (3, 4100), (2, 8192), (1500, 64)]


@pytest.mark.parametrize("dtype,res", [(torch.float32, torch.float32), (torch.bfloat16, torch.float32),
                                       (torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("parts", ["all", "weight", "none", "post", "no_residual"])
@pytest.mark.parametrize("n,size", ADD)
def test_add_norm(n, size, parts, dtype, res):
    print("add", n, size, parts, dtype, res, flush=True)
    x, dout = rand(n, size, seed=1, dtype=dtype), rand(n, size, seed=2, dtype=dtype)
    residual = None if parts == "no_residual" else rand(n, size, seed=3, dtype=res, scale=2.0)
    dres = None if parts == "weight" else rand(n, size, seed=5, dtype=res)
    w = None if parts == "none" else 1 + rand(size, seed=6, scale=0.2)
    s = 0.3 + rand(size, seed=7, scale=0.1) if parts in ("all", "no_residual") else None
    p = 1 + rand(size, seed=8, scale=0.2) if parts in ("all", "post") else None
    y, total = sscan.add_norm(*on(x, residual, w, s, p), eps=EPS, residual_dtype=res)
    ref_y, ref_total = delta_ref.add_norm(x, residual, w, s, p, EPS, torch.float64)
    close(total, ref_total, "total")
    # the norm is that of the total as the call stored it
    stored = total.cpu().double()
    close(y, delta_ref.rms_unit(stored, EPS) * (1 if w is None else w.double()), "y")
    r = sscan.add_norm_bwd(*on(x), total, *on(dout, w), dresidual_out=on(dres)[0], scale=on(s)[0],
                           post_weight=on(p)[0], eps=EPS)
    t = stored.requires_grad_(True)
    wd = None if w is None else w.double().requires_grad_(True)
    out = delta_ref.rms_unit(t, EPS) * (1 if w is None else wd)
    got = torch.autograd.grad(out, [t] + ([] if w is None else [wd]), dout.double())
    dt = got[0] + (0 if dres is None else dres.double())
    terms = delta_ref.norm_terms(stored.detach(), dout.double() * (1 if w is None else w.double()), EPS)
    close(r["dresidual"], dt, "dresidual", terms)
    if w is not None:
        close(r["dweight"], got[1], "dweight")
    gx, gs, gp = grads(lambda x, s, p: delta_ref.add_norm(x, None, None, s, p, EPS, torch.float64)[1], (x, s, p), [dt])
    # what dresidual may be off by passes through the scale and x's own norm
    factor = torch.ones(size, dtype=torch.float64) * (1 if s is None else s.double())
    if p is not None:
        factor = factor * p.double()
        terms = delta_ref.norm_terms(x, (dt.abs() + terms) * factor, EPS)
    else:
        terms *= float(factor.abs().max())
    close(r["dx"], gx, "dx", terms)
    # and sums over the rows
    for name, g in (("dscale", gs), ("dpost_weight", gp)):
        assert (r[name] is None) == (g is None)
        if g is not None:
            close(r[name], g, name, terms if size == 1 else 0.0)


def test_gated_norm_of_strided_views():
    """x as heads of a wider row, z a slice of a packed projection, unaligned."""
    packed = rand(2, 9, 3 + 4 * 64 + 5, seed=1, dtype=torch.bfloat16).to(DEV)
    z = packed[..., 3:3 + 256].unflatten(-1, (4, 64))
    x = rand(2, 9, 4, 128, seed=2, dtype=torch.bfloat16).to(DEV)[..., :64]
    dout, w = rand(2, 9, 4, 64, seed=3, dtype=torch.bfloat16).to(DEV), rand(64, seed=4).to(DEV)
    y = sscan.gated_norm(x, z, w)
    r = sscan.gated_norm_bwd(x, z, dout, w)
    y2 = sscan.gated_norm(x.contiguous(), z.contiguous(), w)
    r2 = sscan.gated_norm_bwd(x.contiguous(), z.contiguous(), dout, w)
    for a, b in ((y, y2), (r["dx"], r2["dx"]), (r["dz"], r2["dz"])):
        close(a, b.cpu().double(), "strided")
    close(r["dweight"], r2["dweight"].cpu(), "dweight")
    with pytest.raises(ValueError):  # batch and token strides that no single row stride covers
        sscan.gated_norm(x.transpose(0, 1), z.transpose(0, 1), w)
    with pytest.raises(ValueError):  # one row broadcast over an inner dimension
        sscan.gated_norm(x[:, :1].expand(2, 9, 4, 64), z)
    one = sscan.gated_norm(x[:1, :1].expand(2, 9, 4, 64), z)  # over all of them: rows of stride 0
    close(one, sscan.gated_norm(x[:1, :1].expand(2, 9, 4, 64).contiguous(), z).cpu().double(), "broadcast")
    # a weight that is not 16-byte aligned
    y3 = sscan.gated_norm(x, z, torch.cat([w[:1], w])[1:])
    close(y3, y2.cpu().double(), "unaligned weight")


def test_add_norm_in_place_and_unaligned():
    x, res, w = on(rand(40, 64, seed=1, dtype=torch.bfloat16), rand(40, 64, seed=2), 1 + rand(65, seed=3))
    y, total = sscan.add_norm(x, res, w[1:])
    kept = res.clone()
    y2, total2 = sscan.add_norm(x, kept, w[1:].clone(), residual_out=kept)
    assert total2 is kept and torch.equal(total, kept)
    close(y2, y.cpu().double(), "y")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [5, 7, 9, 15, 129, 1031, 2047, 4097, 8185])
def test_sizes_with_a_rest(size, dtype):
    test_gated_norm(9, 1, size, "shared", False, dtype)
    test_gated_norm(3, 4, size, "per_head", True, dtype)
    test_add_norm(11, size, "all", dtype, torch.float32)


@pytest.mark.parametrize("size", [9, 513, 2001])
def test_in_place_with_a_rest(size):
    x, res, w = on(rand(700, size, seed=1), rand(700, size, seed=2), 1 + rand(size, seed=3))
    y, total = sscan.add_norm(x, res, w)
    kept = res.clone()
    y2, _ = sscan.add_norm(x, kept, w, residual_out=kept)
    assert torch.equal(total, kept) and torch.equal(y, y2)


def test_reduced_over_no_rows_is_zero():
    r = sscan.gated_norm_bwd(*on(torch.zeros(0, 2, 64), torch.zeros(0, 2, 64), torch.zeros(0, 2, 64), torch.ones(64)))
    assert r["dx"].shape == (0, 2, 64) and not r["dweight"].any()
    r = sscan.gated_norm_bwd(*on(torch.zeros(0, 2, 64), torch.zeros(0, 2, 64), torch.zeros(0, 2, 64), torch.ones(2, 64)))
    assert not r["dweight"].any()
    x = torch.zeros(0, 64, device=DEV)
    y, total = sscan.add_norm(x, x, torch.ones(64, device=DEV))
    assert y.shape == (0, 64) and total.shape == (0, 64)
    r = sscan.add_norm_bwd(x, x, x, torch.ones(64, device=DEV), scale=torch.ones(64, device=DEV))
    assert not r["dweight"].any() and not r["dscale"].any()


def test_zero_rows_stay_finite():
    x = torch.zeros(3, 1, 64)
    z = rand(3, 1, 64, seed=1)
    y = sscan.gated_norm(*on(x, z))
    r = sscan.gated_norm_bwd(*on(x, z, rand(3, 1, 64, seed=2)))
    assert not y.any() and torch.isfinite(r["dx"]).all() and not r["dz"].any()
    # gates far out: silu of -1e30 is 0, of 1e30 the value itself
    z = torch.full((1, 1, 64), -1e30)
    assert not sscan.gated_norm(*on(rand(1, 1, 64, seed=3), z)).any()


def test_autograd_and_repeatability():
    x, z, w, s, p = on(rand(50, 4, 96, seed=1, dtype=torch.bfloat16), rand(50, 4, 96, seed=2, dtype=torch.bfloat16),
                       1 + rand(96, seed=3, scale=0.1), 1 + rand(96, seed=4, scale=0.1), 1 + rand(96, seed=5, scale=0.1))
    leaves = [t.requires_grad_(True) for t in (x, z, w, s, p)]
    res = rand(50, 4, 96, seed=6).to(DEV).requires_grad_(True)

    def loss():
        y = sscan.gated_rms_norm(x, z, w)
        out, total = sscan.add_rms_norm(y, res, w, s, p)
        return (out.float() * total).sum()

    first = torch.autograd.grad(loss(), leaves + [res])
    again = torch.autograd.grad(loss(), leaves + [res])
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    d = [t.detach().cpu().double().requires_grad_(True) for t in leaves + [res]]
    y = delta_ref.gated_norm(d[0], d[1], d[2], EPS, False)
    y = y + (y.detach().bfloat16().double() - y.detach())
    out, total = delta_ref.add_norm(y, d[5], d[2], d[3], d[4], EPS, torch.float64)
    ref = torch.autograd.grad((out * total).sum(), d)
    for a, b in zip(first, ref):  # out is rounded to bf16 on the way, so 2^-8 of the gradients' size
        assert float((a.detach().cpu().double() - b).norm() / b.norm()) < 2.0 ** -7


def test_refusals():
    x, z, w = on(rand(4, 2, 64), rand(4, 2, 64), torch.ones(64))
    with pytest.raises(ValueError):
        sscan.gated_norm(x, z[:2], w)
    with pytest.raises(TypeError):
        sscan.gated_norm(x, z.bfloat16(), w)
    with pytest.raises(ValueError):
        sscan.gated_norm(x, z, torch.ones(3, 64, device=DEV))
    with pytest.raises(TypeError):
        sscan.gated_norm(x, z, w.bfloat16())
    with pytest.raises(ValueError):
        sscan.gated_norm(x.transpose(1, 2), z.transpose(1, 2))
    with pytest.raises(sscan.SScanError):
        sscan.gated_norm(x, z, w, eps=float("nan"))
    with pytest.raises(sscan.SScanError):
        sscan.gated_norm(x, z, w, out=x)
    big = torch.zeros(1, 8193, device=DEV)
    with pytest.raises(sscan.SScanError):
        sscan.add_norm(big, big)
    with pytest.raises(ValueError):
        sscan.add_norm(x, x[:2])
    with pytest.raises(sscan.SScanError):
        sscan.add_norm(x, z, out=z)
    with pytest.raises(ValueError):
        sscan.add_norm(x.cpu(), z)
