"""The norm kernels with more rows than their grids hold, so that blocks walk over several:
the rows loaded ahead, the walk's carry over heads, the buffers of the sums that take turns,
and the weights' gradients added over a block's rows.  Against float64; the tolerances are
delta_ref's, a weight's gradient bounded by the size of its many terms."""
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


def summed(got, ref, terms, name):
    """A sum over many rows in float32: 1e-5 of the root of the sum of its squared terms
    (``terms``, per element) beside delta_ref's bound."""
    err = (got.cpu().double() - ref).abs()
    bound = 1e-5 * (ref.abs() + terms)
    assert float((err / bound).max()) <= 1.0, name


# a vector of 1000 is held by 128 threads, two vectors a block: over 8192 blocks forward
GATED = [(6001, 3, 1000, "shared"), (6001, 3, 1000, "per_head"), (2700, 7, 513, "shared"), (9000, 1, 2001, "none"),
         (8300, 1, 4099, "per_head")]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,h,size,weight", GATED)
def test_gated_norm_over_many_rows(n, h, size, weight, dtype):
    print("gated", n, h, size, weight, dtype, flush=True)
    # heads apart from each other in memory, so that they are not taken for rows
    gate_first = weight == "per_head"
    x, z, dout = (rand(n, h, size + 3, seed=s, dtype=dtype)[..., :size] for s in (1, 2, 3))
    dout = dout.contiguous()
    w = {"none": None, "shared": 1 + rand(size, seed=4, scale=0.2), "per_head": 1 + rand(h, size, seed=4, scale=0.2)}[weight]
    xd, zd = (torch.nn.functional.pad(t, (0, 3)).to(DEV)[..., :size] for t in (x, z))
    y = sscan.gated_norm(xd, zd, *on(w), eps=EPS, gate_first=gate_first)
    close(y, delta_ref.gated_norm(x, z, w, EPS, gate_first), "y")
    r = sscan.gated_norm_bwd(xd, zd, *on(dout, w), eps=EPS, gate_first=gate_first)
    x, z, d = x.double(), z.double(), dout.double()
    wd = 1.0 if w is None else w.double()
    sig = torch.sigmoid(z)
    gate, slope = z * sig, sig * (1 + z * (1 - sig))
    m = x * gate if gate_first else x
    dn = d * wd if gate_first else d * wd * gate
    rms = 1 / (m.square().mean(-1, keepdim=True) + EPS).sqrt()
    dm = rms * (dn - m * rms * rms * (dn * m).mean(-1, keepdim=True))
    terms = delta_ref.norm_terms(m, dn, EPS)
    if gate_first:
        dx, dz, dw = dm * gate, dm * x * slope, d * m * rms
    else:
        dx, dz, dw = dm, d * m * rms * wd * slope, d * gate * m * rms
    close(r["dx"], dx, "dx", terms)
    close(r["dz"], dz, "dz", terms)
    if w is not None:
        over = 0 if weight == "per_head" else (0, 1)
        summed(r["dweight"], dw.sum(over), dw.square().sum(over).sqrt(), "dweight")


# backward 512 blocks of 2, 1 and 1 rows; forward 8192 blocks
ADD = [(2501, 1000), (1400, 2001), (1300, 8185), (9001, 513)]


@pytest.mark.parametrize("dtype,res", [(torch.bfloat16, torch.float32), (torch.float32, torch.float32),
                                       (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("n,size", ADD)
def test_add_norm_over_many_rows(n, size, post, dtype, res):
    print("add", n, size, post, dtype, res, flush=True)
    x, dout = rand(n, size, seed=1, dtype=dtype), rand(n, size, seed=2, dtype=dtype)
    residual, dres = rand(n, size, seed=3, dtype=res, scale=2.0), rand(n, size, seed=5, dtype=res)
    w, s = 1 + rand(size, seed=6, scale=0.2), 0.3 + rand(size, seed=7, scale=0.1)
    p = 1 + rand(size, seed=8, scale=0.2) if post else None
    y, total = sscan.add_norm(*on(x, residual, w, s, p), eps=EPS)
    close(total, delta_ref.add_norm(x, residual, w, s, p, EPS, torch.float64)[1], "total")
    stored = total.cpu().double()
    close(y, delta_ref.rms_unit(stored, EPS) * w.double(), "y")
    kept = residual.to(DEV)
    y2, _ = sscan.add_norm(*on(x), kept, *on(w, s, p), eps=EPS, residual_out=kept)
    assert torch.equal(kept, total) and torch.equal(y2, y)
    r = sscan.add_norm_bwd(*on(x), total, *on(dout, w), dresidual_out=on(dres)[0], scale=on(s)[0], post_weight=on(p)[0],
                           eps=EPS)
    x, d, wd, sd = x.double(), dout.double(), w.double(), s.double()
    rt = 1 / (stored.square().mean(-1, keepdim=True) + EPS).sqrt()
    dn = d * wd
    dt = dres.double() + rt * (dn - stored * rt * rt * (dn * stored).mean(-1, keepdim=True))
    terms = delta_ref.norm_terms(stored, dn, EPS)
    close(r["dresidual"], dt, "dresidual", terms)
    sums = {"dweight": d * stored * rt}
    a, da, factor = x, dt * sd, sd
    if post:
        pd = p.double()
        rx = 1 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
        a, n_x = x * rx * pd, x * rx
        sums["dpost_weight"] = da * n_x
        dnx = da * pd
        da = rx * (dnx - x * rx * rx * (dnx * x).mean(-1, keepdim=True))
        factor = sd * pd
        terms_x = delta_ref.norm_terms(x, (dt.abs() + terms) * factor, EPS)
    else:
        terms_x = terms * float(factor.abs().max())
    sums["dscale"] = dt * a
    close(r["dx"], da, "dx", terms_x)
    for name, t in sums.items():
        summed(r[name], t.sum(0), t.square().sum(0).sqrt(), name)


def test_the_gate_is_as_exact_as_stated():
    """Rows of ones: their norm is 1 / sqrt(1 + eps), off by at most 3 x 2^-24, and the output
    that times silu(z), whose sigmoid is off by at most (1.25 |z| + 5) 2^-24 of itself; two
    more products are rounded.  (Below -87 a sigmoid is smaller than float32's normal numbers.)"""
    z = torch.linspace(-80, 80, 1 << 18, dtype=torch.float32).view(-1, 1, 64)
    y = sscan.gated_norm(torch.ones_like(z).to(DEV), z.to(DEV), eps=EPS).cpu().double()
    zd = z.double()
    ref = zd / (1 + torch.exp(-zd)) / (1 + EPS) ** 0.5
    err = (y - ref).abs() / ((1.25 * zd.abs() + 10) * 2.0 ** -24 * ref.abs() + 1e-45)
    assert float(err.max()) <= 1.0
