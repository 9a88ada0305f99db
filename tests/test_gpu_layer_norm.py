"""Layer norm with the residual sum, both directions, against float64."""
import pytest
import torch

import rec_ref
from rec_ref import U, within
from selective_state_space_sscan_amd import sscan

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16


def rand(*shape, seed=0, dtype=F32, scale=1.0, shift=0.0):
    x = scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) + shift
    return x.to(dtype).to(DEV)


def check(x, residual, w, c, dout, dtotal, res=None, eps=1e-5):
    out, total = sscan.layer_norm(x, w, c, residual, eps, res)
    if residual is None and res is None:
        assert total is x
    else:
        sum_ = x.double() + (0 if residual is None else residual.double())
        # summed in float32, then stored
        within(total, (sum_, U * sum_.abs() if total.dtype == BF16 else 0 * sum_), "total")
    want = rec_ref.layer_norm(total, w, c, eps, dout, dtotal)
    within(out, want["out"], "out")
    got = sscan.layer_norm_bwd(total, dout, w, c, dtotal, eps)
    within(got["dx"], want["dx"], "dx")
    within(got["dresidual"], want["dx"], "dresidual")
    assert got["dx"].dtype == dout.dtype and got["dresidual"].dtype == total.dtype
    for k, v in (("dweight", w), ("dbias", c)):
        assert (got[k] is None) == (v is None)
        if v is not None:
            within(got[k], want[k], k)
    return out, total, got


SIZES = [(1, 1), (3, 2), (7, 5), (4, 8), (5, 33), (130, 128), (9, 200), (4, 257), (33, 768), (6, 1536), (3, 2500),
         (2, 5000), (3, 8191), (2, 8192), (1500, 64), (700, 513), (2100, 1031), (9000, 24)]


@pytest.mark.parametrize("dtype,res", [(F32, F32), (BF16, F32), (BF16, BF16), (F32, BF16), (F32, None), (BF16, None)])
@pytest.mark.parametrize("n,size", SIZES)
def test_layer_norm(n, size, dtype, res):
    print("layer norm", n, size, dtype, res, flush=True)
    x, dout = rand(n, size, seed=1, dtype=dtype), rand(n, size, seed=2, dtype=dtype)
    residual = None if res is None else rand(n, size, seed=3, dtype=res, scale=2.0, shift=0.5)
    dtotal = None if res is None else rand(n, size, seed=4, dtype=res)
    w, c = 1 + rand(size, seed=5, scale=0.2), rand(size, seed=6, scale=0.2)
    check(x, residual, w, c, dout, dtotal)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("parts", ["", "w", "c", "r", "wr", "first"])
def test_parts(parts, dtype):
    n, size = 50, 333
    w = 1 + rand(size, seed=5, scale=0.2) if "w" in parts else None
    c = rand(size, seed=6) if parts == "c" else None
    residual = rand(n, size, seed=3) if "r" in parts and parts != "first" else None
    check(rand(n, size, seed=1, dtype=dtype), residual, w, c, rand(n, size, seed=2, dtype=dtype), None,
          F32 if parts == "first" else None)


def test_means_far_from_zero_and_flat_rows():
    for shift in (30.0, 1000.0):
        check(rand(40, 700, seed=1, shift=shift), None, 1 + rand(700, seed=2), None, rand(40, 700, seed=3), None)
    x = torch.full((4, 100), 3.0, device=DEV)
    out, _ = sscan.layer_norm(x, None, None)
    assert not out.any()
    got = sscan.layer_norm_bwd(x, rand(4, 100, seed=1))
    assert torch.isfinite(got["dx"]).all()
    x = rand(4, 100, seed=2)
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    out, _ = sscan.layer_norm(x)
    assert torch.isnan(out[1]).all() and torch.isnan(out[2]).any()
    assert torch.equal(out[[0, 3]], sscan.layer_norm(x[[0, 3]])[0])


def test_strides_places_and_alignment():
    packed = rand(6, 7, 3 + 130 + 5, seed=1, dtype=BF16)
    x = packed[..., 3:133]
    w = rand(131, seed=2)[1:]
    out, total = sscan.layer_norm(x, w)
    assert total is x and torch.equal(out, sscan.layer_norm(x.contiguous(), w.clone())[0])
    dout = rand(6, 7, 130, seed=3, dtype=BF16)
    a, b = sscan.layer_norm_bwd(x, dout, w), sscan.layer_norm_bwd(x.contiguous(), dout, w.clone())
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dweight"], b["dweight"])
    row = x[:1, :1].expand(6, 7, 130)
    assert torch.equal(sscan.layer_norm(row)[0], sscan.layer_norm(row.contiguous())[0])
    with pytest.raises(ValueError):
        sscan.layer_norm(x.transpose(0, 1))
    for size in (64, 513, 2001):
        x, res, w = rand(700, size, seed=4), rand(700, size, seed=5), rand(size, seed=6)
        out, total = sscan.layer_norm(x, w, None, res)
        kept = res.clone()
        out2, total2 = sscan.layer_norm(x, w, None, kept, residual_out=kept)
        assert total2 is kept and torch.equal(total, kept) and torch.equal(out, out2)


def test_autograd_against_float64():
    x, res = rand(50, 96, seed=1, dtype=BF16), rand(50, 96, seed=2)
    w, c = 1 + rand(96, seed=3, scale=0.1), rand(96, seed=4)
    leaves = [t.requires_grad_(True) for t in (x, res, w, c)]
    dout, dtotal = rand(50, 96, seed=5, dtype=BF16), rand(50, 96, seed=6)
    out, total = sscan.add_layer_norm(x, res, w, c)
    got = torch.autograd.grad([out, total], leaves, [dout, dtotal], retain_graph=True)
    want = rec_ref.layer_norm(total.detach(), w.detach(), c.detach(), 1e-5, dout, dtotal)
    for v, k in zip(got, ("dx", "dx", "dweight", "dbias")):
        within(v, want[k], k)
    again = torch.autograd.grad([out, total], leaves, [dout, dtotal])
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    # without a residual the total is x itself, and both outputs' gradients reach it
    y, same = sscan.add_layer_norm(x, None, w, c)
    (g,) = torch.autograd.grad([y, same], [x], [dout, dtotal.bfloat16()])
    want = rec_ref.layer_norm(x.detach(), w.detach(), c.detach(), 1e-5, dout, dtotal.bfloat16())
    within(g, want["dx"], "dx")
    with pytest.raises(RuntimeError, match="no second derivatives"):
        y, _ = sscan.add_layer_norm(x, None, w, c)
        (g,) = torch.autograd.grad(y.float().sum(), [x], create_graph=True)
        torch.autograd.grad(g.float().sum(), [x])


def test_empty_and_many_rows():
    for lead in ((0,), (2, 0)):
        x, w = torch.zeros(*lead, 64, device=DEV), torch.ones(64, device=DEV)
        assert sscan.layer_norm(x, w)[0].shape == (*lead, 64)
        got = sscan.layer_norm_bwd(x, x, w, w)
        assert not got["dweight"].any() and not got["dbias"].any()
    # more rows than the grids hold
    check(rand(150000, 8, seed=1), rand(150000, 8, seed=2), rand(8, seed=3), rand(8, seed=4), rand(150000, 8, seed=5),
          rand(150000, 8, seed=6))


def test_in_a_graph():
    x, res, w, c = rand(300, 200, seed=1, dtype=BF16), rand(300, 200, seed=2), rand(200, seed=3), rand(200, seed=4)
    dout, dtotal = rand(300, 200, seed=5, dtype=BF16), rand(300, 200, seed=6)

    def both():
        out, total = sscan.layer_norm(x, w, c, res)
        return out, total, *sscan.layer_norm_bwd(total, dout, w, c, dtotal).values()

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for seed in (7, 8, 9):
        x.copy_(rand(300, 200, seed=seed, dtype=BF16))
        want = both()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, want))


def test_refusals():
    x, w = rand(4, 64, seed=1), torch.ones(64, device=DEV)
    for args, error in (((x.cpu(),), ValueError), ((x.half(),), TypeError), ((3,), TypeError), ((x, w[:3]), ValueError),
                        ((x, w.bfloat16()), TypeError), ((x, w, w[:3]), ValueError), ((x, w, w, x[:2]), ValueError),
                        ((x, w, w, x.half()), TypeError), ((x, 5), TypeError), ((x.t(),), ValueError)):
        with pytest.raises(error):
            sscan.layer_norm(*args)
    for kw in (dict(eps=float("nan")), dict(eps=-1.0), dict(out=x), dict(residual=x, residual_out=x)):
        with pytest.raises(sscan.SScanError):
            sscan.layer_norm(x, w, **kw)
    with pytest.raises(sscan.SScanError):
        sscan.layer_norm(torch.zeros(1, 8193, device=DEV))
    for args in ((x, x[:2]), (x, x.half()), (x, 3), (x, x, w, w, x[:1])):
        with pytest.raises((ValueError, TypeError)):
            sscan.layer_norm_bwd(*args)


@pytest.mark.parametrize("size", [2, 5, 64, 120, 128, 200, 513, 1000])
@pytest.mark.parametrize("n", [5, 17, 700])
def test_without_eps(n, size):
    """eps = 0 with fewer rows than a block's threads take, whose idle ones add nothing."""
    x, dout, dtotal = rand(n, size, seed=1), rand(n, size, seed=2), rand(n, size, seed=3)
    x[:, 0] += 4.0  # no two elements next to each other in a row of two
    x[:, 1] -= 4.0
    check(x, None, 1 + rand(size, seed=4, scale=0.2), rand(size, seed=5), dout, dtotal, eps=0.0)


def test_small_rows_without_eps():
    """Rows of 2e-20 with eps = 0: 1 / sd is 5e19, whose square is beyond float32."""
    x, dout, w = rand(30, 200, seed=1, scale=2e-20), rand(30, 200, seed=2), 1 + rand(200, seed=3, scale=0.2)
    out, _ = sscan.layer_norm(x, w, None, eps=0.0)
    got = sscan.layer_norm_bwd(x, dout, w, eps=0.0)
    want = rec_ref.layer_norm(x, w, None, 0.0, dout)
    # squares of 4e-40 are rounded to multiples of 2^-149: off by 2^-150 each, so the deviation by
    # 2^-150 / 4e-40 / 2 = 9e-7 of itself, 15 U, and as much again in n and in the gradients' factors
    v, bound = want["out"]
    within(out, (v, bound + 15 * U * v.abs()), "out")
    v, bound = want["dweight"]
    within(got["dweight"], (v, bound + 15 * U * (dout.double() * want["out"][0] / w.double()).abs().sum(0)), "dweight")
    v, bound = want["dx"]
    size = (dout * w).double().abs() * (1 + want["out"][0].abs())
    within(got["dx"], (v, bound + 60 * U / 2e-20 * (size + size.mean(-1, keepdim=True) * (1 + want["out"][0].abs()))), "dx")


@pytest.mark.parametrize("size", [2, 3, 7, 64, 333, 768, 1536, 2001, 4096, 8191])
def test_rows_of_equal_values(size):
    """Whole rows of one value, whose sum is not exact, have no deviation."""
    value = 1.0 + 9999.0 * torch.rand(50, 1, generator=torch.Generator().manual_seed(size))
    value[:3, 0] = torch.tensor([1234.567, -0.1, 1e-3])
    x, c = value.expand(50, size).contiguous().to(DEV), rand(size, seed=1)
    out, _ = sscan.layer_norm(x, 1 + rand(size, seed=2), c)
    assert torch.equal(out, c.expand(50, size))
    dout = rand(50, size, seed=3)
    got = sscan.layer_norm_bwd(x, dout, torch.ones(size, device=DEV), c)
    assert not got["dweight"].any()
    # with no deviation dx = (dout - mean(dout)) / sqrt(eps): the mean within 20 U of the mean magnitude,
    # the quotient by four roundings
    d = dout.double()
    want, r = (d - d.mean(-1, keepdim=True)) / 1e-5 ** 0.5, 1e-5 ** -0.5
    within(got["dx"], (want, r * U * (20 * d.abs().mean(-1, keepdim=True) + 5 * d.abs())), "dx")


@pytest.mark.parametrize("size", [64, 333, 1536, 8191])
@pytest.mark.parametrize("shift", [100.0, 3e4])
def test_deviations_far_below_the_mean(shift, size):
    """The mean's own rounding, up to 17 U of its size, is taken out again."""
    x, dout = rand(40, size, seed=1, shift=shift), rand(40, size, seed=2)
    w = 1 + rand(size, seed=3, scale=0.2)
    out, _ = sscan.layer_norm(x, w, None)
    y = x.double() - x.double().mean(-1, keepdim=True)
    sd = (y.square().mean(-1, keepdim=True) + 1e-5).sqrt()
    # x - m for a rounded mean m: off by U of its size, which is |y| + |m - mean|, 17 U of the shift;
    # the mean of these by sixteen additions in a row and a quotient; the difference
    gap = 17 * U * (shift + 1)
    E = (2 * U * (y.abs() + gap) + 19 * U * (y.abs() + gap).mean(-1, keepdim=True)) / sd
    n = y / sd
    value = n * w.double()
    bound = w.double().abs() * (E + n.abs() * (2 * E.amax(-1, keepdim=True) + 26 * U))
    within(out, (value, bound), "out")
    # gradients at the same rounding of n: their own sums add 24 U of the mean magnitudes
    got = sscan.layer_norm_bwd(x, dout, w)
    d = dout.double()
    dn = d * w.double()
    m1, m2 = dn.mean(-1, keepdim=True), (dn * n).mean(-1, keepdim=True)
    a1, a2 = dn.abs().mean(-1, keepdim=True), (dn * n).abs().mean(-1, keepdim=True)
    Em = E.amax(-1, keepdim=True)
    dy = E + n.abs() * (2 * Em + 26 * U)
    err = dn.abs() * 4 * U + 20 * U * a1 + n.abs() * (30 * U * a2 + (dn.abs() * dy).mean(-1, keepdim=True)) + dy * a2
    err = (err + (dn.abs() + a1 + n.abs() * a2) * (2 * Em + 30 * U)) / sd
    within(got["dx"], ((dn - m1 - n * m2) / sd, err), "dx")
    within(got["dweight"], ((d * n).sum(0), (d.abs() * dy).sum(0) + 101 * U * (d * n).abs().sum(0)), "dweight")


@pytest.mark.parametrize("size", [64, 333, 2001, 8192])
@pytest.mark.parametrize("shift", [0.0, 1e30])
def test_rows_whose_squares_overflow(size, shift):
    """Deviations whose squares are beyond float32 count as infinitely far apart: 1 / sd is 0."""
    x, c, dout, dtotal = rand(20, size, seed=1, scale=1e26, shift=shift), rand(size, seed=2), rand(20, size, seed=3), \
        rand(20, size, seed=4)
    w = 1 + rand(size, seed=5, scale=0.2)
    out, _ = sscan.layer_norm(x, w, c)
    assert torch.equal(out, c.expand(20, size))
    got = sscan.layer_norm_bwd(x, dout, w, c, dtotal)
    assert torch.equal(got["dx"], dtotal) and not got["dweight"].any()
