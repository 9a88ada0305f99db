"""Activations in 8 bits: whole steps and scales exactly as float32 arithmetic on the CPU has them."""
import pytest
import torch

import rec_ref
from selective_state_space_sscan_amd import sscan

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def same(a, b):
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def check(x):
    p = sscan.pack8(x)
    q, scale, value = rec_ref.eight(x.cpu())
    assert torch.equal(p.q.cpu(), q) and same(p.scale.cpu(), scale)
    for dtype in (torch.float32, torch.bfloat16):
        back = sscan.unpack8(p, dtype)
        assert back.dtype == dtype and same(back.cpu(), (q.float() * scale.repeat_interleave(64, -1)[..., :x.shape[-1]]).to(dtype))
    return p


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(1,), (64,), (65,), (3, 63), (5, 128), (2, 3, 200), (7, 1), (1, 8191), (1000, 66),
                                   (300, 1536), (4, 100000)])
def test_shapes(shape, dtype):
    x = torch.randn(shape, generator=torch.Generator().manual_seed(1)) * torch.exp(torch.arange(shape[-1]) % 7 - 3.0)
    check(x.to(dtype).to(DEV))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_far_values(dtype):
    x = torch.randn(8, 192, generator=torch.Generator().manual_seed(2)).to(dtype)
    x[0, :64] = 0.0
    x[1, 70] = float("inf")
    x[2, 70] = -float("inf")
    x[3, 130] = float("nan")
    x[4, :64] *= 1e-35
    x[5, :64] *= 1e35
    x[6, 64:128] = torch.finfo(dtype).max
    x[7, 64:128] = -2.0 ** -100
    p = check(x.to(DEV))
    back = sscan.unpack8(p)
    assert not back[0, :64].any() and torch.isnan(back[1, 64:128]).all() and torch.isfinite(back[1, :64]).all()
    assert not back[4, :64].any() and torch.isfinite(back[5]).all() and back[7, 64:128].all()


def test_strided_rows_and_given_outputs():
    x = torch.randn(6, 5, 300, device=DEV)
    assert torch.equal(sscan.pack8(x[..., 3:203]).q, sscan.pack8(x[..., 3:203].contiguous()).q)
    row = x[:1, :1, :100].expand(6, 5, 100)
    assert torch.equal(sscan.pack8(row).q, sscan.pack8(row.contiguous()).q)
    p = sscan.pack8(x)
    held = sscan.Packed8(torch.empty_like(p.q), torch.empty_like(p.scale))
    version = held.q._version
    assert sscan.pack8(x, out=held) is held and torch.equal(held.q, p.q) and held.q._version > version
    out = torch.empty_like(x)
    assert sscan.unpack8(p, torch.float32, out=out) is out and torch.equal(out, sscan.unpack8(p))
    for shape in ((0, 64), (3, 0)):
        e = sscan.pack8(torch.zeros(shape, device=DEV))
        assert sscan.unpack8(e).shape == shape


def test_refusals():
    x = torch.randn(4, 6, 100, device=DEV)
    p = sscan.pack8(x)
    for bad, error in ((x.cpu(), ValueError), (x.half(), TypeError), (3, TypeError), (x[0, 0, 0], ValueError),
                       (x.transpose(1, 2), ValueError), (x.transpose(0, 1), ValueError)):
        with pytest.raises(error):
            sscan.pack8(bad)
    for bad, error in ((p.q, TypeError), (sscan.Packed8(p.q, p.scale[..., :1]), ValueError),
                       (sscan.Packed8(p.q.float(), p.scale), TypeError), (sscan.Packed8(p.q, p.q), TypeError),
                       (sscan.Packed8(p.q, 2), TypeError)):
        with pytest.raises(error):
            sscan.unpack8(bad)
    with pytest.raises(TypeError):
        sscan.unpack8(p, torch.float16)
    with pytest.raises(TypeError):
        sscan.unpack8(p, torch.bfloat16, out=x)
    with pytest.raises(TypeError):
        sscan.pack8(x, out=(p.q, p.scale))
