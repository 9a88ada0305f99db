"""Per-head weights of very many heads: their gradient's sums walk over heads and columns."""
import pytest
import torch

from selective_state_space_sscan_amd import sscan

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("rows,heads,size", [(2, 3000, 360), (1, 65536, 1024), (1, 1 << 20, 67)])
def test_gradients_of_weights_per_head(rows, heads, size):
    """The last two have 2^22 and more groups of sixteen columns.  With the gate after the
    norm and as few rows each weight's gradient is a sum of a term or two; float32 roundings
    and the gate's sigmoid leave 1e-5 of the terms."""
    print("weights per head", rows, heads, size, flush=True)
    gen = torch.Generator(device=DEV).manual_seed(heads)
    x, z, dout = (torch.randn(rows, heads, size, device=DEV, generator=gen).bfloat16() for _ in range(3))
    w = 1 + 0.2 * torch.randn(heads, size, device=DEV, generator=gen)
    r = sscan.gated_norm_bwd(x, z, dout, w, eps=1e-6)
    torch.cuda.synchronize()
    pick = torch.tensor([0, 1, heads // 3, heads // 2 + 1, heads - 2, heads - 1], device=DEV)
    xs, zs, ds = (t[:, pick].double() for t in (x, z, dout))
    n = xs / (xs.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    terms = ds * n * zs * torch.sigmoid(zs)
    err = (r["dweight"][pick].double() - terms.sum(0)).abs()
    assert float((err / (1e-5 * terms.abs().sum(0) + 1e-12)).max()) <= 1.0
    # and all of them: against the same terms in float32
    step = max(1, heads // 64)
    for h in range(0, heads, step):
        xs, zs, ds = (t[:, h:h + step].float() for t in (x, z, dout))
        t = ds * xs * torch.rsqrt(xs.square().mean(-1, keepdim=True) + 1e-6) * zs * torch.sigmoid(zs)
        assert bool(((r["dweight"][h:h + step] - t.sum(0)).abs() <= 2e-5 * t.abs().sum(0) + 1e-12).all()), h


@pytest.mark.parametrize("shape", [(1, (1 << 20) + 7, 24), (2, 3000, 40), (3, 1025, 1, 40)])
def test_tokens_are_no_heads(shape):
    """[batch, len, size] of any length, and gradients whose workspace does not grow with it."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    x, dout = (torch.randn(*shape, device=DEV, generator=gen).bfloat16() for _ in range(2))
    z = torch.randn(*shape[:-1], shape[-1] + 8, device=DEV, generator=gen).bfloat16()[..., 8:]
    w = 1 + 0.2 * torch.randn(shape[-1], device=DEV, generator=gen)
    flat = [t.reshape(-1, shape[-1]) for t in (x, z, dout)]
    y, want = sscan.gated_norm(x, z, w), sscan.gated_norm(*flat[:2], w)
    assert torch.equal(y.view_as(want), want)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    r = sscan.gated_norm_bwd(x, z, dout, w)
    assert torch.cuda.max_memory_allocated() - before <= 2 * x.numel() * 2 + (1 << 21)
    want = sscan.gated_norm_bwd(*flat, w)
    for name in ("dx", "dz", "dweight"):
        assert torch.equal(r[name].view_as(want[name]), want[name]), name
