"""The entry points under another default dtype than float32, as model code often sets."""
import contextlib

import pytest
import torch

from selective_state_space_sscan_amd import sscan


@contextlib.contextmanager
def default(dtype):
    old = torch.get_default_dtype()
    torch.set_default_dtype(dtype)
    try:
        yield
    finally:
        torch.set_default_dtype(old)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float64])
def test_scales_are_float32(dtype):
    with default(dtype):
        kept = sscan._kept_new(torch.device("cpu"), (2, 3, 100), (True, True, False, True))
    assert kept.i is None
    for p in (kept.x, kept.g, kept.z):
        assert p.q.dtype == torch.int8 and p.q.shape == (2, 3, 100)
        assert p.scale.dtype == torch.float32 and p.scale.shape == (2, 3, 2) and p.scale.is_contiguous()


def calls():
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float32).to("cuda")
    x, g, i, z, dout = (r(2, 70, 130).bfloat16().requires_grad_(k < 4) for k in range(5))
    lam, h0 = r(130), r(2, 130)
    out, last = sscan.gated_recurrence(x, g, i, lam, z, h0, checkpoint=True)
    yield from (out, last, *torch.autograd.grad([out, last], [x, g, i, z], [dout, h0]))
    out, last, kept = sscan.rec_fwd(x, g, i, lam, z, h0, keep=True)
    yield from (t for p in kept for t in p)
    yield from sscan.rec_bwd(x, g, dout, i, lam, z, h0, h0).values()
    yield sscan.rec_step(h0.clone(), x[:, 0], g[:, 0], lam=lam)
    p = sscan.pack8(x)
    yield from (*p, sscan.unpack8(p))
    w = r(130)
    out, total = sscan.layer_norm(x, w, w, r(2, 70, 130))
    yield from (out, total, *sscan.layer_norm_bwd(total, dout, w, w).values())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float64])
def test_calls_do_not_see_it(dtype):
    want = list(calls())
    with default(dtype):
        got = list(calls())
    assert len(want) == len(got)
    for p, q in zip(want, got):
        assert p.dtype == q.dtype and torch.equal(p, q)
