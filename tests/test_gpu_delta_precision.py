"""bfloat16 outputs of the gated delta rule come from float32 values: where the parts of an
output cancel, what is left keeps its bits.

Tolerances, from the number formats: a factor cut to sixteen bits is off by up to 2^-17 of
itself, so sums of n such terms of size 1 are off by about 2^-17 sqrt(n / 3), 5e-5 for the
sums here; float32 sums stay within n 2^-24 of their largest partial sum.
"""
import pytest
import torch

import delta_ref
from selective_state_space_sscan_amd import sscan

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("rows", [1, 512])  # 512 rows of two chunks: the walks of eight waves
@pytest.mark.parametrize("dk", [64, 128])
def test_queries_against_a_state_that_cancels(dk, rows):
    """beta = 0, g = 0: every output is scale q . S of the entry state, whose rows come in
    pairs x, -x + 1e-5."""
    gen = torch.Generator().manual_seed(dk)
    L, dv = 80, 128
    sign = torch.randint(0, 2, (1, L, 1, dk // 2), generator=gen).repeat_interleave(2, -1) * 2 - 1
    q = sign.bfloat16()
    k = torch.randn(1, L, 1, dk, generator=gen).bfloat16()
    v = torch.randn(1, L, 1, dv, generator=gen).bfloat16()
    g = beta = torch.zeros(1, L, 1)
    x = 1 + torch.rand(1, 1, dk // 2, dv, generator=gen)
    h0 = torch.stack([x, 1e-5 * torch.randn(x.shape, generator=gen) - x], 3).reshape(1, 1, dk, dv)
    ref, _ = delta_ref.delta(q, k, v, g, beta, h0, scale=1.0)
    print("delta_fwd, cancelling state", rows, dk, flush=True)
    out, last = sscan.delta_fwd(*[t.to(DEV).expand(rows, *t.shape[1:]) for t in (q, k, v, g, beta)],
                                h0=h0.to(DEV).repeat(rows, 1, 1, 1), scale=1.0)
    assert torch.equal(last, h0.to(DEV).expand_as(last))
    assert torch.equal(out, out[:1].expand_as(out))
    err = (out[:1].cpu().double() - ref).abs()
    # partial sums of the pairs stay below 2
    worst = float((err / (2.0 ** -8 * ref.abs() + dk * 2.0 ** -24 * 2)).max())
    assert worst <= 1.0, worst


def test_a_chunks_own_values_against_its_entry_state():
    """Thirty-two rows of the state are written inside the chunk (one-hot keys, beta = 1), the
    others entered it as what cancels them: both the state's part of an output and the
    chunk's own have to be exact."""
    gen = torch.Generator().manual_seed(1)
    L, dk, dv, n = 64, 64, 128, 32
    k = torch.zeros(1, L, 1, dk)
    k[0, torch.arange(n), 0, torch.arange(n)] = 1.0
    q = torch.ones(1, L, 1, dk)
    v = torch.randn(1, L, 1, dv, generator=gen).bfloat16()
    g = -0.05 * torch.rand(1, L, 1, generator=gen)
    beta = torch.zeros(1, L, 1)
    beta[0, :n] = 1.0
    decay = torch.exp(-g.double().cumsum(1)[0, :n])  # of row j's value back to the chunk's start
    h0 = torch.randn(1, 1, dk, dv, generator=gen)
    h0[0, 0, n:] = (-decay * v[0, :n, 0].double()).float() + 1e-5 * torch.randn(n, dv, generator=gen)
    ins = (q.bfloat16(), k.bfloat16(), v, g, beta)
    ref, _ = delta_ref.delta(*ins, h0, scale=1.0)
    out, _ = sscan.delta_fwd(*[t.to(DEV) for t in ins], h0=h0.to(DEV), scale=1.0)
    err, want = out.cpu().double()[:, n:] - ref[:, n:], ref[:, n:]
    # 96 terms of size 1, each with some roundings of its exponentials and factors
    rms = float(err.square().mean().sqrt())
    assert rms <= 2.0 ** -8 * float(want.square().mean().sqrt()) + 96 ** 0.5 * 8 * 2.0 ** -24, rms
