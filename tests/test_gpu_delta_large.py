"""The gated delta rule's kernels at the sizes that training, prefill and full batches take:
walks of eight waves a block (bf16, more than 64 value columns, 1024 chunks or more in all
rows and heads), whole and in segments, and the token kernel in blocks of four waves.  The
float64 recurrence is computed for some rows and heads; the tolerances are delta_ref's."""
import pytest
import torch

import delta_ref
from delta_ref import close
from selective_state_space_sscan_amd import sscan
from test_gpu_delta import DEV, inputs, on, state
from test_gpu_delta_bwd import NAMES, reference

pytestmark = pytest.mark.gpu

# b, L, hk, hv, dk, dv; segments or whole; rows' lengths (None: all); sampled (row, key head)
WALKS = [
    ((64, 65, 8, 16, 128, 128), False, None, [(0, 0), (63, 7), (17, 3)]),
    ((32, 130, 16, 32, 64, 72), False, [130, 64, 1, 0] + [129, 65] * 14, [(0, 0), (1, 15), (2, 1), (3, 2), (31, 9)]),
    ((64, 100, 16, 16, 33, 200), False, None, [(5, 11)]),  # elements loaded by themselves
    ((2, 2100, 8, 16, 128, 128), True, [2100, 700], [(0, 7), (1, 0)]),
    ((2, 2100, 16, 16, 64, 200), True, None, [(1, 15)]),
    ((2, 2100, 16, 16, 64, 100), True, [2099, 1], [(0, 4), (1, 3)]),
]


def sample(ins, row, key, share):
    q, k, v, g, beta = ins
    hs = slice(key * share, (key + 1) * share)
    return [x[row:row + 1, :, key:key + 1] for x in (q, k)] + [x[row:row + 1, :, hs] for x in (v, g, beta)], hs


def setup(shape, segments, lengths):
    b, L, hk, hv, dk, dv = shape
    plan = sscan.delta_plan(*shape)
    assert plan["waves"] == 8 and (plan["nseg"] > 2 if segments else plan["nseg"] == 1), plan
    print("walks of eight waves", shape, plan, flush=True)
    ins = inputs(*shape, torch.bfloat16, seed=L + dv, g_scale=0.05 if segments else 0.3)
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    return ins, state(b, hv, dk, dv), n


@pytest.mark.parametrize("shape,segments,lengths,sampled", WALKS)
def test_forward_of_eight_waves(shape, segments, lengths, sampled):
    ins, h0, n = setup(shape, segments, lengths)
    out, last = sscan.delta_fwd(*on(*ins), *on(h0, n))
    torch.cuda.synchronize()
    assert torch.isfinite(out).all() and torch.isfinite(last).all()
    for row, key in sampled:
        some, hs = sample(ins, row, key, shape[3] // shape[2])
        ref, ref_last = delta_ref.delta(*some, h0[row:row + 1, hs], None if n is None else n[row:row + 1])
        close(out[row:row + 1, :, hs], ref, f"out of {row}, {key}")
        close(last[row:row + 1, hs], ref_last, f"h_last of {row}, {key}")


BACK = [
    ((64, 65, 8, 16, 128, 128), False, None, [(0, 0), (63, 7)]),
    ((32, 130, 16, 32, 64, 72), False, [130, 64, 1, 0] + [129, 65] * 14, [(0, 0), (1, 15), (3, 2), (31, 9)]),
    ((64, 100, 16, 16, 33, 200), False, None, [(5, 11)]),
    ((2, 2100, 8, 16, 96, 72), True, [2100, 700], [(0, 7), (1, 0)]),
    ((2, 2100, 16, 16, 64, 100), True, None, [(1, 15)]),
]


@pytest.mark.parametrize("shape,segments,lengths,sampled", BACK)
def test_gradients_of_eight_waves(shape, segments, lengths, sampled):
    b, L, hk, hv, dk, dv = shape
    ins, h0, n = setup(shape, segments, lengths)
    dh = state(b, hv, dk, dv, seed=8)
    dout = torch.randn(b, L, hv, dv, generator=torch.Generator().manual_seed(99)).bfloat16()
    r = sscan.delta_bwd(*on(*ins, dout), h0=on(h0)[0], dh_last=on(dh)[0], lengths=on(n)[0])
    torch.cuda.synchronize()
    for row, key in sampled:
        some, hs = sample(ins, row, key, hv // hk)
        rows = slice(row, row + 1)
        refs = reference(some, dout[rows, :, hs], h0[rows, hs], dh[rows, hs], lengths=None if n is None else n[rows])
        for name, ref in zip(NAMES, refs):
            heads = slice(key, key + 1) if name in ("dq", "dk") else hs
            got = r[name][rows, heads] if name == "dh0" else r[name][rows, :, heads]
            close(got, ref, f"{name} of {row}, {key}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("b,L,hk,hv,dk,dv", [(43, 1, 3, 3, 64, 130), (131, 1, 1, 4, 33, 50), (67, 1, 2, 4, 128, 128),
                                             (35, 9, 1, 3, 64, 132)])
def test_tokens_of_full_batches(b, L, hk, hv, dk, dv, dtype):
    """More than 512 waves: blocks of four, the last of them with a rest."""
    waves = b * hv * (-(-dv // 32))
    assert waves > 512
    ins = inputs(b, L, hk, hv, dk, dv, dtype, seed=b, unit=False)
    s = state(b, hv, dk, dv)
    got = s.to(DEV)
    print("tokens", b, L, hk, hv, dk, dv, dtype, flush=True)
    if L == 1:
        out = sscan.delta_step(got, *[x[:, 0] for x in on(*ins)], qk_norm=True)[:, None]
    else:
        out, _ = sscan.delta_fwd(*on(*ins), h0=got, h_last=got, qk_norm=True)
    ref, ref_s = delta_ref.delta(*ins, s, qk_norm=True)
    close(out, ref, "out")
    close(got, ref_s, "state")
