"""The last state in the entry state's place, where rows are walked in segments: blocks that
read the entry state and blocks that write the last one belong to one launch.  In place
equals out of place, bit for bit."""
import pytest
import torch

from selective_state_space_sscan_amd import sscan
from test_gpu_delta import DEV, inputs, on, state

pytestmark = pytest.mark.gpu


def both(ins, h0, n, **kw):
    out, last = sscan.delta_fwd(*ins, h0=h0, lengths=n, **kw)
    s = h0.clone()
    out2, last2 = sscan.delta_fwd(*ins, h0=s, h_last=s, lengths=n, **kw)
    torch.cuda.synchronize()
    assert last2 is s and torch.equal(out, out2) and torch.equal(last, s)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", [(64, 48), (128, 130), (33, 50)])
def test_rows_that_leave_segments_empty(dk, dv, dtype):
    """Rows that end in the first, a middle and the last segment, on a segment's edge, at
    once, and not at all: the last segments of short rows have nothing to walk."""
    shape = (6, 1300, 1, 2, dk, dv)
    plan = sscan.delta_plan(*shape, io_dtype=dtype)
    assert plan["nseg"] > 2, plan
    edge = 64 * plan["seg_chunks"]
    print("in place", shape, dtype, plan, flush=True)
    n = torch.tensor([1300, 7, edge, 1290, 0, 2 * edge + 1], dtype=torch.int32)
    both(on(*inputs(*shape, dtype, seed=21, g_scale=0.02)), state(6, 2, dk, dv).to(DEV), n.to(DEV))


def random_rows(b, L, hk, hv, dk, dv):
    gen = torch.Generator(device=DEV).manual_seed(5)
    q, k, v = (torch.randn(b, L, h, d, device=DEV, generator=gen).bfloat16() for h, d in ((hk, dk), (hk, dk), (hv, dv)))
    g = -0.05 * torch.rand(b, L, hv, device=DEV, generator=gen)
    beta = torch.rand(b, L, hv, device=DEV, generator=gen)
    return [q, k, v, g, beta], torch.randn(b, hv, dk, dv, device=DEV, generator=gen)


# two segments, between which there is no chain; twelve heads in seven segments, 504 blocks
# of a CU's whole LDS
@pytest.mark.parametrize("shape,nseg", [((259, 3450, 1, 1, 128, 72), 2), ((261, 3267, 1, 1, 128, 16), 2),
                                        ((3, 65536, 1, 12, 128, 256), 7)])
def test_more_blocks_than_the_gpu_holds(shape, nseg):
    """A head's segments do not all run at once."""
    b, L, hk, hv, dk, dv = shape
    plan = sscan.delta_plan(*shape)
    assert plan["nseg"] == nseg and b * hv * nseg * (-(-dv // (16 * plan["waves"]))) > 256, plan
    print("in place", shape, plan, flush=True)
    ins, h0 = random_rows(*shape)
    both(ins, h0, None, qk_norm=True)
    n = torch.tensor([300, L, L // 3] * b, dtype=torch.int32, device=DEV)[:b].contiguous()
    both(ins, h0, n, qk_norm=True)
