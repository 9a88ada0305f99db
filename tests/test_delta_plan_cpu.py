"""How the gated delta rule's walks are planned, without a GPU: which calls need a workspace,
and what ``delta_plan`` says of the sizes that the GPU tests rely on."""
import pytest
import torch

from selective_state_space_sscan_amd import sscan
from test_delta_abi_cpu import bwd, fwd, lib  # noqa: F401

RECURRENT = 10  # tokens up to which a call goes token by token


@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("L", [2, 9, RECURRENT, RECURRENT + 1, 12])
def test_workspaces_of_few_tokens(lib, L, io):  # noqa: F811
    n = lib.sscan_delta_workspace_bytes(2, L, 1, 2, 64, 64, io)
    assert (n > 0) == (L > RECURRENT)
    assert fwd(lib, b=2, L=L, hk=1, hv=2, dk=64, dv=64, io=io, ws=None if n == 0 else 1 << 42, ws_bytes=n) == 0
    back = lib.sscan_delta_bwd_workspace_bytes(2, L, 1, 2, 64, 64, io)
    assert back > 0 and bwd(lib, b=2, L=L, hk=1, hv=2, dk=64, dv=64, io=io, ws=1 << 42, ws_bytes=back) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", [(1, 10, 1, 1, 64, 64), (1, 11, 1, 1, 64, 64), (2, 640, 8, 16, 128, 128),
                                   (1, 32768, 8, 16, 128, 128), (5, 1300, 1, 1, 128, 130), (3, 65536, 1, 12, 128, 256)])
def test_plan_covers_the_chunks(lib, sizes, dtype):  # noqa: F811
    p = sscan.delta_plan(*sizes, io_dtype=dtype)
    chunks = -(-sizes[1] // 64)
    if sizes[1] <= RECURRENT:
        assert p["nchunk"] == 0
        return
    assert p["nchunk"] == chunks and p["waves"] in (4, 8)
    assert p["nseg"] >= 1 and (p["nseg"] - 1) * p["seg_chunks"] < chunks <= p["nseg"] * p["seg_chunks"]


def test_plan_refusals(lib):  # noqa: F811
    for bad in ((-1, 10, 1, 1, 64, 64), (1, 10, 2, 3, 64, 64), (1, 10, 1, 1, 129, 64), (1, 10, 1, 1, 64, 300)):
        with pytest.raises(sscan.SScanError):
            sscan.delta_plan(*bad)
    assert lib.sscan_delta_plan(1, 10, 1, 1, 64, 64, 0, None) == -1
    assert sscan.delta_plan(0, 100, 1, 1, 64, 64)["nchunk"] == 0
