"""Alignment of the states that the gated delta rule's C entry points take, without a GPU."""
from test_delta_abi_cpu import EALIGN, OK, bwd, delta, fwd, lib  # noqa: F401


def test_gradients_of_states_need_their_own_alignment_only(lib):  # noqa: F811
    _, r = delta()
    for at in (4, 8, 12):
        assert bwd(lib, dh=r["dh"] + at) == OK and bwd(lib, dh0=r["dh0"] + at) == OK
    assert bwd(lib, dh=r["dh"] + 2) == EALIGN and bwd(lib, dh0=r["dh0"] + 1) == EALIGN
    # the entry and last states are read and written sixteen bytes at a time
    assert fwd(lib, last=r["last"] + 8) == EALIGN and bwd(lib, h0=r["last"] + 8) == EALIGN
