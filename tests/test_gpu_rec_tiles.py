"""The recurrence's kernels with tiles of sixteen tokens, which large calls run, and inputs kept
in 8 bits over rows of several runs of segments, against float64."""
import pytest
import torch

import rec_ref
from rec_ref import within
from selective_state_space_sscan_amd import sscan
from test_gpu_rec import check_backward, check_forward, draw, forward

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def workspace_of(b, l, d, tokens):
    """The forward's workspace where a wave's tile holds `tokens` tokens: two words of 64 bits
    for every segment that a row has beyond sixteen tiles, and for every run of eight."""
    lane = 2 - d % 2
    tiles = -(-l // tokens)
    if tiles <= 16:
        return 0
    segments = -(-tiles // 8)
    return (segments + segments // 8) * b * -(-d // (64 * lane)) * 64 * lane * 8 + 256


def ragged(b, l):
    return [(l, 0, l - 1, 17, 1, l // 2, 16, 2 * l)[k % 8] for k in range(b)]


# three runs of segments and a rest, odd channels, and many short rows whose one segment has
# sixteen waves; float32 has tiles of sixteen with odd channels alone
SIZES = [(4, 1030, 1152, BF16), (4, 1030, 1153, BF16), (4, 1030, 1153, F32), (160, 250, 130, BF16), (160, 250, 65, BF16),
         (160, 250, 65, F32), (1, 2100, 2050, BF16)]


@pytest.mark.parametrize("gated,reverse,parts,short", [(True, False, "izhl", False), (True, True, "izhl", True),
                                                       (False, False, "", True), (False, True, "ih", False),
                                                       (True, False, "zl", True)])
@pytest.mark.parametrize("b,l,d,dtype", SIZES)
def test_tiles_of_sixteen(b, l, d, dtype, gated, reverse, parts, short):
    print("rec tiles", b, l, d, dtype, gated, reverse, parts, short, flush=True)
    # that the call does run them, whatever becomes of the rule
    assert sscan.rec_workspace_bytes(b, l, d, dtype) == workspace_of(b, l, d, 16) != workspace_of(b, l, d, 8)
    t = draw(b, l, d, dtype, seed=l + d, gated=gated, parts=parts, lengths=ragged(b, l) if short else None)
    check_forward(t, reverse=reverse)
    check_backward(t, reverse=reverse)


KEPT = [(2, 1100, 256, BF16), (2, 1100, 260, BF16), (2, 1100, 131, BF16), (1, 1100, 131, F32), (1, 1100, 130, F32),
        (2, 650, 130, BF16), (4, 1030, 1152, BF16), (4, 1030, 1153, F32)]


@pytest.mark.parametrize("gated,reverse,parts,short", [(True, False, "izhl", False), (True, True, "izhl", True),
                                                       (False, False, "", False), (False, True, "zl", True)])
@pytest.mark.parametrize("b,l,d,dtype", KEPT)
def test_kept_over_runs_of_segments(b, l, d, dtype, gated, reverse, parts, short):
    """Two runs of eight segments of 64 tokens and more: what is kept of the rows' tokens are the
    inputs in 8 bits, and the gradients are those there."""
    print("rec kept", b, l, d, dtype, gated, reverse, parts, short, flush=True)
    t = draw(b, l, d, dtype, seed=l + d, gated=gated, parts=parts, lengths=ragged(b, l) if short else None)
    out, h_last, kept = forward(t, keep=True, reverse=reverse)
    plain = forward(t, reverse=reverse)
    assert torch.equal(out, plain[0]) and torch.equal(h_last, plain[1])
    rows = [l] * b if not short else [min(n, l) for n in ragged(b, l)]
    back = dict(t)
    for k, p in zip(("x", "g", "i", "z"), kept):
        assert (p is None) == (t[k] is None)
        if p is not None:
            q, scale, value = rec_ref.eight(t[k].cpu())
            for row, n in enumerate(rows):
                assert torch.equal(p.q[row, :n].cpu(), q[row, :n]) and torch.equal(p.scale[row, :n].cpu(), scale[row, :n]), k
            back[k] = value.to(t["x"].device)
    got = sscan.rec_bwd(kept.x, kept.g, t["dout"], kept.i, t["lam"], kept.z, t["h0"], t["dh_last"], t["lengths"],
                        reverse=reverse)
    want = rec_ref.rec_bwd(back["x"], back["g"], t["dout"], back["i"], t["lam"], back["z"], t["h0"], t["dh_last"],
                           t["lengths"], reverse=reverse)
    for k, v in want.items():
        # a value in 8 bits is itself rounded to float32: half a step of it, within every bound
        within(got[k], (v[0], v[1] * 1.25), k)
