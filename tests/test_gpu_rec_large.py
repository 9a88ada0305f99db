"""Tensors whose elements lie beyond 2^31 and 2^32 bytes, and grids of many blocks."""
import pytest
import torch

import rec_ref
from rec_ref import within
from selective_state_space_sscan_amd import sscan
from test_gpu_rec import DEV, FWD, draw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("reverse", [False, True])
def test_far_batch_rows_and_tokens(reverse):
    """Rows 2.4e9 elements apart and tokens 2^24 apart, read through views of one buffer."""
    b, l, d = 2, 100, 130
    t = draw(b, l, d, torch.bfloat16, seed=31)
    step = 1 << 24
    buf = torch.zeros(l * step + 8 * d + (1 << 31), dtype=torch.bfloat16, device=DEV)
    views = dict(t)
    for k, name in enumerate(("x", "g", "i", "z")):
        views[name] = buf.as_strided((b, l, d), ((1 << 31) + 777, step, 1), 2 * d * k + 1)
        views[name].copy_(t[name])
    for src in (t, views):
        src["out"] = sscan.rec_fwd(*(src[k] for k in FWD[:5]), h0=t["h0"], reverse=reverse)
        src["grads"] = sscan.rec_bwd(src["x"], src["g"], t["dout"], src["i"], t["lam"], src["z"], t["h0"], reverse=reverse)
    assert all(torch.equal(p, q) for p, q in zip(t["out"], views["out"]))
    assert all(torch.equal(t["grads"][k], views["grads"][k]) for k in t["grads"])


def test_outputs_beyond_4_gib():
    """3 x 200000 x 4098 bfloat16: 4.9 GB a tensor; the last row's last tokens against float64."""
    b, l, d = 3, 200000, 4098
    gen = torch.Generator(device=DEV).manual_seed(1)
    x, g = (torch.randn(b, l, d, device=DEV, dtype=torch.bfloat16, generator=gen) for _ in range(2))
    lam = torch.full((d,), -3.0, device=DEV)  # forgets within a few hundred tokens
    out, h_last, kept = sscan.rec_fwd(x, g, lam=lam, keep=True)
    tail = slice(l - 3000, l)
    want = rec_ref.rec(x[2:, tail], g[2:, tail], lam=lam)
    near = slice(2000, 3000)  # the state 2000 tokens before has decayed to nothing (0.68^1000)
    within(out[2:, tail][:, near], tuple(v[:, near] for v in want["out"]), "out")
    within(h_last[2:], want["h_last"], "h_last")
    q, scale, _ = rec_ref.eight(x[2, -5:].cpu())
    assert torch.equal(kept.x.q[2, -5:].cpu(), q) and torch.equal(kept.x.scale[2, -5:].cpu(), scale)
    del g, kept
    p = sscan.pack8(x)
    assert torch.equal(p.q[2, -5:].cpu(), q)
    back = sscan.unpack8(p, torch.bfloat16)
    assert torch.equal(back[2, -5:].cpu(), (q.float() * scale.repeat_interleave(64, -1)[:, :d]).bfloat16())
    del back, p
    dout = x  # any values
    r = sscan.rec_bwd(out, x, dout, lam=lam)
    head = slice(0, 3000)  # adjoints of the first tokens do not see further
    want = rec_ref.rec_bwd(out[2:, head], x[2:, head], dout[2:, head], lam=lam)
    within(r["dx"][2:, :1000], tuple(v[:, :1000] for v in want["dx"]), "dx")
    within(r["dg"][2:, :1000], tuple(v[:, :1000] for v in want["dg"]), "dg")


def test_many_rows():
    b, l, d = 30000, 5, 70
    t = draw(b, l, d, torch.float32, seed=32)
    out, h_last = sscan.rec_fwd(*(t[k] for k in FWD[:5]), h0=t["h0"])
    want = rec_ref.rec(*(t[k] for k in FWD))
    within(out, want["out"], "out")
    within(h_last, want["h_last"], "h_last")
    got = sscan.rec_bwd(t["x"], t["g"], t["dout"], t["i"], t["lam"], t["z"], t["h0"], t["dh_last"])
    want = rec_ref.rec_bwd(t["x"], t["g"], t["dout"], t["i"], t["lam"], t["z"], t["h0"], t["dh_last"])
    for k, v in want.items():
        within(got[k], v, k)
