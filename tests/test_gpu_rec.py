"""The gated recurrence, its gradients and its single tokens against float64."""
import itertools

import pytest
import torch

import rec_ref
from rec_ref import within
from selective_state_space_sscan_amd import sscan

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def draw(b, l, d, dtype, seed=0, gated=True, parts="izhl", lengths=None):
    """Inputs on the device by name; parts: i, z, h (entry state), l (gradient of the last state)."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    t = dict(x=r(b, l, d), g=r(b, l, d) if gated else -torch.exp(-6.9 * torch.rand(b, l, d, generator=gen)),
             i=r(b, l, d) if "i" in parts else None, z=r(b, l, d) if "z" in parts else None, dout=r(b, l, d))
    t = {k: None if v is None else v.to(dtype) for k, v in t.items()}
    lam = torch.log(torch.expm1(-torch.log(0.9 + 0.099 * torch.rand(d, generator=gen)) / 8))
    t.update(lam=lam if gated else None, h0=r(b, d) if "h" in parts else None, dh_last=r(b, d) if "l" in parts else None,
             lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32))
    return {k: None if v is None else v.to(DEV) for k, v in t.items()}


FWD = ("x", "g", "i", "lam", "z", "h0", "lengths")


def forward(t, **kw):
    return sscan.rec_fwd(*(t[k] for k in FWD[:5]), h0=t["h0"], lengths=t["lengths"], **kw)


def backward(t, **kw):
    return sscan.rec_bwd(t["x"], t["g"], t["dout"], t["i"], t["lam"], t["z"], t["h0"], t["dh_last"], t["lengths"], **kw)


def check_forward(t, name="", **kw):
    out, h_last = forward(t, **kw)
    want = rec_ref.rec(*(t[k] for k in FWD), **kw)
    within(out, want["out"], name + "out")
    within(h_last, want["h_last"], name + "h_last")
    return out, h_last


def check_backward(t, name="", **kw):
    got = backward(t, **kw)
    want = rec_ref.rec_bwd(t["x"], t["g"], t["dout"], t["i"], t["lam"], t["z"], t["h0"], t["dh_last"], t["lengths"], **kw)
    for k in ("dx", "dg", "di", "dz", "dlam", "dh0"):
        assert (got[k] is None) == (k not in want), k
        if got[k] is not None:
            within(got[k], want[k], name + k)
    return got


# one token to several segments, channels from one to odd and whole tiles
SIZES = [(1, 1, 1), (2, 5, 3), (3, 77, 384), (1, 15, 66), (1, 16, 64), (2, 17, 65), (1, 333, 70), (2, 1000, 130),
         (1, 128, 256), (3, 129, 7), (1, 4097, 64), (4, 64, 1000), (70, 3, 2), (1, 2050, 2)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("b,l,d", SIZES)
def test_sizes(b, l, d, dtype):
    print("rec", b, l, d, dtype, flush=True)
    for gated, reverse in itertools.product([True, False], repeat=2):
        t = draw(b, l, d, dtype, seed=l + d, gated=gated)
        check_forward(t, f"{gated} {reverse} ", reverse=reverse)
        check_backward(t, f"{gated} {reverse} ", reverse=reverse)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("parts", ["", "i", "z", "iz", "h", "l", "izl"])
def test_parts(parts, gated, dtype):
    t = draw(2, 300, 130, dtype, seed=5, gated=gated, parts=parts)
    check_forward(t)
    check_backward(t)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("d", [130, 65, 64])
def test_lengths(d, reverse, dtype):
    """Rows of no tokens, one, some, all and (clamped) more than all; what lies past a row's
    end is not read."""
    lengths = [0, 1, 200, 300, 1000, -5, 299, 17]
    t = draw(8, 300, d, dtype, seed=6, lengths=lengths)
    for row, n in enumerate(lengths):
        for k in ("x", "g", "i", "z", "dout"):
            t[k][row, min(max(n, 0), 300):] = float("nan")
    clean = {k: torch.where(torch.isnan(v), torch.zeros_like(v), v) if v is not None and v.is_floating_point() else v
             for k, v in t.items()}
    out, h_last = forward(t, reverse=reverse)
    want = rec_ref.rec(*(clean[k] for k in FWD), reverse=reverse)
    within(out, want["out"], "out")
    within(h_last, want["h_last"], "h_last")
    got = backward(t, reverse=reverse)
    want = rec_ref.rec_bwd(clean["x"], clean["g"], clean["dout"], clean["i"], clean["lam"], clean["z"], clean["h0"],
                           clean["dh_last"], clean["lengths"], reverse=reverse)
    for k, v in want.items():
        within(got[k], v, k)
    for row, n in enumerate(lengths):
        n = min(max(n, 0), 300)
        assert not out[row, n:].any() and not any(got[k][row, n:].any() for k in ("dx", "dg", "di", "dz"))
        if n == 0:
            assert torch.equal(h_last[row], t["h0"][row]) and torch.equal(got["dh0"][row], t["dh_last"][row])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_views(dtype):
    """Slices of a packed projection at odd offsets, a batch-second layout, broadcast inputs."""
    b, l, d = 3, 150, 66
    t = draw(b, l, d, dtype, seed=7)
    packed = torch.zeros(b, l, 4 * d + 7, dtype=dtype, device=DEV)
    views = dict(t)
    for k, name in enumerate(("x", "g", "i", "z")):
        views[name] = packed[..., 3 + k * d:3 + (k + 1) * d]
        views[name].copy_(t[name])
    for kw in (dict(), dict(reverse=True)):
        want, got = forward(t, **kw), forward(views, **kw)
        assert all(torch.equal(p, q) for p, q in zip(want, got))
        want, got = backward(t, **kw), backward(views, **kw)
        assert all(torch.equal(want[k], got[k]) for k in want)
    turned = dict(t, **{k: t[k].transpose(0, 1).contiguous().transpose(0, 1) for k in ("x", "g", "i", "z")})
    assert torch.equal(forward(t)[0], forward(turned)[0])
    one = dict(t, g=t["g"][:1, :1].expand(b, l, d))
    assert torch.equal(forward(one)[0], forward(dict(one, g=one["g"].contiguous()))[0])
    assert torch.equal(backward(one)["dg"], backward(dict(one, g=one["g"].contiguous()))["dg"])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("b,d", [(1, 1), (1, 2560), (7, 66), (3, 65), (256, 130)])
def test_step(b, d, dtype):
    for gated in (True, False):
        t = draw(b, 4, d, dtype, seed=8, gated=gated)
        want = rec_ref.rec(*(t[k] for k in FWD))
        state, rows = t["h0"].clone(), []
        for k in range(4):
            rows.append(sscan.rec_step(state, *(None if t[n] is None else t[n] if n == "lam" else t[n][:, k]
                                                for n in FWD[:5])))
        within(torch.stack(rows, 1), want["out"], "out")
        within(state, want["h_last"], "state")
    lengths = torch.tensor([k % 2 for k in range(b)], dtype=torch.int32, device=DEV)
    state = t["h0"].clone()
    out = sscan.rec_step(state, t["x"][:, 0], t["g"][:, 0], lengths=lengths)
    assert torch.equal(state[::2], t["h0"][::2]) and not out[::2].any()
    whole = t["h0"].clone()
    assert torch.equal(sscan.rec_step(whole, t["x"][:, 0], t["g"][:, 0])[1::2], out[1::2])
    assert torch.equal(whole[1::2], state[1::2])


@pytest.mark.parametrize("l", [5, 700])
def test_pieces_and_states_in_place(l):
    """Consecutive pieces, each state handed on in place, are the whole."""
    t = draw(2, l, 130, torch.float32, seed=9)
    want = rec_ref.rec(*(t[k] for k in FWD))
    h, cut = t["h0"].clone(), l // 3
    parts = []
    for piece in (slice(0, cut), slice(cut, l)):
        out, last = sscan.rec_fwd(*(t[k][:, piece] if k != "lam" else t[k] for k in FWD[:5]), h0=h, h_last=h)
        assert last is h
        parts.append(out)
    within(torch.cat(parts, 1), want["out"], "out")
    within(h, want["h_last"], "state")


@pytest.mark.parametrize("d", [2, 65])
@pytest.mark.parametrize("l", [200, 300, 1000, 5000])
def test_state_in_place_of_many_segments(l, d):
    """The exit state written over the entry state, which the row's first segment alone reads."""
    t = draw(3, l, d, torch.float32, seed=21)
    t["lam"].fill_(-12.0)  # decays near 1: every token sees the entry state
    want = forward(t)
    for _ in range(10):
        h = t["h0"].clone()
        out, last = forward(dict(t, h0=h), h_last=h)
        assert last is h and torch.equal(out, want[0]) and torch.equal(last, want[1])


def test_infinite_parameters():
    """lam of -inf: no decay and no input; of +inf: a state of one token."""
    t = draw(2, 300, 4, torch.float32, seed=22)
    t["lam"][:] = torch.tensor([-float("inf"), float("inf"), 1e30, float("nan")])
    out, last = forward(t)
    assert torch.equal(last[:, 0], t["h0"][:, 0])
    one = sscan.rec_fwd(*(t[k] if k == "lam" else t[k][:, -1:] for k in FWD[:5]))
    for c in (1, 2):
        assert torch.equal(out[:, -1:, c], one[0][..., c]) and torch.isfinite(out[..., c]).all()
    assert torch.isnan(out[..., 3]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_kept_blocks_that_are_not_finite(dtype):
    t = draw(1, 40, 130, dtype, seed=23)
    t["x"][0, 3, 5], t["g"][0, 20, 70], t["z"][0, 39, 129] = float("nan"), float("inf"), -float("inf")
    t["i"][0, 7, :64] = 0.0
    _, _, kept = forward(t, keep=True)
    for k, p in zip(("x", "g", "i", "z"), kept):
        q, scale, _ = rec_ref.eight(t[k].cpu())
        assert torch.equal(p.q.cpu(), q), k
        assert torch.equal(torch.isnan(p.scale.cpu()), torch.isnan(scale))
        assert torch.equal(torch.nan_to_num(p.scale.cpu()), torch.nan_to_num(scale)), k


def test_resets_and_far_values():
    """Log decays of -inf start a row anew; gates far out; no channel leaks into another."""
    t = draw(1, 400, 130, torch.float32, seed=10, gated=False)
    t["g"][:, 150] = -float("inf")
    out, _ = check_forward(t)
    fresh = {k: v[:, 150:] if k in ("x", "g", "i", "z") else v for k, v in t.items()}
    fresh["h0"] = None
    fresh["g"] = fresh["g"].clone()
    fresh["g"][:, 0] = -1.0
    assert torch.allclose(forward(fresh)[0], out[:, 150:], rtol=1e-5, atol=1e-6)
    got = check_backward(t)
    assert not got["dg"][:, 150].any()
    t = draw(1, 40, 130, torch.float32, seed=11)
    t["g"][:, ::3], t["g"][:, 1::3] = 60.0, -60.0
    t["lam"][::2], t["lam"][1::4] = 30.0, -30.0
    t["i"][:, ::5], t["z"][:, ::7] = -1e30, -1e30
    check_forward(t)
    got = backward(t)
    assert all(torch.isfinite(v).all() for v in got.values())
    # gates so far shut that the decay rounds to 1: the state stays, slopes are 0
    t["g"].fill_(-1e4)
    out, last = forward(t)
    assert torch.equal(last, t["h0"])
    got = backward(t)
    assert not got["dg"].any() and not got["dx"].any() and not got["dlam"].any()


def test_not_a_number_stays_in_its_channel():
    t = draw(2, 500, 130, torch.float32, seed=12)
    clean = forward(t)
    t["x"][0, 200, 7] = float("nan")
    t["x"][1, 300, 9] = float("inf")
    out, last = forward(t)
    assert torch.isnan(out[0, 200:, 7]).all() and torch.isnan(last[0, 7])
    assert torch.isinf(last[1, 9]) or torch.isnan(last[1, 9])
    keep = torch.ones(2, 130, dtype=torch.bool, device=DEV)
    keep[0, 7] = keep[1, 9] = False
    assert torch.equal(last[keep], clean[1][keep])
    assert torch.equal(out[:, :200], clean[0][:, :200])
    assert torch.equal(out.transpose(1, 2)[keep], clean[0].transpose(1, 2)[keep])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("parts", ["izhl", "", "i", "z"])
@pytest.mark.parametrize("b,l,d", [(1, 1, 1), (2, 300, 130), (3, 77, 384), (1, 200, 65), (2, 33, 64)])
def test_kept_in_8_bits(b, l, d, parts, dtype):
    """What the forward keeps are the inputs in 8 bits, and the gradients are those there."""
    t = draw(b, l, d, dtype, seed=13, parts=parts)
    out, h_last, kept = forward(t, keep=True)
    plain = forward(t)
    assert torch.equal(out, plain[0]) and torch.equal(h_last, plain[1])
    back = dict(t)
    for k, p in zip(("x", "g", "i", "z"), kept):
        assert (p is None) == (t[k] is None)
        if p is not None:
            q, scale, value = rec_ref.eight(t[k].cpu())
            assert torch.equal(p.q.cpu(), q) and torch.equal(p.scale.cpu(), scale), k
            back[k] = value.to(DEV)
    got = sscan.rec_bwd(kept.x, kept.g, t["dout"], kept.i, t["lam"], kept.z, t["h0"], t["dh_last"])
    want = rec_ref.rec_bwd(back["x"], back["g"], t["dout"], back["i"], t["lam"], back["z"], t["h0"], t["dh_last"])
    for k, v in want.items():
        # a value in 8 bits is itself rounded to float32: half a step of it, within every bound
        within(got[k], (v[0], v[1] * 1.25), k)


@pytest.mark.parametrize("checkpoint", [False, True])
def test_autograd(checkpoint):
    t = draw(2, 200, 130, torch.bfloat16, seed=14, lengths=[200, 77])
    names = ("x", "g", "i", "lam", "z", "h0")
    for k in names:
        t[k].requires_grad_(True)
    out, h_last = sscan.gated_recurrence(*(t[k] for k in FWD[:5]), h0=t["h0"], lengths=t["lengths"], checkpoint=checkpoint)
    got = torch.autograd.grad([out, h_last], [t[k] for k in names], [t["dout"], t["dh_last"]], retain_graph=True)
    with torch.no_grad():
        src = t
        if checkpoint:
            kept = forward(t, keep=True)[2]
            src = dict(t, **{k: p for k, p in zip(("x", "g", "i", "z"), kept)})
        want = backward(src)
    for k, v in zip(names, got):
        assert torch.equal(v, want["d" + k]), k
    # only one of the outputs used
    (one,) = torch.autograd.grad(h_last.sum(), [t["x"]], retain_graph=True)
    with torch.no_grad():
        zero = torch.zeros_like(t["dout"])
        assert torch.equal(one, backward(dict(src, dout=zero, dh_last=torch.ones_like(t["dh_last"])))["dx"])
    with pytest.raises(RuntimeError, match="no second derivatives"):
        (g,) = torch.autograd.grad(out.float().sum(), [t["x"]], create_graph=True)
        torch.autograd.grad(g.float().sum(), [t["x"]])


def test_written_in_place_counts():
    t = draw(2, 20, 64, torch.float32, seed=15)
    x = t["x"].requires_grad_(True)
    out, _ = sscan.gated_recurrence(x, t["g"], h0=t["h0"])
    with torch.no_grad():
        sscan.rec_step(t["h0"], x[:, 0], t["g"][:, 0])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(out.sum(), [x])


def test_repeatable_and_on_another_stream():
    t = draw(2, 3000, 130, torch.bfloat16, seed=16)
    want, grads = forward(t), backward(t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again, grads2 = forward(t), backward(t)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(p, q) for p, q in zip(want, again))
    assert all(torch.equal(grads[k], grads2[k]) for k in grads)


def test_in_a_graph():
    """Captured forward, backward and step, replayed with new inputs in the same places and
    other work between; two graphs share one workspace."""
    t = draw(2, 700, 130, torch.bfloat16, seed=17)
    other = draw(2, 700, 130, torch.bfloat16, seed=18)
    n = max(sscan.rec_workspace_bytes(2, 700, 130), sscan.rec_workspace_bytes(2, 700, 130, backward=True), 1)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    state = torch.zeros(2, 130, device=DEV)
    step = lambda: sscan.rec_step(state, t["x"][:, 0], t["g"][:, 0], None, t["lam"])
    forward(t, workspace=ws), backward(t, workspace=ws), step()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        out, last = forward(t, workspace=ws)
        y = step()
    with torch.cuda.graph(g2):
        grads = backward(t, workspace=ws)
    for src in (t, other, t, other):
        new = {k: v.clone() for k, v in src.items() if v is not None and k not in ("lam", "lengths")}
        for k, v in new.items():
            t[k].copy_(v)
        state.copy_(new["h0"])
        want, wgrads = forward(t), backward(t)
        kept = state.clone()
        wy = sscan.rec_step(kept, t["x"][:, 0], t["g"][:, 0], None, t["lam"])
        torch.cuda.synchronize()
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(last, want[1]) and torch.equal(y, wy) and torch.equal(state, kept)
        assert all(torch.equal(grads[k], wgrads[k]) for k in grads)


def test_empty():
    for b, l, d in ((0, 5, 8), (2, 0, 8), (2, 5, 0)):
        t = draw(b, l, d, torch.float32, seed=19)
        out, h_last = forward(t)
        assert out.shape == (b, l, d) and torch.equal(h_last, t["h0"])
        got = backward(t)
        assert got["dx"].shape == (b, l, d) and not got["dlam"].any()
        if l == 0:
            assert torch.equal(got["dh0"], t["dh_last"])
        assert not forward(dict(t, h0=None))[1].any()
        out, _, kept = forward(t, keep=True)
        assert kept.x.q.shape == (b, l, d)
        got = sscan.rec_bwd(kept.x, kept.g, t["dout"], kept.i, t["lam"], kept.z, t["h0"], t["dh_last"])
        assert not got["dlam"].any()


def test_refusals():
    t = draw(2, 6, 8, torch.float32, seed=20)
    x, g = t["x"], t["g"]
    for bad, error in ((dict(g=g[:1]), ValueError), (dict(g=g.bfloat16()), TypeError), (dict(x=x.half(), g=g.half()), TypeError),
                       (dict(x=x[0], g=g[0]), ValueError), (dict(x=x.cpu(), g=g.cpu()), ValueError), (dict(g=3), TypeError),
                       (dict(i=g[..., :4]), ValueError), (dict(z=[1]), TypeError), (dict(lam=t["lam"][:4]), ValueError),
                       (dict(lam=t["lam"].double()), TypeError), (dict(h0=t["h0"][:1]), ValueError),
                       (dict(x=x.transpose(1, 2), g=g.transpose(1, 2)), ValueError),
                       (dict(lengths=torch.zeros(2, device=DEV)), TypeError)):
        args = dict(dict(x=x, g=g), **bad)
        with pytest.raises(error):
            sscan.rec_fwd(**args)
        with pytest.raises(error):
            sscan.rec_bwd(dout=x, **args)
    for kw in (dict(c=float("nan")), dict(c=-1.0), dict(out=x), dict(h_last=t["h0"], out=g)):
        with pytest.raises(sscan.SScanError):
            sscan.rec_fwd(x, g, **kw)
    with pytest.raises(sscan.SScanError):
        sscan.rec_fwd(x, g, h0=t["h0"], out=t["h0"].new_empty(0).set_(x.untyped_storage(), 0, x.shape, x.stride()))
    with pytest.raises(ValueError):
        sscan.rec_step(None, x[:, 0], g[:, 0])
    with pytest.raises(ValueError):
        sscan.rec_step(t["h0"][:1], x[:, 0], g[:, 0])
    _, _, kept = sscan.rec_fwd(x, g, keep=True)
    for args in ((kept.x, g, x), (kept.x, kept.g, 3), (kept.x, None, x), (x, kept.g, x)):
        with pytest.raises(TypeError):
            sscan.rec_bwd(*args)
    with pytest.raises(ValueError):
        sscan.rec_bwd(kept.x, sscan.Packed8(kept.g.q[:1], kept.g.scale[:1]), x)
    with pytest.raises(ValueError):
        sscan.rec_bwd(x, g, None)
    for dout in (x[:1], x.bfloat16()):
        with pytest.raises((ValueError, TypeError)):
            sscan.rec_bwd(x, g, dout)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kept", [False, True])
def test_decays_that_round_to_one(kept, dtype):
    """w^2 = 1 - a^2 on both sides of 2^-126, the smallest number that the hardware's square root
    and its reciprocal take: w may count as 0 there."""
    pairs = [(-30.0, -61.0), (-5.0, -86.0), (-60.0, -35.0), (-85.0, -6.0), (-30.0, -60.0), (-30.0, -59.0), (-86.0, -1.0),
             (-87.0, 0.0), (-88.0, 2.0), (-20.0, -70.0),
             (30.0, -88.0)]
    d = 64 * len(pairs)  # a block of 64 channels for each: the 8 bits hold its one value of g exactly
    t = draw(2, 150, d, dtype, seed=24)
    for k, (lam, g) in enumerate(pairs):
        t["lam"][64 * k:64 * k + 64] = lam
        t["g"][..., 64 * k:64 * k + 64] = g
    src, args = dict(t), [t[k] for k in ("x", "g", "i", "z")]
    if kept:
        args = forward(t, keep=True)[2]
        src.update((k, rec_ref.eight(t[k].cpu())[2].to(DEV)) for k in ("x", "g", "i", "z"))
    x, g, i, z = args
    got = sscan.rec_bwd(x, g, t["dout"], i, t["lam"], z, t["h0"], t["dh_last"])
    want = rec_ref.rec_bwd(src["x"], src["g"], t["dout"], src["i"], t["lam"], src["z"], t["h0"], t["dh_last"])
    out, h_last = forward(t)
    states = rec_ref.rec(*(t[k] for k in FWD))
    # a w below 2^-56 may count as 0: that much of |D s x|, |D s| or |s x| for each token (the slope
    # of w has 1 / w, but times c softplus(lam) r = w^2 / 2).  |D| is at most the sum over the row of
    # |dout silu(z)| and |dh_last|; states that lack an input reach dlog a, dz and out with such factors.
    x, dout, z = (src[k].double().abs() for k in ("x", "dout", "z"))
    D = (dout * (1 + z)).sum(1, keepdim=True) + t["dh_last"].double().abs()[:, None]
    add = 2.0 ** -56 * 150 * (1 + D) * (1 + x.amax(1, keepdim=True)) * (1 + z.amax())
    for name in ("dx", "dg", "di", "dz", "dh0"):
        v, bound = want[name]
        within(got[name], (v, 1.25 * bound + (add if v.dim() == 3 else add[:, 0])), name)
    v, bound = want["dlam"]
    within(got["dlam"], (v, 1.25 * bound + 150 * add.sum((0, 1))), "dlam")
    for name, v in (("out", out), ("h_last", h_last)):
        value, bound = states[name]
        within(v, (value, bound + (add if value.dim() == 3 else add[:, 0])), name)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [128, 130, 65])
def test_gates_shut_by_the_lowest_value(d, dtype):
    """Gates of some tokens shut by their type's lowest value, in the gradients from 8 bits too:
    the other elements of its blocks are then below half a step, 0."""
    t = draw(2, 100, d, dtype, seed=25)
    low = torch.finfo(dtype).min
    t["g"][0, 10, 3], t["i"][0, 20, 5], t["g"][1, 30, 64], t["i"][1, 99, :7] = low, low, low, low
    if dtype == torch.bfloat16:  # float32's lowest value is read back from 8 bits as an infinity
        t["z"][1, 40, 0] = low
    _, _, kept = forward(t, keep=True)
    back = dict(t, **{k: rec_ref.eight(t[k].cpu())[2].to(DEV) for k in ("x", "g", "i", "z")})
    assert not back["g"][0, 10, 4:64].any() and back["g"][0, 10, 3] < -3e38
    got = sscan.rec_bwd(kept.x, kept.g, t["dout"], kept.i, t["lam"], kept.z, t["h0"], t["dh_last"])
    want = rec_ref.rec_bwd(back["x"], back["g"], t["dout"], back["i"], t["lam"], back["z"], t["h0"], t["dh_last"])
    for k, v in want.items():
        within(got[k], (v[0], v[1] * 1.25), k)


def test_nothing_is_kept_without_a_backward_pass(monkeypatch):
    """checkpoint=True where no gradient can be asked for: the plain forward, with the same bits."""
    t = draw(2, 200, 130, torch.bfloat16, seed=26)
    args = [t[k] for k in FWD[:5]]
    made, new = [], sscan._kept_new
    monkeypatch.setattr(sscan, "_kept_new", lambda *a: made.append(a) or new(*a))
    want = forward(t)
    for got in (sscan.gated_recurrence(*args, h0=t["h0"], checkpoint=True),):
        assert not made and all(torch.equal(p, q) for p, q in zip(got, want))
    t["lam"].requires_grad_(True)
    with torch.no_grad():
        got = sscan.gated_recurrence(*args, h0=t["h0"], checkpoint=True)
    assert not made and all(torch.equal(p, q) for p, q in zip(got, want)) and not got[0].requires_grad
    with torch.inference_mode():
        sscan.gated_recurrence(*args, h0=t["h0"], checkpoint=True)
    assert not made
    got = sscan.gated_recurrence(*args, h0=t["h0"], checkpoint=True)
    assert len(made) == 1 and all(torch.equal(p, q) for p, q in zip(got, want)) and got[0].requires_grad


@pytest.mark.parametrize("l", [0, 6])
def test_a_missing_gate_is_refused(l):
    """x and g are required, with i given or not, with tokens or without."""
    t = draw(2, l, 8, torch.float32, seed=27)
    for i in (None, t["i"]):
        for x, g in ((t["x"], None), (None, t["g"]), (None, None)):
            with pytest.raises(TypeError, match="must be a torch.Tensor"):
                sscan.rec_fwd(x, g, i)
            with pytest.raises(TypeError, match="must be a torch.Tensor"):
                sscan.rec_bwd(x, g, t["dout"], i)
            with pytest.raises(TypeError, match="must be a torch.Tensor"):
                sscan.gated_recurrence(x, g, i)
            if l:
                with pytest.raises(TypeError, match="must be a torch.Tensor"):
                    sscan.rec_step(t["h0"].clone(), None if x is None else x[:, 0], None if g is None else g[:, 0],
                                   None if i is None else i[:, 0])


@pytest.mark.parametrize("kept", [False, True])
def test_gradients_at_infinite_parameters(kept):
    """lam of +inf (and beyond where c softplus(lam) fits float32): every state is its own token's
    input, so dg, dlam and dh0 are 0 and the others are those of h = sigmoid(i) x.  lam of -inf: no
    decay and no input."""
    t = draw(2, 150, 256, torch.float32, seed=28)
    t["lam"][:128], t["lam"][64:128], t["lam"][128:] = float("inf"), 3e38, -float("inf")
    args = forward(t, keep=True)[2] if kept else [t[k] for k in ("x", "g", "i", "z")]
    src = {k: rec_ref.eight(t[k].cpu())[2].to(DEV) if kept else t[k].double() for k in ("x", "g", "i", "z")}
    x, g, i, z = args
    got = sscan.rec_bwd(x, g, t["dout"], i, t["lam"], z, t["h0"], t["dh_last"])
    # the same at a rate of 8e4, whose decays are 0 too in float64
    near = dict(t, lam=t["lam"].clamp(-1e5, 1e4))
    want = rec_ref.rec_bwd(src["x"], src["g"], t["dout"], src["i"], near["lam"], src["z"], t["h0"], t["dh_last"])
    for k, (v, bound) in want.items():
        within(got[k], (v, 1.25 * bound), k)
    assert not got["dg"].any() and not got["dlam"].any() and not got["dh0"][:, :128].any()
    # a gate so far shut that it is 0 keeps the state
    t["g"].fill_(-1e4)
    assert torch.equal(forward(t)[1], t["h0"])
