"""The gated delta rule's forward and decode step against the float64 token recurrence."""
import pytest
import torch

import delta_ref
from delta_ref import close
from selective_state_space_sscan_amd import sscan

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def inputs(b, L, hk, hv, dk, dv, dtype, seed=0, unit=True, g_scale=0.3):
    gen = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(b, L, h, d, generator=gen) for h, d in ((hk, dk), (hk, dk), (hv, dv)))
    if unit:
        q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
    g = -g_scale * torch.rand(b, L, hv, generator=gen)
    beta = torch.sigmoid(torch.randn(b, L, hv, generator=gen))
    return q.to(dtype), k.to(dtype), v.to(dtype), g, beta


def state(b, hv, dk, dv, seed=7):
    return 0.5 * torch.randn(b, hv, dk, dv, generator=torch.Generator().manual_seed(seed))


def on(*xs):
    return [None if x is None else x.to(DEV) for x in xs]


def run(ins, h0=None, lengths=None, **kw):
    print("delta_fwd", [tuple(x.shape) for x in ins], ins[0].dtype, kw, flush=True)
    out, last = sscan.delta_fwd(*on(*ins), *on(h0, lengths), **kw)
    torch.cuda.synchronize()
    return out, last


SHAPES = [  # b, L, hk, hv, dk, dv
    (1, 1, 1, 1, 1, 1), (2, 3, 1, 2, 16, 8), (1, 8, 2, 2, 128, 128), (2, 9, 1, 1, 64, 64), (1, 63, 1, 3, 33, 50),
    (2, 64, 2, 4, 128, 128), (1, 65, 1, 1, 128, 256), (1, 200, 3, 3, 48, 72), (1, 257, 1, 2, 128, 100),
    (3, 130, 1, 1, 7, 17), (1, 577, 2, 2, 96, 128), (1, 1500, 1, 1, 64, 16),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, dtype):
    b, L, hk, hv, dk, dv = shape
    ins = inputs(*shape, dtype, seed=L)
    h0 = state(b, hv, dk, dv)
    out, last = run(ins, h0)
    ref, ref_last = delta_ref.delta(*ins, h0)
    close(out, ref.to(dtype) if dtype is torch.float32 else ref, "out")
    close(last, ref_last, "h_last")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L", [5, 100])
def test_forward_qk_norm_scale_and_no_entry_state(L, dtype):
    ins = inputs(2, L, 2, 4, 64, 40, dtype, seed=3, unit=False)
    out, last = run(ins, qk_norm=True, scale=0.7)
    ref, ref_last = delta_ref.delta(*ins, qk_norm=True, scale=0.7)
    close(out, ref, "out")
    close(last, ref_last, "h_last")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L,lengths", [(6, [0, 1, 6, 4]), (150, [0, 64, 150, 65]), (150, [-3, 200, 128, 1])])
def test_lengths_leave_the_rest_unread(L, lengths, dtype):
    ins = inputs(4, L, 1, 2, 64, 64, dtype, seed=5)
    h0 = state(4, 2, 64, 64)
    n = torch.tensor(lengths, dtype=torch.int32)
    ref, ref_last = delta_ref.delta(*ins, h0, n)
    for i, m in enumerate(lengths):  # what is masked may be anything
        for x in ins:
            x[i, max(m, 0):] = float("nan")
    out, last = run(ins, h0, n)
    close(out, ref, "out")
    close(last, ref_last, "h_last")
    for i, m in enumerate(lengths):
        assert not out[i, max(m, 0):].any()
        if m <= 0:
            assert torch.equal(last[i].cpu(), h0[i])


@pytest.mark.parametrize("L", [7, 200])
def test_resets_and_strong_decays(L):
    ins = inputs(1, L, 1, 2, 64, 64, torch.float32, seed=11)
    g = ins[3]
    g[0, L // 2, 0] = float("-inf")
    g[0, : L // 3, 1] = -200.0
    g[0, L // 3, 1] = torch.finfo(torch.float32).min
    out, last = run(ins, state(1, 2, 64, 64))
    ref, ref_last = delta_ref.delta(*ins, state(1, 2, 64, 64))
    close(out, ref, "out")
    close(last, ref_last, "h_last")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", [(64, 48), (128, 130)])
def test_long_rows_walked_in_segments(dk, dv, dtype):
    """Few rows, many chunks: entry states come from the segments' transitions; rows end
    inside the first, a middle and the last segment, on a segment's edge, and not at all."""
    ins = inputs(5, 1300, 1, 1, dk, dv, dtype, seed=21, g_scale=0.02)
    h0 = state(5, 1, dk, dv)
    n = torch.tensor([1300, 7, 640, 1290, 0], dtype=torch.int32)
    out, last = run(ins, h0, n)
    ref, ref_last = delta_ref.delta(*ins, h0, n)
    close(out, ref, "out")
    close(last, ref_last, "h_last")


def test_correlated_keys():
    """Keys that nearly repeat make the chunk's triangular system as ill behaved as it gets."""
    gen = torch.Generator().manual_seed(2)
    ins = list(inputs(1, 256, 1, 1, 64, 32, torch.float32, seed=2, g_scale=0.01))
    base = torch.randn(1, 1, 1, 64, generator=gen)
    k = base + 0.05 * torch.randn(1, 256, 1, 64, generator=gen)
    ins[1] = k / k.norm(dim=-1, keepdim=True)
    ins[4] = torch.ones(1, 256, 1)
    out, last = run(ins)
    ref, ref_last = delta_ref.delta(*ins)
    close(out, ref, "out")
    close(last, ref_last, "h_last")


def test_zero_beta_and_zero_keys():
    ins = list(inputs(1, 80, 1, 1, 64, 64, torch.float32, seed=4, unit=False))
    ins[4][0, 10:20] = 0.0
    ins[1][0, 30:40] = 0.0
    ins[0][0, 35:45] = 0.0
    out, last = run(ins, qk_norm=True)
    ref, ref_last = delta_ref.delta(*ins, qk_norm=True)
    close(out, ref, "out")
    close(last, ref_last, "h_last")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L", [4, 90])
def test_strided_views(L, dtype):
    """q, k, v out of one packed projection, heads before tokens, gates interleaved."""
    b, hk, hv, dk, dv = 2, 2, 4, 64, 48
    ins = inputs(b, L, hk, hv, dk, dv, dtype, seed=8)
    ref, ref_last = delta_ref.delta(*ins)
    q, k, v, g, beta = on(*ins)
    packed = torch.full((b, L, 2 * hk * dk + hv * dv + 3), float("nan"), device=DEV, dtype=dtype)
    views, at = [], 3  # an offset of three elements: no 16-byte alignment
    for x in (q, k, v):
        n = x.shape[2] * x.shape[3]
        view = packed[:, :, at:at + n].unflatten(-1, x.shape[2:])
        view.copy_(x)
        views.append(view)
        at += n
    gates = torch.stack([g, beta], -1)
    out, last = sscan.delta_fwd(*views, gates[..., 0], gates[..., 1])
    close(out, ref, "packed out")
    close(last, ref_last, "packed h_last")
    head_major = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v, g, beta)]
    out2, last2 = sscan.delta_fwd(*head_major)
    close(out2, ref, "head-major out")
    close(last2, ref_last, "head-major h_last")


def test_shared_inputs_by_broadcast():
    """One key and one gate for all batch rows (stride 0)."""
    ins = inputs(1, 70, 1, 2, 64, 64, torch.float32, seed=9)
    wide = [x.expand(3, *x.shape[1:]) for x in on(*ins)]
    out, last = sscan.delta_fwd(*wide)
    ref, ref_last = delta_ref.delta(*ins)
    close(out, ref.expand(3, -1, -1, -1), "out")
    close(last, ref_last.expand(3, -1, -1, -1), "h_last")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("L", [5, 70, 1300])
def test_rows_that_overlap(L, dtype):
    """One key and value for all tokens (token stride 0) and windows sliding by less than a
    row: the tokens past the end of the last chunk are not taken for live ones."""
    q, k, v, g, beta = inputs(1, L, 1, 1, 64, 64, dtype, seed=9)
    q_line = torch.randn(L * 16 + 64, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV) / 8
    q_win = q_line.as_strided((1, L, 1, 64), (0, 16, 64, 1))
    k0, v0 = k[:, :1].to(DEV), v[:, :1].to(DEV)
    out, last = sscan.delta_fwd(q_win, k0.expand(1, L, 1, 64), v0.expand(1, L, 1, 64), g.to(DEV), beta.to(DEV))
    full = [q_win.cpu().clone(), k[:, :1].expand(1, L, 1, 64), v[:, :1].expand(1, L, 1, 64), g, beta]
    ref, ref_last = delta_ref.delta(*full)
    close(out, ref, "out")
    close(last, ref_last, "h_last")
    dout = torch.randn(1, L, 1, 64, generator=torch.Generator().manual_seed(2)).to(dtype).to(DEV)
    r = sscan.delta_bwd(q_win, k0.expand(1, L, 1, 64), v0.expand(1, L, 1, 64), g.to(DEV), beta.to(DEV), dout)
    r2 = sscan.delta_bwd(*[x.contiguous().to(DEV) for x in full], dout)
    for name in r:
        assert torch.equal(r[name], r2[name]), name


def test_one_token_of_a_huge_stride():
    x = [t.to(DEV) for t in inputs(1, 1, 1, 1, 64, 64, torch.float32, seed=3)]
    odd = [t.as_strided(t.shape, (t.stride(0), 1 << 40, *t.stride()[2:])) for t in x]
    out, last = sscan.delta_fwd(*odd)
    want, want_last = sscan.delta_fwd(*x)
    assert torch.equal(out, want) and torch.equal(last, want_last)
    dout = torch.ones(1, 1, 1, 64, device=DEV)
    a, b = sscan.delta_bwd(*odd, dout), sscan.delta_bwd(*x, dout)
    for name in a:
        assert torch.equal(a[name], b[name]), name


def test_empty_calls():
    ins = inputs(2, 0, 1, 1, 64, 64, torch.float32)
    h0 = state(2, 1, 64, 64)
    out, last = run(ins, h0)
    assert out.shape == (2, 0, 1, 64) and torch.equal(last.cpu(), h0)
    _, last = run(ins)
    assert not last.any()
    out, last = run(inputs(0, 5, 1, 1, 64, 64, torch.float32))
    assert out.shape == (0, 5, 1, 64) and last.shape == (0, 1, 64, 64)


@pytest.mark.parametrize("L", [6, 100])
def test_pieces_equal_the_whole_and_state_in_place(L):
    ins = on(*inputs(2, L, 1, 2, 64, 64, torch.float32, seed=10))
    whole, last = sscan.delta_fwd(*ins, h0=state(2, 2, 64, 64).to(DEV))
    s = state(2, 2, 64, 64).to(DEV)
    cut = L // 3
    parts = []
    for sl in (slice(0, cut), slice(cut, L)):
        o, s2 = sscan.delta_fwd(*[x[:, sl] for x in ins], h0=s, h_last=s)
        assert s2 is s
        parts.append(o)
    close(torch.cat(parts, 1), whole.cpu(), "out")
    close(s, last.cpu(), "state")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(1, 1, 1, 128, 128), (3, 2, 4, 64, 96), (2, 1, 3, 33, 50), (5, 1, 1, 1, 1),
                                   (2, 2, 2, 128, 256)])
def test_step(shape, dtype):
    b, hk, hv, dk, dv = shape
    s = state(b, hv, dk, dv)
    got = s.to(DEV)
    for t in range(3):
        ins = inputs(b, 1, hk, hv, dk, dv, dtype, seed=20 + t, unit=False)
        out = sscan.delta_step(got, *[x[:, 0] for x in on(*ins)], qk_norm=True)
        ref, s = delta_ref.delta(*ins, s, qk_norm=True)
        close(out, ref[:, 0], f"out {t}")
        close(got, s, f"state {t}")


def test_step_skips_rows_of_length_zero():
    s = state(3, 1, 64, 64)
    ins = inputs(3, 1, 1, 1, 64, 64, torch.float32)
    ref, ref_s = delta_ref.delta(*ins, s, torch.tensor([1, 0, 1]))
    got = s.to(DEV)
    for x in ins:
        x[1] = float("nan")
    out = sscan.delta_step(got, *[x[:, 0] for x in on(*ins)], lengths=torch.tensor([1, 0, 1], dtype=torch.int32).to(DEV))
    close(out, ref[:, 0], "out")
    close(got, ref_s, "state")
    assert torch.equal(got[1].cpu(), s[1]) and not out[1].any()


def test_refusals():
    q, k, v, g, beta = on(*inputs(1, 10, 1, 2, 64, 64, torch.float32))
    with pytest.raises(ValueError):
        sscan.delta_fwd(q.cpu(), k, v, g, beta)
    with pytest.raises(ValueError):
        sscan.delta_fwd(q, k[:, :5], v, g, beta)
    with pytest.raises(TypeError):
        sscan.delta_fwd(q, k.bfloat16(), v, g, beta)
    with pytest.raises(TypeError):
        sscan.delta_fwd(q, k, v, g.bfloat16(), beta)
    with pytest.raises(TypeError):
        sscan.delta_fwd(q, k, v, g, beta, lengths=torch.ones(1, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):  # three value heads over two key heads
        sscan.delta_fwd(torch.cat([q, q], 2), torch.cat([k, k], 2), torch.cat([v, v[:, :, :1]], 2),
                        torch.cat([g, g[..., :1]], 2), torch.cat([beta, beta[..., :1]], 2))
    with pytest.raises(ValueError):  # last dimension not contiguous
        sscan.delta_fwd(q.transpose(2, 3).contiguous().transpose(2, 3), k, torch.stack([v, v], -1)[..., 0], g, beta)
    big = torch.zeros(1, 10, 1, 129, device=DEV)
    with pytest.raises(sscan.SScanError):
        sscan.delta_fwd(big, big, v, g, beta)
    with pytest.raises(sscan.SScanError):  # output over an input
        sscan.delta_fwd(q, k, v, g, beta, out=v)
    with pytest.raises(sscan.SScanError):  # workspace too small
        x = on(*inputs(1, 100, 1, 1, 64, 64, torch.float32))
        sscan.delta_fwd(*x, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))


def test_on_another_stream_and_graph_replays():
    ins = on(*inputs(1, 100, 1, 2, 64, 64, torch.bfloat16, seed=12))
    ref, ref_last = sscan.delta_fwd(*ins)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out, last = sscan.delta_fwd(*ins)
    side.synchronize()
    assert torch.equal(out, ref) and torch.equal(last, ref_last)
    ws = torch.empty(sscan.delta_workspace_bytes(1, 100, 1, 2, 64, 64), dtype=torch.uint8, device=DEV)
    o, h = torch.empty_like(ref), torch.empty_like(ref_last)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sscan.delta_fwd(*ins, out=o, h_last=h, workspace=ws)
    for seed in (13, 14, 15):
        for x, y in zip(ins, inputs(1, 100, 1, 2, 64, 64, torch.bfloat16, seed=seed)):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        want, want_last = sscan.delta_fwd(*ins)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(h, want_last)
