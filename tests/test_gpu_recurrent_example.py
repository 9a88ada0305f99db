"""The gated-recurrence block: it runs, and its gradients are those of the same block written
in torch operations in float64, token by token."""
import importlib.util
import math
import os

import pytest
import torch

import rec_ref

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "recurrent_block.py")


def example():
    spec = importlib.util.spec_from_file_location("recurrent_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs():
    losses, off = example().main()
    assert len(losses) == 20 and all(math.isfinite(v) for v in losses)
    # two ways to the same outputs through four bfloat16 roundings a block, two blocks: eight of
    # at most 2^-8 each
    assert off < 8 * 2.0 ** -8


def plain(p, branch, residual, kept):
    """The block in float64; with `kept` the recurrence's inputs are replaced by what 8 bits
    hold of them, and differentiated as if they were themselves."""
    total = branch if residual is None else residual + branch
    y = torch.nn.functional.layer_norm(total, total.shape[-1:], p["norm"], p["bias"], 1e-5)
    parts = (y @ p["w_in"]).chunk(4, -1)
    exact = rows(parts, p["lam"])
    if kept:
        parts = [v + (rec_ref.eight(v.detach().float())[2] - v.detach()) for v in parts]
    o = rows(parts, p["lam"])
    # the outputs are those of the inputs themselves, the gradients those at the kept values
    return (o + (exact - o).detach()) @ p["w_out"], total


def rows(parts, lam):
    x, g, i, z = parts
    a = torch.exp(-8 * torch.nn.functional.softplus(lam) * torch.sigmoid(g))
    u = torch.sqrt(1 - a * a) * torch.sigmoid(i) * x
    h, out = torch.zeros_like(x[:, 0]), []
    for t in range(x.shape[1]):
        h = a[:, t] * h + u[:, t]
        out.append(h)
    return torch.stack(out, 1) * z * torch.sigmoid(z)


@pytest.mark.parametrize("kept", [False, True])
def test_gradients_of_two_blocks(kept):
    m = example()
    torch.manual_seed(1)
    blocks = [m.GatedRecurrenceBlock(48, 130, dtype=torch.float32, checkpoint=kept) for _ in range(2)]
    x = torch.randn(2, 150, 48, device="cuda", requires_grad=True)
    weight = torch.randn(2, 150, 48, device="cuda")
    branch, residual = x, None
    for k in blocks:
        branch, residual, _ = k(branch, residual)
    params = [p for k in blocks for p in k.parameters()]
    got = torch.autograd.grad(((residual + branch) * weight).sum(), [x] + params)
    x64 = x.detach().double().requires_grad_(True)
    p64 = [{n: p.detach().double().requires_grad_(True) for n, p in k.named_parameters()} for k in blocks]
    branch, residual = x64, None
    for p in p64:
        branch, residual = plain(p, branch, residual, kept)
    leaves = [x64] + [p[n] for k, p in zip(blocks, p64) for n, _ in k.named_parameters()]
    want = torch.autograd.grad(((residual + branch) * weight.double()).sum(), leaves)
    # float32 products over up to 300 terms in and out of each block, 300 * 2^-24 = 2e-5 of a
    # gradient's size at worst; in 8 bits a value within 1e-5 of the middle between two steps may
    # fall on the other side (its share of all is as small, a step 1/127 of a block's largest)
    for v, w in zip(got, want):
        assert float((v.double() - w).norm() / w.norm()) < (2e-4 if kept else 4e-5)
