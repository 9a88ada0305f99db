"""A gated-recurrence block: residual sum and layer norm, projections, the recurrence with its
output gate, and the projection back, for training and for decoding.

    python examples/recurrent_block.py        # a few training steps, then prefill and decode

The block's operators are this library's (``add_layer_norm``, ``gated_recurrence``;
decoding: ``layer_norm``, ``rec_step``); the projections are torch's matrix products.  With
``checkpoint`` the recurrence keeps its inputs for the backward pass in 8 bits.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from selective_state_space_sscan_amd import sscan  # noqa: E402


class GatedRecurrenceBlock(torch.nn.Module):
    """Takes the stream as (branch, residual): what the last block computed and the sum
    before it.  Returns the same for the next block."""

    def __init__(self, dim: int, width: int, device="cuda", dtype=torch.bfloat16, checkpoint: bool = False):
        super().__init__()
        self.checkpoint = checkpoint
        self.w_in = torch.nn.Parameter(torch.randn(dim, 4 * width, device=device, dtype=dtype) / math.sqrt(dim))
        self.w_out = torch.nn.Parameter(torch.randn(width, dim, device=device, dtype=dtype) / math.sqrt(width))
        self.norm = torch.nn.Parameter(torch.ones(dim, device=device))
        self.bias = torch.nn.Parameter(torch.zeros(dim, device=device))
        # exp(-8 softplus(lam)) from 0.9 to 0.999: the decay of a channel whose gate is open
        self.lam = torch.nn.Parameter(torch.log(torch.expm1(-torch.linspace(0.9, 0.999, width, device=device).log() / 8)))

    def forward(self, branch, residual, state=None, lengths=None):
        y, residual = sscan.add_layer_norm(branch, residual, self.norm, self.bias, residual_dtype=torch.float32)
        x, g, i, z = (y @ self.w_in).chunk(4, -1)
        o, state = sscan.gated_recurrence(x, g, i, self.lam, z, h0=state, lengths=lengths, checkpoint=self.checkpoint)
        return o @ self.w_out, residual, state

    @torch.no_grad()
    def step(self, branch, residual, state):
        """One token [batch, dim]; state is updated in place."""
        y, residual = sscan.layer_norm(branch, self.norm, self.bias, residual, residual_dtype=torch.float32)
        x, g, i, z = (y @ self.w_in).chunk(4, -1)
        return sscan.rec_step(state, x, g, i, self.lam, z) @ self.w_out, residual


def main():
    torch.manual_seed(0)
    b, l, dim = 2, 300, 256
    blocks = [GatedRecurrenceBlock(dim, 320, checkpoint=k == 1) for k in range(2)]
    params = [p for m in blocks for p in m.parameters()]
    opt = torch.optim.Adam(params, lr=1e-3)
    x = torch.randn(b, l, dim, device="cuda", dtype=torch.bfloat16)
    target = torch.roll(x, 1, dims=1).float()

    def run(x, states=None):
        branch, residual, out = x, None, []
        for k, m in enumerate(blocks):
            branch, residual, s = m(branch, residual, None if states is None else states[k])
            out.append(s)
        return residual + branch, out

    losses = []
    for _ in range(20):
        y, _ = run(x)
        loss = (y.float() - target).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")

    with torch.no_grad():
        whole, _ = run(x)
        prompt, states = run(x[:, :200].contiguous())
        rows = [prompt]
        for t in range(200, l):
            branch, residual = x[:, t].contiguous(), None
            for m, s in zip(blocks, states):
                branch, residual = m.step(branch, residual, s)
            rows.append((residual + branch)[:, None])
        again = torch.cat(rows, 1)
    off = float((again - whole).norm() / whole.norm())
    print(f"prefill and decode against one pass: {off:.2e}")
    return losses, off


if __name__ == "__main__":
    main()
