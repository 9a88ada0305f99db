"""Plain float64 forms of the gated delta rule and of the norms around a mixer, for the
tests: token by token from the definitions, on the CPU, with gradients by torch's
differentiation of these forms.

Tolerances, fixed from the number formats:

* float32 outputs: every product has float32 accuracy (2^-24 relative to its largest
  term) and sums of a few hundred such terms pass from one token's output to the next
  through a contracting recurrence, so an error of some tens of 2^-24 of the output's
  size is expected; 1e-5 of (|ref| + rms) leaves a factor of about ten.
* bfloat16 outputs: one rounding (2^-9 of the value), which may go the other way than
  the reference's (2^-8), and 1e-4 rms for what precedes it.
"""
import torch


def close(got, ref, name="", terms=0.0):
    got, ref = got.detach().cpu(), ref.detach()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    g, r = got.double(), ref.double()
    assert torch.isfinite(r).all(), name
    assert torch.isfinite(g).all(), (name, "not finite")
    if r.numel() == 0:
        return 0.0
    rms = float(r.square().mean().sqrt())
    if got.dtype == torch.bfloat16:
        bound = 2.0 ** -8 * r.abs() + 1e-4 * rms
    else:
        bound = 1e-5 * (r.abs() + rms)
    bound = bound + 1e-5 * float(terms) + 1e-30
    worst = float(((g - r).abs() / bound).max())
    assert worst <= 1.0, f"{name}: {worst:.3g} times the bound (rms {rms:.3g})"
    return worst


def delta(q, k, v, g, beta, h0=None, lengths=None, scale=None, qk_norm=False):
    """q, k [b, l, hk, dk], v [b, l, hv, dv], g, beta [b, l, hv]: (out, last state)."""
    q, k, v, g, beta = (x.double() for x in (q, k, v, g, beta))
    b, L, hk, dk = q.shape
    hv, dv = v.shape[2:]
    scale = dk ** -0.5 if scale is None else scale
    S = torch.zeros(b, hv, dk, dv, dtype=torch.float64) if h0 is None else h0.double()
    n = [L] * b if lengths is None else [min(max(int(x), 0), L) for x in lengths]
    outs, lasts = [], []
    for i in range(b):
        s, rows = S[i], []
        for t in range(n[i]):
            qt, kt = q[i, t], k[i, t]
            if qk_norm:
                qt = qt / (qt.square().sum(-1, keepdim=True) + 1e-6).sqrt()
                kt = kt / (kt.square().sum(-1, keepdim=True) + 1e-6).sqrt()
            qt, kt = (x.repeat_interleave(hv // hk, 0) for x in (qt, kt))
            s = s * g[i, t].exp()[:, None, None]
            u = beta[i, t][:, None] * (v[i, t] - (kt[:, :, None] * s).sum(1))
            s = s + kt[:, :, None] * u[:, None, :]
            rows.append(scale * (qt[:, :, None] * s).sum(1))
        rows += [torch.zeros(hv, dv, dtype=torch.float64)] * (L - n[i])
        outs.append(torch.stack(rows) if rows else torch.zeros(0, hv, dv, dtype=torch.float64))
        lasts.append(s)
    return torch.stack(outs), torch.stack(lasts)


def rms_unit(x, eps):
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt()


def gated_norm(x, z, weight, eps, gate_first):
    x, z = x.double(), z.double()
    w = 1.0 if weight is None else weight.double()
    gate = z / (1 + torch.exp(-z))
    return rms_unit(x * gate, eps) * w if gate_first else rms_unit(x, eps) * w * gate


def add_norm(x, residual, weight, scale, post_weight, eps, stored):
    """(out, total), the total rounded to `stored` (straight through for gradients)."""
    a = x.double()
    if post_weight is not None:
        a = rms_unit(a, eps) * post_weight.double()
    if scale is not None:
        a = a * scale.double()
    total = a if residual is None else residual.double() + a
    total = total + (total.detach().float().to(stored).double() - total.detach())
    y = rms_unit(total, eps)
    return y if weight is None else y * weight.double(), total


def norm_terms(x, dn, eps=1e-6):
    """Size of the terms that the gradient of rms_unit at x subtracts, given dn."""
    x, dn = x.double(), dn.double()
    return float((dn / (x.square().mean(-1, keepdim=True) + eps).sqrt()).square().mean().sqrt()) if x.numel() else 0.0
