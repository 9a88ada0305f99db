"""Plain float64 forms of the gated recurrence, of activations in 8 bits and of the layer
norm, token by token from the definitions, each value with a bound on how far a float32
evaluation may be off.

The bounds are running error analyses in units of U = 2^-24 (half a step of float32,
relative): every product or sum is off by U of its size, the hardware's exp2, reciprocal and
square root by 2 U, the library's exp and log1p by 4 U.  So

* sigmoid(v): (1.25 |v| + 5) U of its value (its exponent is rounded twice);
* rate = c softplus(lam): 8 U; m = rate sigmoid(g): (14 + 1.25 |g|) U;
* 1 - a = 1 - e^-m: an error of m passes on at most in full, the evaluation adds 10 U at
  most (below 1/4 a series of seven terms, above it 2 e^-m (1 + m) <= 2 of a value >= 0.22):
  (24 + 1.25 |g|) U of 1 - a; a: that and U; w = sqrt((1 - a) (1 + a)): (16 + 0.63 |g|) U;
* a = exp(g): (2 |g| + 4) U (the exponent g log2 e rounded twice, exp2);
* the state passes its error on by a, and each token adds the errors of a and of its input
  and its own roundings.  A scan that joins parts of a row rounds products of decays, one
  rounding a token, and sums of parts: 2 U a more for each token and 4 U of the state, taken
  of the state that the inputs' magnitudes have (which no order of the sum exceeds).

A bfloat16 output adds half a step, 2^-8 of its value.
"""
import torch

U = 2.0 ** -24
TINY = 2.0 ** -100
BLOCK = 64


def half_step(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else U


def within(got, want, name=""):
    """got (a tensor of the library) against want = (value, bound) in float64."""
    value, bound = want
    got = got.detach()
    assert tuple(got.shape) == tuple(value.shape), (name, got.shape, value.shape)
    if not got.numel():
        return 0.0
    g = got.double().to(value.device)
    assert torch.isfinite(value).all() and torch.isfinite(g).all(), (name, "not finite")
    bound = bound + half_step(got.dtype) * (value.abs() + bound) + 1e-30
    worst = float(((g - value).abs() / bound).max())
    assert worst <= 1.0, f"{name}: {worst:.3g} times the bound"
    return worst


def _sig(v):
    """sigmoid and its error relative to it."""
    return torch.sigmoid(v), (1.25 * v.abs() + 5) * U


class _Tokens:
    """Decays, inputs and their errors, [b, l, d]."""

    def __init__(self, x, g, i, lam, z, c):
        self.x, self.z = x.double(), None if z is None else z.double()
        x, g = self.x, g.double()
        self.s, self.ds = (torch.ones_like(x), torch.zeros_like(x)) if i is None else _sig(i.double())
        self.g, self.gated = g, lam is not None
        if self.gated:
            lam = lam.double()
            self.rate = c * (lam.clamp(min=0) + torch.log1p(torch.exp(-lam.abs())))
            self.slope = c * torch.sigmoid(lam)
            self.r, self.dr = _sig(g)
            m = self.rate * self.r
            loss = -torch.expm1(-m)
            rel = (24 + 1.25 * g.abs()) * U
            self.a = torch.exp(-m)
            self.da = loss * rel + U * self.a
            self.w = torch.sqrt(loss * (2 - loss))
            self.dw = (16 + 0.63 * g.abs()) * U
        else:
            self.a = torch.exp(g)
            self.da = torch.where(torch.isinf(g), torch.zeros_like(g), (2 * g.abs() + 4) * U * self.a)
            self.w, self.dw = torch.ones_like(x), torch.zeros_like(x)
        self.u = x * self.w * self.s
        self.du = self.u.abs() * (self.dw + self.ds + 2 * U)
        if z is not None:
            self.q, self.dq = _sig(self.z)


def _rows(x, lengths):
    b, l = x.shape[:2]
    return [l] * b if lengths is None else [min(max(int(n), 0), l) for n in lengths]


def _order(n, reverse):
    return range(n - 1, -1, -1) if reverse else range(n)


def _live(x, lengths):
    if lengths is None:
        return torch.ones(x.shape[:2], dtype=torch.bool, device=x.device)[..., None]
    n = torch.tensor(_rows(x, lengths), device=x.device)
    return (torch.arange(x.shape[1], device=x.device)[None] < n[:, None])[..., None]


def _walk(T, h0, live, reverse):
    """States before and after every token, with magnitudes and errors: each [b, l, d]."""
    b, l, d = T.x.shape
    zero = torch.zeros(b, d, dtype=torch.float64, device=T.x.device)
    h = zero if h0 is None else h0.double()
    mag, err = h.abs(), zero
    keep = {k: [None] * l for k in ("h", "mag", "err", "h_", "mag_", "err_")}
    for t in _order(l, reverse):
        keep["h_"][t], keep["mag_"][t], keep["err_"][t] = h, mag, err
        a, on = T.a[:, t], live[:, t]
        m2 = a * mag + T.u[:, t].abs()
        e2 = a * err + (T.da[:, t] + 2 * U * a) * mag + T.du[:, t] + 4 * U * m2
        h = torch.where(on, a * h + T.u[:, t], h)
        mag, err = torch.where(on, m2, mag), torch.where(on, e2, err)
        keep["h"][t], keep["mag"][t], keep["err"][t] = h, mag, err
    out = {k: torch.stack(v, 1) if l else torch.zeros(b, 0, d, dtype=torch.float64, device=T.x.device)
           for k, v in keep.items()}
    return out, h, err


def rec(x, g, i=None, lam=None, z=None, h0=None, lengths=None, c=8.0, reverse=False):
    """{"out", "h_last"}: (value, bound) each."""
    T, live = _Tokens(x, g, i, lam, z, c), _live(x, lengths)
    s, h_last, err = _walk(T, h0, live, reverse)
    out, bound = s["h"], s["err"]
    if z is not None:
        gate = T.z * T.q
        out, bound = out * gate, gate.abs() * (bound + s["mag"] * (T.dq + 3 * U))
    zero = torch.zeros_like(out)
    return {"out": (torch.where(live, out, zero), torch.where(live, bound, zero)), "h_last": (h_last, err)}


def rec_bwd(x, g, dout, i=None, lam=None, z=None, h0=None, dh_last=None, lengths=None, c=8.0, reverse=False):
    """Gradients of sum(dout out) + sum(dh_last h_last): {name: (value, bound)}."""
    T, live = _Tokens(x, g, i, lam, z, c), _live(x, lengths)
    s, _, _ = _walk(T, h0, live, reverse)
    b, l, d = T.x.shape
    zero = torch.zeros_like(T.x)
    dout = torch.where(live, dout.double(), zero)
    gate, dgate = (torch.ones_like(T.x), zero) if z is None else (T.z * T.q, T.dq + 3 * U)
    e = dout * gate
    de = e.abs() * dgate
    cv = torch.zeros(b, d, dtype=torch.float64, device=T.x.device) if dh_last is None else dh_last.double()
    cm, ce = cv.abs(), torch.zeros_like(cv)
    D, Dm, De = [None] * l, [None] * l, [None] * l
    for t in reversed(_order(l, reverse)):
        v, m = e[:, t] + cv, e[:, t].abs() + cm
        err = de[:, t] + ce + 4 * U * m
        D[t], Dm[t], De[t] = v, m, err
        a, on = T.a[:, t], live[:, t]
        cv = torch.where(on, a * v, cv)
        ce = torch.where(on, a * err + (T.da[:, t] + 2 * U * a) * m, ce)
        cm = torch.where(on, a * m, cm)
    if l:
        D, Dm, De = (torch.stack(v, 1) for v in (D, Dm, De))
    else:
        D = Dm = De = zero
    out = {}
    ws = T.w * T.s
    out["dx"] = (D * ws, ws * (De + Dm * (T.dw + T.ds + 2 * U)))
    if i is not None:
        rest = 1 - T.s
        v = D * T.w * T.x * T.s * rest
        size = Dm * T.w * T.x.abs() * T.s
        out["di"] = (v, T.w * T.x.abs() * T.s * rest * De + size * (rest * (T.dw + T.ds + 5 * U) + T.s * T.ds + U))
    if z is not None:
        slope = T.q * (1 + T.z * (1 - T.q))
        dslope = T.q * T.dq * (1 + T.z.abs()) + T.q * T.z.abs() * (T.q * T.dq + 2 * U) + 3 * U * T.q * (1 + T.z.abs())
        out["dz"] = (dout * s["h"] * slope, dout.abs() * (s["err"] * slope.abs() + s["mag"] * (dslope + 2 * U * slope.abs())))
    dlog = D * T.a * s["h_"]
    err = T.a * s["mag_"] * De + T.a * Dm * s["err_"] + Dm * s["mag_"] * (T.da + 3 * U * T.a)
    if T.gated:
        f = torch.where(T.w > 0, T.a * T.a / torch.where(T.w > 0, T.w, torch.ones_like(T.w)), zero) * T.s * T.x.abs()
        dlog = dlog - D * f * torch.sign(T.x)
        err = err + f * (De + Dm * (2 * T.da / T.a.clamp(min=1e-300) + T.dw + T.ds + 7 * U)) + U * dlog.abs()
        size = Dm * (T.a * s["mag_"] + f)
        rest = 1 - T.r
        scale = T.rate * T.r
        out["dg"] = (-dlog * scale * rest, scale * (rest * err + size * (rest * (8 * U + T.dr + 4 * U) + T.r * T.dr + U)))
        term, terr = dlog * T.r, T.r * (err + size * (T.dr + 2 * U))
        term, terr, size = (torch.where(live, v, zero) for v in (term, terr, size * T.r))
        # a sum of b l terms: parts of at most 64 in a row, then over the parts
        out["dlam"] = (-T.slope * term.sum((0, 1)),
                       T.slope * (terr.sum((0, 1)) + size.sum((0, 1)) * (100 + b * l / 64) * U))
    else:
        out["dg"] = (dlog, err)
    out = {k: (torch.where(live, v, zero), torch.where(live, e, zero)) if v.dim() == 3 else (v, e)
           for k, (v, e) in out.items()}
    out["dh0"] = (cv, ce)
    return out


def eight(x):
    """(q, scale) of float32 x, and the float64 values that they stand for."""
    x = x.float()
    d = x.shape[-1]
    n = -(-d // BLOCK)
    y = torch.nn.functional.pad(x, (0, n * BLOCK - d)).unflatten(-1, (n, BLOCK))
    top = y.abs().amax(-1, keepdim=True)
    fine = torch.isfinite(top) & (top >= TINY)
    safe = torch.where(fine, top, torch.ones_like(top))
    full = torch.full_like(top, 127.0)  # quotients of tensors: torch multiplies by a number's reciprocal
    q = torch.where(fine, torch.round(y * (full / safe)), torch.zeros_like(y))
    scale = torch.where(fine, top / full, torch.where(torch.isfinite(top), torch.zeros_like(top),
                                                     torch.full_like(top, float("nan"))))
    value = q.double() * scale.double()
    return q.flatten(-2)[..., :d].to(torch.int8), scale[..., 0], value.flatten(-2)[..., :d]


def layer_norm(total, weight, bias, eps, dout=None, dtotal=None):
    """The norm of the rows of `total` and, with dout, its gradients: {name: (value, bound)}.
    Sums over a row are trees of at most sixteen additions in a row: 16 U of the mean magnitude."""
    x = total.double()
    n = x.shape[-1]
    one = torch.ones(n, dtype=torch.float64, device=x.device)
    w = one if weight is None else weight.double()
    c = 0 * one if bias is None else bias.double()
    mean = x.mean(-1, keepdim=True)
    y = x - mean
    sd = (y.square().mean(-1, keepdim=True) + eps).sqrt()
    y = y / sd
    # the mean's error, relative to the deviation, moves every value; the deviation scales them
    E = 17 * U * x.abs().mean(-1, keepdim=True) / sd + U * x.abs() / sd
    Em = E.amax(-1, keepdim=True)
    dy = E + y.abs() * (2 * Em + 24 * U)
    out = {"out": (y * w + c, w.abs() * (dy + 2 * U * y.abs()) + U * c.abs())}
    if dout is None:
        return out
    d = dout.double()
    dn = d * w
    m1, m2 = dn.mean(-1, keepdim=True), (dn * y).mean(-1, keepdim=True)
    a1, a2 = dn.abs().mean(-1, keepdim=True), (dn * y).abs().mean(-1, keepdim=True)
    dx = (dn - m1 - y * m2) / sd
    err = dn.abs() * 4 * U + 20 * U * a1 + y.abs() * (24 * U * a2 + (dn.abs() * dy).mean(-1, keepdim=True)) + dy * a2
    err = (err + (dn.abs() + a1 + y.abs() * a2) * (2 * Em + 30 * U)) / sd
    if dtotal is not None:
        dx = dx + dtotal.double()
        err = err + U * dx.abs()
    rows = x.numel() // n if n else 0
    lead = tuple(range(x.dim() - 1))
    chain = (100 + rows / 64) * U
    out.update(dx=(dx, err), dweight=((d * y).sum(lead), (d.abs() * dy).sum(lead) + chain * (d * y).abs().sum(lead)),
               dbias=(d.sum(lead), chain * d.abs().sum(lead)))
    return out
