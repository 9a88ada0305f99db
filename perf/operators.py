"""Cases of the gated delta rule and of the norms around a mixer, for timing and comparison.

Operators (``sscan`` names): ``delta_fwd``, ``delta_bwd`` and ``delta_step`` (the gated
delta rule over whole sequences, its gradients, and one token from a stored state),
``gated_norm`` / ``gated_norm_bwd`` (RMS norm of a mixer's heads fused with its silu
gate) and ``add_norm`` / ``add_norm_bwd`` (residual scale, residual sum and the next
block's RMS norm).  ``run`` calls them where ``own`` is true and otherwise computes the
same in plain float32 torch operations.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64
QK_EPS = 1e-6
NORM_EPS = 1e-6


def delta_case(op, b, l, hk, hv, dk, dv, dtype, qk_norm=True, state=False, ragged=False, name=None):
    c = dict(op=op, b=b, l=l, hk=hk, hv=hv, dk=dk, dv=dv, dtype=dtype, qk_norm=qk_norm, state=state, ragged=ragged)
    return c if name is None else dict(c, name=name)


def gated_case(op, n, h, g, dtype, gate_first=False, per_head=False, name=None):
    c = dict(op=op, n=n, h=h, g=g, dtype=dtype, gate_first=gate_first, per_head=per_head)
    return c if name is None else dict(c, name=name)


def add_case(op, n, d, dtype, res, scale=True, post=False, name=None):
    c = dict(op=op, n=n, d=d, dtype=dtype, res=res, scale=scale, post=post)
    return c if name is None else dict(c, name=name)


def listed():
    return [
        # one sequence being answered: the latency of one layer's step
        delta_case("delta_step", 1, 1, 8, 16, 128, 128, "bf16", name="step, one sequence"),
        # a full serving batch: every sequence's state is read and written
        delta_case("delta_step", 128, 1, 16, 32, 128, 128, "bf16", name="step, 128 sequences"),
        # short prompts of an odd length, small heads
        delta_case("delta_fwd", 3, 77, 2, 4, 64, 64, "bf16", state=True, name="prompts of 77"),
        # an ordinary training or prefill forward, keys shared by two value heads
        delta_case("delta_fwd", 4, 2048, 8, 16, 128, 128, "bf16", name="forward, 4 x 2048"),
        # one long document: few rows, a long axis
        delta_case("delta_fwd", 1, 32768, 8, 16, 128, 128, "bf16", state=True, name="document of 32768"),
        # float32, heads of odd sizes, a padded batch with its own lengths
        delta_case("delta_fwd", 3, 1000, 3, 3, 48, 72, "f32", qk_norm=False, state=True, ragged=True,
                   name="padded batch, f32"),
        # gradients of an ordinary training step's layer
        delta_case("delta_bwd", 2, 4096, 8, 16, 128, 128, "bf16", name="gradients, 2 x 4096"),
        # gradients in float32 with a learned entry state, odd length
        delta_case("delta_bwd", 2, 333, 2, 4, 64, 96, "f32", qk_norm=False, state=True, ragged=True,
                   name="gradients, f32, 333"),
        # the norm of the mixer's heads in training, forward
        gated_case("gated_norm", 16384, 16, 128, "bf16", name="gated norm of heads"),
        # and its gradients, one norm over the whole width, gate taken first
        gated_case("gated_norm_bwd", 8192, 1, 1536, "bf16", gate_first=True, per_head=True,
                   name="gated norm gradients, 1536"),
        # a few sequences being answered: latency of the residual sum and norm
        add_case("add_norm", 4, 768, "bf16", "f32", name="residual norm, 4 tokens"),
        # a training batch's residual sum with its block's output normed, gradients
        add_case("add_norm_bwd", 16384, 1536, "bf16", "f32", post=True, name="residual norm gradients"),
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["delta_step", "delta_fwd", "delta_fwd", "delta_bwd", "gated_norm", "gated_norm_bwd", "add_norm",
                     "add_norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op.startswith("delta"):
        hk = rng.choice([1, 2, 3, 4, 8])
        hv = hk * rng.choice([1, 1, 2, 3])
        dk = rng.choice([128, 128, 64, 64, 96, 40, 33, 128])
        dv = rng.choice([128, 128, 64, 96, 80, 50])
        if op == "delta_step":
            return delta_case(op, size(1, 160), 1, hk, hv, dk, dv, dtype, qk_norm=rng.random() < 0.7)
        most = (1 << 19 if op == "delta_fwd" else 1 << 17) // hv  # tokens in the batch
        l = size(1, min(most, 32768 if op == "delta_fwd" else 8192))
        b = size(1, max(1, min(32, most // l)))
        return delta_case(op, b, l, hk, hv, dk, dv, dtype, qk_norm=rng.random() < 0.7, state=rng.random() < 0.5,
                          ragged=rng.random() < 0.3)
    if op.startswith("gated"):
        g = size(32, 4096)
        h = rng.choice([1, 2, 8, 16]) if g <= 256 else rng.choice([1, 1, 2])
        n = size(1, max(2, (1 << 24) // (g * h)))
        return gated_case(op, n, h, g, dtype, gate_first=rng.random() < 0.4, per_head=rng.random() < 0.5)
    d = size(64, 8192)
    n = size(1, max(2, (1 << 24) // d))
    return add_case(op, n, d, dtype, rng.choice(["f32", "f32", dtype]), scale=rng.random() < 0.7,
                    post=rng.random() < 0.4)


# ---- inputs -----------------------------------------------------------------------

def _generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    return gen


def prepare(case, seed):
    gen = _generator(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    def rand(*shape):
        return torch.rand(shape, device="cuda", generator=gen)

    s = dict(case=case)
    if case["op"].startswith("delta"):
        b, l, hk, hv, dk, dv = (case[k] for k in ("b", "l", "hk", "hv", "dk", "dv"))
        # as after the short convolution and its silu
        q, k, v = (torch.nn.functional.silu(randn(b, l, h, d)) for h, d in ((hk, dk), (hk, dk), (hv, dv)))
        if not case["qk_norm"]:
            q = q * torch.rsqrt(q.square().sum(-1, keepdim=True) + QK_EPS)
            k = k * torch.rsqrt(k.square().sum(-1, keepdim=True) + QK_EPS)
        # g = -exp(A_log) * softplus(a + bias): decay rates 1..16, step sizes 1e-3..1e-1
        rate = 1 + 15 * rand(hv)
        step = torch.exp(math.log(1e-3) + rand(hv) * math.log(100.0))
        bias = torch.log(torch.expm1(step))
        s.update(q=q.to(dt), k=k.to(dt), v=v.to(dt),
                 g=-rate * torch.nn.functional.softplus(0.5 * randn(b, l, hv) + bias), beta=torch.sigmoid(randn(b, l, hv)))
        s["h0"] = 0.3 * randn(b, hv, dk, dv) if case["state"] or case["op"] == "delta_step" else None
        s["lengths"] = None
        if case["ragged"]:
            s["lengths"] = (rand(b) * (l + 1)).to(torch.int32).clamp_(0, l)
        if case["op"] == "delta_step":
            for key in ("q", "k", "v", "g", "beta"):
                s[key] = s[key][:, 0].contiguous()
        if case["op"] == "delta_bwd":
            s["dout"] = randn(b, l, hv, dv).to(dt)
            s["dh_last"] = 0.3 * randn(b, hv, dk, dv) if case["state"] else None
        return s
    if case["op"].startswith("gated"):
        n, h, g = case["n"], case["h"], case["g"]
        s.update(x=randn(n, h, g).to(dt), z=randn(n, h, g).to(dt),
                 weight=1 + 0.1 * (randn(h, g) if case["per_head"] else randn(g)))
        if case["op"].endswith("bwd"):
            s["dout"] = randn(n, h, g).to(dt)
        return s
    n, d = case["n"], case["d"]
    s.update(x=randn(n, d).to(dt), residual=(3 * randn(n, d)).to(DTYPES[case["res"]]), weight=1 + 0.1 * randn(d),
             scale=0.1 + 0.02 * randn(d) if case["scale"] else None,
             post_weight=1 + 0.1 * randn(d) if case["post"] else None)
    if case["op"].endswith("bwd"):  # here "residual" is the sum that the forward stored
        s.update(dout=randn(n, d).to(dt), dresidual=randn(n, d).to(DTYPES[case["res"]]))
    return s


# ---- one pass ---------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else PLAIN[state["case"]["op"]](state)


def _run_own(s):
    from selective_state_space_sscan_amd import sscan

    c = s["case"]
    if c["op"] == "delta_step":
        out = sscan.delta_step(s["h0"], s["q"], s["k"], s["v"], s["g"], s["beta"], qk_norm=c["qk_norm"])
        return {"out": out, "state": s["h0"]}
    if c["op"] == "delta_fwd":
        out, h_last = sscan.delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], h0=s["h0"], lengths=s["lengths"],
                                      qk_norm=c["qk_norm"])
        return {"out": out, "h_last": h_last}
    if c["op"] == "delta_bwd":
        return sscan.delta_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dout"], h0=s["h0"],
                               dh_last=s["dh_last"], lengths=s["lengths"], qk_norm=c["qk_norm"])
    if c["op"] == "gated_norm":
        return sscan.gated_norm(s["x"], s["z"], s["weight"], eps=NORM_EPS, gate_first=c["gate_first"])
    if c["op"] == "gated_norm_bwd":
        return sscan.gated_norm_bwd(s["x"], s["z"], s["dout"], s["weight"], eps=NORM_EPS, gate_first=c["gate_first"])
    if c["op"] == "add_norm":
        return sscan.add_norm(s["x"], s["residual"], s["weight"], scale=s["scale"], post_weight=s["post_weight"],
                              eps=NORM_EPS)
    g = sscan.add_norm_bwd(s["x"], s["residual"], s["dout"], s["weight"], dresidual_out=s["dresidual"],
                           scale=s["scale"], post_weight=s["post_weight"], eps=NORM_EPS)
    return {k: v for k, v in g.items() if v is not None}


# ---- plain forms ------------------------------------------------------------------

def _unit(x):
    return x * torch.rsqrt(x.square().sum(-1, keepdim=True) + QK_EPS)


def _keep(c, s, x):
    """x [b, l, ...] with zeros from each row's length on (chosen, not multiplied)."""
    if s["lengths"] is None:
        return x
    t = torch.arange(c["l"], device=x.device)
    inside = t[None, :] < s["lengths"][:, None]
    return torch.where(inside.view(inside.shape + (1,) * (x.dim() - 2)), x, torch.zeros_like(x))


def _delta_chunks(c, s, q, k, v, g, beta, h0):
    """The gated delta rule in chunks of 64 tokens, float32: (out, last state)."""
    b, l, hv, dk, dv = c["b"], c["l"], c["hv"], c["dk"], c["dv"]
    q, k, v, g, beta = (_keep(c, s, x) for x in (q, k, v, g, beta))
    if c["qk_norm"]:
        q, k = _unit(q), _unit(k)
    share = hv // c["hk"]
    q, k = (x.repeat_interleave(share, dim=2) for x in (q, k))
    n = -(-l // CHUNK)

    def chunks(x):  # [b, l, h, ...] -> [b, h, n, CHUNK, ...]
        x = torch.nn.functional.pad(x.movedim(1, -1), (0, n * CHUNK - l)).movedim(-1, 1)
        return x.reshape((b, n, CHUNK) + x.shape[2:]).movedim(3, 1)

    q, k, v, g, beta = (chunks(x) for x in (q, k, v, g, beta))
    q = q * dk ** -0.5
    run_g = g.cumsum(-1)
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    decay = torch.where(lower, run_g[..., :, None] - run_g[..., None, :], run_g.new_zeros(())).exp()
    kt = k.transpose(-1, -2).contiguous()
    a = torch.where(lower.tril(-1), beta[..., None] * decay * torch.matmul(k, kt), run_g.new_zeros(()))
    # (I + a)^-1 of a nilpotent a: (I - a)(I + a^2)(I + a^4)...
    eye = torch.eye(CHUNK, device=q.device)
    inv, power = eye - a, a
    for _ in range(5):
        power = torch.matmul(power, power)
        inv = inv + torch.matmul(inv, power)
    attn = torch.where(lower, decay * torch.matmul(q, kt), run_g.new_zeros(()))
    u0 = torch.matmul(inv, beta[..., None] * v)
    w = torch.matmul(inv, (beta * run_g.exp())[..., None] * k)
    q_in = q * run_g.exp()[..., None]
    k_out = (k * (run_g[..., -1:] - run_g).exp()[..., None]).transpose(-1, -2).contiguous()
    last = run_g[..., -1, None].exp()
    h = q.new_zeros(b, hv, dk, dv) if h0 is None else h0
    outs = []
    for i in range(n):
        u = u0[:, :, i] - torch.matmul(w[:, :, i], h)
        outs.append(torch.matmul(q_in[:, :, i], h) + torch.matmul(attn[:, :, i], u))
        h = last[:, :, i, None] * h + torch.matmul(k_out[:, :, i], u)
    out = torch.stack(outs, 2).reshape(b, hv, n * CHUNK, dv)[:, :, :l].transpose(1, 2)
    return _keep(c, s, out), h


def _plain_delta_fwd(s):
    c = s["case"]
    out, h = _delta_chunks(c, s, *(s[k].float() for k in ("q", "k", "v", "g", "beta")), s["h0"])
    return {"out": out.to(DTYPES[c["dtype"]]).contiguous(), "h_last": h}


def _plain_delta_bwd(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    ins = [s[k].float().clone().requires_grad_(True) for k in ("q", "k", "v", "g", "beta")]
    h0 = s["h0"] if s["h0"] is not None else torch.zeros(c["b"], c["hv"], c["dk"], c["dv"], device="cuda")
    h0 = h0.clone().requires_grad_(True)
    with torch.enable_grad():
        out, h = _delta_chunks(c, s, *ins, h0)
        dh = torch.zeros_like(h) if s["dh_last"] is None else s["dh_last"]
        grads = torch.autograd.grad([out, h], ins + [h0], [s["dout"].float(), dh])
    cast = (dt, dt, dt, torch.float32, torch.float32, torch.float32)
    return {n: g.to(t).contiguous() for n, g, t in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), grads, cast)}


def _plain_delta_step(s):
    c = s["case"]
    q, k, v = (s[x].float() for x in ("q", "k", "v"))
    if c["qk_norm"]:
        q, k = _unit(q), _unit(k)
    share = c["hv"] // c["hk"]
    q, k = (x.repeat_interleave(share, dim=1) for x in (q, k))
    h = s["h0"].mul_(s["g"].exp()[..., None, None])
    u = s["beta"][..., None] * (v - (k[..., None] * h).sum(-2))
    h += k[..., None] * u[..., None, :]
    out = ((q * c["dk"] ** -0.5)[..., None] * h).sum(-2)
    return {"out": out.to(DTYPES[c["dtype"]]), "state": h}


def _rms(x):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + NORM_EPS)


def _rms_back(x, r, dn):
    """Gradient of n = x * r at x, r = 1 / rms."""
    return r * (dn - x * (r * r) * (dn * x).mean(-1, keepdim=True))


def _plain_gated_norm(s):
    c, x, z = s["case"], s["x"].float(), s["z"].float()
    gate = z / (1 + torch.exp(-z))
    if c["gate_first"]:
        y = x * gate
        y = y * _rms(y) * s["weight"]
    else:
        y = x * _rms(x) * s["weight"] * gate
    return y.to(s["x"].dtype)


def _plain_gated_norm_bwd(s):
    c, x, z, dout, w = s["case"], s["x"].float(), s["z"].float(), s["dout"].float(), s["weight"]
    sig = 1 / (1 + torch.exp(-z))
    gate, slope = z * sig, sig * (1 + z * (1 - sig))
    if c["gate_first"]:
        y = x * gate
        r = _rms(y)
        dw = dout * y * r
        dy = _rms_back(y, r, dout * w)
        dx, dz = dy * gate, dy * x * slope
    else:
        r = _rms(x)
        dw = dout * gate * x * r
        dx, dz = _rms_back(x, r, dout * gate * w), dout * x * r * w * slope
    dw = dw.sum(0) if c["per_head"] else dw.sum((0, 1))
    return {"dx": dx.to(s["x"].dtype), "dz": dz.to(s["x"].dtype), "dweight": dw}


def _plain_add_norm(s):
    a = s["x"].float()
    if s["post_weight"] is not None:
        a = a * _rms(a) * s["post_weight"]
    if s["scale"] is not None:
        a = a * s["scale"]
    total = (s["residual"].float() + a).to(s["residual"].dtype)
    y = total.float()
    return (y * _rms(y) * s["weight"]).to(s["x"].dtype), total


def _plain_add_norm_bwd(s):
    x, total, dout = s["x"].float(), s["residual"].float(), s["dout"].float()
    r = _rms(total)
    out = {"dweight": (dout * total * r).sum(0)}
    dres = s["dresidual"].float() + _rms_back(total, r, dout * s["weight"])
    out["dresidual"] = dres.to(s["residual"].dtype)
    a = x
    if s["post_weight"] is not None:
        rx = _rms(x)
        a = x * rx * s["post_weight"]
    da = dres
    if s["scale"] is not None:
        out["dscale"] = (dres * a).sum(0)
        da = dres * s["scale"]
    if s["post_weight"] is not None:
        out["dpost_weight"] = (da * x * rx).sum(0)
        da = _rms_back(x, rx, da * s["post_weight"])
    out["dx"] = da.to(s["x"].dtype)
    return out


PLAIN = {"delta_step": _plain_delta_step, "delta_fwd": _plain_delta_fwd, "delta_bwd": _plain_delta_bwd,
         "gated_norm": _plain_gated_norm, "gated_norm_bwd": _plain_gated_norm_bwd, "add_norm": _plain_add_norm,
         "add_norm_bwd": _plain_add_norm_bwd}


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    esz = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("delta"):
        b, l, hk, hv, dk, dv = (case[k] for k in ("b", "l", "hk", "hv", "dk", "dv"))
        t = b * l
        qk, vo, gates, st = t * hk * dk * esz, t * hv * dv * esz, t * hv * 4, b * hv * dk * dv * 4
        if case["op"] == "delta_bwd":
            # the recurrence recomputed (6 dk dv a token), its adjoint (12 dk dv)
            return {"bytes": 4 * qk + 3 * vo + 4 * gates + st * (3 if case["state"] else 1),
                    "flops": 18.0 * t * hv * dk * dv}
        reads_state = case["state"] or case["op"] == "delta_step"
        return {"bytes": 2 * qk + 2 * vo + 2 * gates + st * (2 if reads_state else 1),
                "flops": 6.0 * t * hv * dk * dv}
    if case["op"].startswith("gated"):
        e = case["n"] * case["h"] * case["g"]
        w = 4 * case["g"] * (case["h"] if case["per_head"] else 1)
        back = case["op"].endswith("bwd")
        return {"bytes": e * esz * (5 if back else 3) + w * (2 if back else 1), "flops": e * (24.0 if back else 9.0)}
    e, rsz = case["n"] * case["d"], 4 if case["res"] == "f32" else 2
    vecs = 4 * case["d"] * (1 + case["scale"] + case["post"])
    if case["op"].endswith("bwd"):
        return {"bytes": e * (3 * esz + 3 * rsz) + 2 * vecs, "flops": 24.0 * e}
    return {"bytes": e * (2 * esz + 2 * rsz) + vecs, "flops": 9.0 * e}


# ---- the definition in 64 bits ----------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if case["op"].startswith("delta"):
        return _exact_delta(case, d)
    return _exact_norms(case, s, d)


def _exact_delta(c, d):
    """Token by token: S <- e^g S; u = beta (v - S^T k); S <- S + k u^T; o = S^T q / sqrt(dk)."""
    step = c["op"] == "delta_step"
    q, k, v, g, beta = (d[n][:, None] if step else d[n] for n in ("q", "k", "v", "g", "beta"))
    b, l, hv, dk, dv = c["b"], c["l"], c["hv"], c["dk"], c["dv"]
    share, back = hv // c["hk"], c["op"] == "delta_bwd"
    if back and b * hv * dk * dv * l * 8 > 1 << 36:
        return None
    rq = rk = None
    if c["qk_norm"]:
        rq, rk = ((x * x).sum(-1, keepdim=True).add(QK_EPS).rsqrt() for x in (q, k))
    qn, kn = ((x if r is None else x * r).repeat_interleave(share, 2) for x, r in ((q, rq), (k, rk)))
    qn = qn / math.sqrt(dk)
    lengths = torch.full((b,), l, device="cuda") if d["lengths"] is None else d["lengths"]
    live = (torch.arange(l, device="cuda")[:, None] < lengths[None, :])[..., None]  # [l, b, 1]
    # a token past its row's length leaves the state as it is
    eg = torch.where(live, g.exp().movedim(1, 0), g.new_ones(()))
    bt = torch.where(live, beta.movedim(1, 0), g.new_zeros(()))
    qt, kt, vt = (torch.where(live[..., None], x.movedim(1, 0), x.new_zeros(())) for x in (qn, kn, v))
    h = torch.zeros(b, hv, dk, dv, dtype=torch.float64, device="cuda") if d["h0"] is None else d["h0"].clone()
    before, errs, outs = [], [], []
    for t in range(l):
        if back:
            before.append(h)
        h = h * eg[t][..., None, None]
        e = vt[t] - torch.matmul(kt[t][..., None, :], h)[..., 0, :]
        h = h + kt[t][..., None] * (bt[t][..., None] * e)[..., None, :]
        errs.append(e)
        outs.append(torch.matmul(qt[t][..., None, :], h)[..., 0, :])
    if step:
        return {"out": outs[0], "state": h}
    if not back:
        return {"out": torch.stack(outs, 1), "h_last": h}
    dh = torch.zeros_like(h) if d["dh_last"] is None else d["dh_last"].clone()
    dout = torch.where(live[..., None], d["dout"].movedim(1, 0), h.new_zeros(()))
    dq, dk_, dv_, dg, db = [], [], [], [], []
    for t in range(l - 1, -1, -1):
        decayed = before[t] * eg[t][..., None, None]
        u = bt[t][..., None] * errs[t]
        after = decayed + kt[t][..., None] * u[..., None, :]
        dq.append(torch.matmul(after, dout[t][..., None])[..., 0])
        dh = dh + qt[t][..., None] * dout[t][..., None, :]
        du = torch.matmul(kt[t][..., None, :], dh)[..., 0, :]
        de = bt[t][..., None] * du
        db.append((du * errs[t]).sum(-1))
        dv_.append(de)
        dk_.append(torch.matmul(dh, u[..., None])[..., 0] - torch.matmul(decayed, de[..., None])[..., 0])
        dh = dh - kt[t][..., None] * de[..., None, :]
        dg.append((dh * decayed).sum((-1, -2)))
        dh = dh * eg[t][..., None, None]
    alive = live.movedim(0, 1)

    def rows(parts, heads=None):
        x = torch.stack(parts[::-1], 1)
        x = torch.where(alive if x.dim() == 3 else alive[..., None], x, x.new_zeros(()))
        return x if heads is None else x.reshape(b, l, heads, share, dk).sum(3)

    gq, gk = rows(dq, c["hk"]) / math.sqrt(dk), rows(dk_, c["hk"])
    if c["qk_norm"]:
        gq = rq * (gq - q * rq * rq * (gq * q).sum(-1, keepdim=True))
        gk = rk * (gk - k * rk * rk * (gk * k).sum(-1, keepdim=True))
    return {"dq": gq, "dk": gk, "dv": rows(dv_), "dg": rows(dg), "dbeta": rows(db), "dh0": dh}


def _exact_norms(c, s, d):
    """From the definitions, gradients by differentiation in 64 bits."""
    def norm(x):
        return x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + NORM_EPS).sqrt()

    back = c["op"].endswith("bwd")
    w = d["weight"]
    if c["op"].startswith("gated"):
        ins = [x.detach().requires_grad_(back) for x in (d["x"], d["z"], w)]
        x, z, w = ins
        gate = z * torch.sigmoid(z)
        y = norm(x * gate) * w if c["gate_first"] else norm(x) * w * gate
        if not back:
            return y
        return dict(zip(("dx", "dz", "dweight"), torch.autograd.grad(y, ins, d["dout"])))
    x, scale, post = d["x"], d["scale"], d["post_weight"]

    def branch(x, scale, post):
        a = x if post is None else norm(x) * post
        return a if scale is None else a * scale

    if not back:
        total = d["residual"] + branch(x, scale, post)
        if s["residual"].dtype is torch.float32:
            return norm(total) * w, total
        # a sum stored in fewer bits is normed as it was stored, and that is rounded from 32 bits
        return None, total
    total = d["residual"].detach().requires_grad_(True)
    w = w.detach().requires_grad_(True)
    dres, dw = torch.autograd.grad(norm(total) * w, [total, w], d["dout"])
    dres = dres + d["dresidual"]
    names, ins = ["dx"], [x.detach().requires_grad_(True)]
    for n, t in (("dscale", scale), ("dpost_weight", post)):
        if t is not None:
            names.append(n)
            ins.append(t.detach().requires_grad_(True))
    it = iter(ins[1:])
    y = branch(ins[0], next(it) if scale is not None else None, next(it) if post is not None else None)
    got = dict(zip(names, torch.autograd.grad(y, ins, dres)))
    return dict(got, dresidual=dres, dweight=dw)
