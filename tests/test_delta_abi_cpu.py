"""Argument checks of the gated delta rule's and the norms' C entry points, without a GPU:
fake addresses, never dereferenced."""
import ctypes
import os

import pytest

from selective_state_space_sscan_amd import sscan

OK, ENULL, ESHAPE, EUNSUP, EALIGN, EWS, EHIP, EALIAS = 0, -1, -2, -3, -4, -5, -6, -7


@pytest.fixture(scope="module")
def lib():
    other = os.environ.get("SSCAN_TEST_LIBRARY")
    if other:
        return sscan.load_library(other)
    if not os.path.exists(sscan.LIB_PATH):
        from selective_state_space_sscan_amd import build
        build.build()
    return sscan.load_library()


class Fake:
    def __init__(self):
        self.next = 1 << 40

    def __call__(self, nbytes):
        p = self.next
        self.next += (nbytes + 4096) // 256 * 256 + 256
        return p


B, L, HK, HV, DK, DV = 2, 100, 2, 4, 64, 96


def delta(b=B, L=L, hk=HK, hv=HV, dk=DK, dv=DV, io=1, **over):
    f = Fake()
    e = 2 if io == 1 else 4
    I3 = ctypes.c_int64 * 3
    qk, vv, gg = I3(L * hk * dk, hk * dk, dk), I3(L * hv * dv, hv * dv, dv), I3(L * hv, hv, 1)
    a = dict(q=f(b * L * hk * dk * e), k=f(b * L * hk * dk * e), v=f(b * L * hv * dv * e), g=f(b * L * hv * 4),
             beta=f(b * L * hv * 4), lengths=f(b * 4), h0=f(b * hv * dk * dv * 4), q_stride=qk, k_stride=qk,
             v_stride=vv, g_stride=gg, beta_stride=gg, batch=b, len=L, qk_heads=hk, v_heads=hv, dk=dk, dv=dv,
             scale=0.125, qk_norm=1, io_dtype=io)
    rest = dict(out=f(b * L * hv * dv * e), last=f(b * hv * dk * dv * 4), ws=f(1 << 34), ws_bytes=1 << 34,
                dout=f(b * L * hv * dv * e), dh=f(b * hv * dk * dv * 4), dq=f(b * L * hk * dk * e),
                dk_=f(b * L * hk * dk * e), dv_=f(b * L * hv * dv * e), dg=f(b * L * hv * 4), dbeta=f(b * L * hv * 4),
                dh0=f(b * hv * dk * dv * 4))
    for key, v in over.items():
        (a if key in a else rest)[key] = v
    return sscan.DeltaParams(**a), rest


def fwd(lib, **over):
    p, r = delta(**over)
    return lib.sscan_validate_delta_fwd(ctypes.byref(p), r["out"], r["last"], r["ws"], r["ws_bytes"])


def bwd(lib, **over):
    p, r = delta(**over)
    g = sscan.DeltaGrads(r["dq"], r["dk_"], r["dv_"], r["dg"], r["dbeta"], r["dh0"])
    return lib.sscan_validate_delta_bwd(ctypes.byref(p), r["dout"], r["dh"], ctypes.byref(g), r["ws"], r["ws_bytes"])


I3 = ctypes.c_int64 * 3

DELTA = [
    (dict(), OK), (dict(lengths=None, h0=None), OK), (dict(io=0), OK), (dict(q=None), ENULL), (dict(beta=None), ENULL),
    (dict(batch=-1), ESHAPE), (dict(len=(1 << 30) + 1), ESHAPE), (dict(qk_heads=3), ESHAPE), (dict(qk_heads=0), ESHAPE),
    (dict(dk=129), EUNSUP), (dict(dk=0), EUNSUP), (dict(dv=257), EUNSUP), (dict(io_dtype=7), EUNSUP),
    (dict(qk_norm=2), EUNSUP), (dict(scale=float("inf")), EUNSUP), (dict(scale=float("nan")), EUNSUP),
    (dict(q=(1 << 40) + 1), EALIGN), (dict(g=(1 << 40) + 2), EALIGN), (dict(h0=(1 << 41) + 8), EALIGN),
    (dict(q_stride=I3(-1, 128, 64)), ESHAPE), (dict(v_stride=I3(0, 1 << 23, 96)), EUNSUP),
    (dict(k_stride=I3(1 << 60, 128, 64)), ESHAPE), (dict(ws=None), EWS), (dict(ws_bytes=1000), EWS),
    (dict(ws=(1 << 42) + 16), EALIGN), (dict(batch=1 << 40, len=1), ESHAPE),
]


@pytest.mark.parametrize("over,status", DELTA)
def test_validate_delta(lib, over, status):
    assert fwd(lib, **over) == status
    assert bwd(lib, **over) == status


def test_validate_delta_outputs(lib):
    p, r = delta()
    assert fwd(lib, out=None) == ENULL and fwd(lib, last=None) == ENULL
    assert fwd(lib, last=p.h0) == OK  # the state in place
    assert fwd(lib, last=p.h0 + 16) == EALIAS
    assert fwd(lib, out=p.v) == EALIAS and fwd(lib, out=p.g) == EALIAS and fwd(lib, out=r["last"]) == EALIAS
    assert fwd(lib, last=r["ws"] + 256) == EALIAS
    assert bwd(lib, dout=None) == ENULL and bwd(lib, dg=None) == ENULL and bwd(lib, dh0=None) == OK
    assert bwd(lib, dq=r["dk_"]) == EALIAS and bwd(lib, dq=p.q) == EALIAS and bwd(lib, dv_=r["dout"]) == EALIAS
    assert bwd(lib, dh0=r["dh"]) == EALIAS and bwd(lib, dbeta=r["ws"]) == EALIAS
    assert lib.sscan_validate_delta_fwd(None, 0, 0, 0, 0) == ENULL
    assert lib.sscan_validate_delta_bwd(ctypes.byref(p), r["dout"], None, None, r["ws"], 1 << 34) == ENULL


def test_validate_delta_empty(lib):
    assert fwd(lib, batch=0, q=None, k=None, v=None, g=None, beta=None, out=None, last=None, ws=None) == OK
    assert fwd(lib, L=0, len=0, q=None, k=None, v=None, g=None, beta=None, out=None, ws=None) == OK
    assert fwd(lib, L=0, len=0, q=None, k=None, v=None, g=None, beta=None, out=None, ws=None, last=None) == ENULL
    assert bwd(lib, L=0, len=0, q=None, k=None, v=None, g=None, beta=None, dout=None, dq=None, dk_=None, dv_=None,
               dg=None, dbeta=None, ws=None) == OK


def test_validate_delta_step(lib):
    def step(state=None, out=None, **over):
        p, r = delta(L=1, h0=None, **over)
        return lib.sscan_validate_delta_step(ctypes.byref(p), state or r["last"], out or r["out"])

    assert step() == OK
    p, r = delta(L=1)
    assert lib.sscan_validate_delta_step(ctypes.byref(p), r["last"], r["out"]) == EUNSUP  # h0 given
    p, r = delta(L=2, h0=None)
    assert lib.sscan_validate_delta_step(ctypes.byref(p), r["last"], r["out"]) == ESHAPE
    assert step(state=(1 << 41) + 4) == EALIGN
    p, r = delta(L=1, h0=None)
    assert lib.sscan_validate_delta_step(ctypes.byref(p), p.q, r["out"]) == EALIAS
    assert lib.sscan_validate_delta_step(ctypes.byref(p), None, r["out"]) == ENULL


@pytest.mark.parametrize("b,L,hk,hv,dk,dv", [(1, 1, 1, 1, 1, 1), (4, 2048, 8, 16, 128, 128), (1, 32768, 8, 16, 128, 128),
                                             (3, 1000, 3, 3, 48, 72), (1, 1 << 20, 1, 1, 128, 256)])
@pytest.mark.parametrize("io", [0, 1])
def test_delta_workspaces(lib, b, L, hk, hv, dk, dv, io):
    """What a call asks for is enough for it, and one byte less is not."""
    for back in (False, True):
        f = lib.sscan_delta_bwd_workspace_bytes if back else lib.sscan_delta_workspace_bytes
        n = f(b, L, hk, hv, dk, dv, io)
        assert n % 256 == 0
        chunks = -(-L // 64) * b * hv
        if back or L > 8:
            assert n >= chunks * 6 * 1024 * 3
            call = bwd if back else fwd
            kw = dict(b=b, L=L, hk=hk, hv=hv, dk=dk, dv=dv, io=io)
            assert call(lib, **kw, ws_bytes=n) == OK
            assert call(lib, **kw, ws_bytes=n - 1) == EWS
        else:
            assert n == 0
        assert f(-1, L, hk, hv, dk, dv, io) == 0 and f(b, L, hk, hv, 500, dv, io) == 0 and f(b, L, 0, hv, dk, dv, io) == 0


def gated(rows=5, heads=3, size=64, io=1, per_head=0, **over):
    f = Fake()
    e = 2 if io == 1 else 4
    n = rows * heads * size * e
    I2 = ctypes.c_int64 * 2
    a = dict(x=f(n), z=f(n), weight=f(heads * size * 4), x_stride=I2(heads * size, size), z_stride=I2(heads * size, size),
             rows=rows, heads=heads, size=size, eps=1e-6, gate_first=0, per_head=per_head, io_dtype=io)
    r = dict(out=f(n), dout=f(n), dx=f(n), dz=f(n), dw=f(heads * size * 4), ws=f(1 << 30), ws_bytes=1 << 30)
    for key, v in over.items():
        (a if key in a else r)[key] = v
    return sscan.GatedNormParams(**a), r


I2 = ctypes.c_int64 * 2
GATED = [(dict(), OK), (dict(io=0, per_head=1), OK), (dict(x=None), ENULL), (dict(z=None), ENULL),
         (dict(per_head=1, weight=None), ENULL), (dict(rows=-1), ESHAPE), (dict(size=0), EUNSUP), (dict(size=8193), EUNSUP),
         (dict(eps=float("nan")), EUNSUP), (dict(eps=-1.0), EUNSUP), (dict(gate_first=3), EUNSUP), (dict(io_dtype=9), EUNSUP),
         (dict(x=(1 << 40) + 1), EALIGN), (dict(z_stride=I2(-4, 1)), ESHAPE), (dict(rows=1 << 50), ESHAPE)]


@pytest.mark.parametrize("over,status", GATED)
def test_validate_gated_norm(lib, over, status):
    p, r = gated(**over)
    assert lib.sscan_validate_gated_norm(ctypes.byref(p), r["out"]) == status
    w = None if over.get("weight", 1) is None else r["dw"]
    assert lib.sscan_validate_gated_norm_bwd(ctypes.byref(p), r["dout"], r["dx"], r["dz"], w, r["ws"], r["ws_bytes"]) == status


def test_validate_gated_norm_outputs(lib):
    p, r = gated()
    v, vb = lib.sscan_validate_gated_norm, lib.sscan_validate_gated_norm_bwd
    ref = ctypes.byref(p)
    assert v(ref, None) == ENULL and v(ref, p.x) == EALIAS and v(ref, p.weight) == EALIAS and v(None, r["out"]) == ENULL
    args = [r["dout"], r["dx"], r["dz"], r["dw"], r["ws"], r["ws_bytes"]]
    for k, x, status in ((0, None, ENULL), (1, None, ENULL), (2, r["dx"], EALIAS), (1, r["dout"], EALIAS), (3, p.x, EALIAS),
                         (4, None, EWS), (5, 16, EWS), (4, r["ws"] + 8, EALIGN), (3, None, OK)):
        assert vb(ref, *[x if i == k else y for i, y in enumerate(args)]) == status, k
    q, _ = gated(weight=None)
    assert vb(ctypes.byref(q), *args) == ENULL  # a gradient of a weight that is not there
    n = lib.sscan_gated_norm_bwd_workspace_bytes(5, 3, 64)
    assert vb(ref, *args[:5], n) == OK and vb(ref, *args[:5], n - 1) == EWS
    assert lib.sscan_gated_norm_bwd_workspace_bytes(0, 3, 64) == 0


def add(rows=5, size=64, io=1, res=0, **over):
    f = Fake()
    e, s = (2 if t == 1 else 4 for t in (io, res))
    a = dict(x=f(rows * size * e), residual=f(rows * size * s), weight=f(size * 4), scale=f(size * 4),
             post_weight=f(size * 4), rows=rows, size=size, eps=1e-6, io_dtype=io, residual_dtype=res)
    r = dict(out=f(rows * size * e), total=f(rows * size * s), dout=f(rows * size * e), dtotal=f(rows * size * s),
             dx=f(rows * size * e), dres=f(rows * size * s), dw=f(size * 4), ds=f(size * 4), dp=f(size * 4), ws=f(1 << 30),
             ws_bytes=1 << 30)
    for key, v in over.items():
        (a if key in a else r)[key] = v
    return sscan.AddNormParams(**a), r


ADD = [(dict(), OK), (dict(res=1, io=0), OK), (dict(x=None), ENULL), (dict(rows=-2), ESHAPE), (dict(size=0), EUNSUP),
       (dict(size=9000), EUNSUP), (dict(eps=float("inf")), EUNSUP), (dict(io_dtype=3), EUNSUP), (dict(residual_dtype=3), EUNSUP),
       (dict(residual=(1 << 40) + 2), EALIGN), (dict(scale=(1 << 40) + 1), EALIGN), (dict(rows=1 << 49), ESHAPE)]


@pytest.mark.parametrize("over,status", ADD)
def test_validate_add_norm(lib, over, status):
    p, r = add(**over)
    assert lib.sscan_validate_add_norm(ctypes.byref(p), r["out"], r["total"]) == status
    assert lib.sscan_validate_add_norm_bwd(ctypes.byref(p), r["dout"], r["dtotal"], r["dx"], r["dres"], r["dw"], r["ds"],
                                           r["dp"], r["ws"], r["ws_bytes"]) == status


def test_validate_add_norm_outputs(lib):
    p, r = add()
    ref = ctypes.byref(p)
    v, vb = lib.sscan_validate_add_norm, lib.sscan_validate_add_norm_bwd
    assert v(ref, r["out"], p.residual) == OK  # the residual in place
    assert v(ref, r["out"], p.residual + 4) == EALIAS and v(ref, r["out"], p.x) == EALIAS and v(ref, r["total"], r["total"]) == EALIAS
    assert v(ref, None, r["total"]) == ENULL and v(ref, p.weight, r["total"]) == EALIAS
    q, _ = add(residual=None)
    assert v(ctypes.byref(q), r["out"], r["total"]) == OK
    args = [r["dout"], r["dtotal"], r["dx"], r["dres"], r["dw"], r["ds"], r["dp"], r["ws"], r["ws_bytes"]]
    assert vb(ctypes.byref(q), *args) == ENULL  # the stored sum is needed
    for k, x, status in ((1, None, OK), (3, r["dtotal"], OK), (3, r["dtotal"] + 4, EALIAS), (2, r["dout"], EALIAS),
                         (2, None, ENULL), (4, None, OK), (5, r["dw"], EALIAS), (7, None, EWS), (8, 8, EWS)):
        assert vb(ref, *[x if i == k else y for i, y in enumerate(args)]) == status, (k, x)
    for name, k in (("weight", 4), ("scale", 5), ("post_weight", 6)):
        q, _ = add(**{name: None})
        assert vb(ctypes.byref(q), *args) == ENULL, name
        assert vb(ctypes.byref(q), *[None if i == k else y for i, y in enumerate(args)]) == OK, name


def test_run_entry_points_reject_before_any_hip_call(lib):
    p, r = delta(dk=500)
    ref = ctypes.byref(p)
    assert lib.sscan_delta_fwd(ref, r["out"], r["last"], None, r["ws"], r["ws_bytes"]) == EUNSUP
    assert lib.sscan_delta_step(ref, r["last"], r["out"], None) == ESHAPE
    g = sscan.DeltaGrads(r["dq"], r["dk_"], r["dv_"], r["dg"], r["dbeta"], r["dh0"])
    assert lib.sscan_delta_bwd(ref, r["dout"], None, ctypes.byref(g), None, r["ws"], r["ws_bytes"]) == EUNSUP
    p, r = gated(size=0)
    assert lib.sscan_gated_norm(ctypes.byref(p), r["out"], None) == EUNSUP
    p, r = add(size=0)
    assert lib.sscan_add_norm(ctypes.byref(p), r["out"], r["total"], None) == EUNSUP


def test_packed_parameters_match_the_structs():
    """The bindings pack the parameter structs by hand: field by field the same bytes."""
    p, _ = delta()
    order = [getattr(p, n) or 0 for n in ("q", "k", "v", "g", "beta", "lengths", "h0")]
    strides = [x for n in ("q", "k", "v", "g", "beta") for x in getattr(p, n + "_stride")]
    raw = sscan._DELTA.pack(*order, *strides, p.batch, p.len, p.qk_heads, p.v_heads, p.dk, p.dv, p.scale, p.qk_norm, p.io_dtype)
    assert raw == bytes(p)
    p, _ = gated()
    assert sscan._GATED.pack(p.x, p.z, p.weight, *p.x_stride, *p.z_stride, p.rows, p.heads, p.size, p.eps, p.gate_first,
                             p.per_head, p.io_dtype) == bytes(p)
    p, _ = add()
    assert sscan._ADD.pack(p.x, p.residual, p.weight, p.scale, p.post_weight, p.rows, p.size, p.eps, p.io_dtype,
                           p.residual_dtype) == bytes(p)
