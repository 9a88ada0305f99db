"""Argument checks of the C entry points of the gated recurrence, of activations in 8 bits
and of the layer norm, without a GPU: fake addresses, never dereferenced."""
import ctypes

import pytest

from selective_state_space_sscan_amd import sscan
from test_delta_abi_cpu import EALIAS, EALIGN, ENULL, ESHAPE, EUNSUP, EWS, OK, Fake, lib  # noqa: F401

I2 = ctypes.c_int64 * 2
B, L, D = 2, 100, 96
KEPT = ("kx", "kg", "ki", "kz", "sx", "sg", "si", "sz")


def rec(b=B, L=L, d=D, io=1, **over):
    f, e = Fake(), 2 if io == 1 else 4
    n = b * L * d
    st = I2(L * d, d)
    a = dict(x=f(n * e), g=f(n * e), i=f(n * e), z=f(n * e), lam=f(d * 4), lengths=f(b * 4), h0=f(b * d * 4), x_stride=st,
             g_stride=st, i_stride=st, z_stride=st, batch=b, len=L, dim=d, c=8.0, reverse=0, io_dtype=io)
    rest = dict(out=f(n * e), last=f(b * d * 4), ws=f(1 << 34), ws_bytes=1 << 34, dout=f(n * e), dh=f(b * d * 4),
                dx=f(n * e), dg=f(n * e), di=f(n * e), dz=f(n * e), dlam=f(d * 4), dh0=f(b * d * 4))
    rest.update((k, f(n if k[0] == "k" else 4 * n)) for k in KEPT)
    for key, v in over.items():
        assert key in a or key in rest
        (a if key in a else rest)[key] = v
    return sscan.RecParams(**a), rest


def kept_of(r):
    return sscan.RecKept(*(r[k] for k in KEPT))


def fwd(lib, kept=False, **over):  # noqa: F811
    p, r = rec(**over)
    k = ctypes.byref(kept_of(r)) if kept else None
    return lib.sscan_validate_rec_fwd(ctypes.byref(p), r["out"], r["last"], k, r["ws"], r["ws_bytes"])


def bwd(lib, kept=False, **over):  # noqa: F811
    p, r = rec(**(dict(x=None, g=None, i=None, z=None, **over) if kept else over))
    g = sscan.RecGrads(*(r[k] for k in ("dx", "dg", "di", "dz", "dlam", "dh0")))
    k = ctypes.byref(kept_of(r)) if kept else None
    return lib.sscan_validate_rec_bwd(ctypes.byref(p), k, r["dout"], r["dh"], ctypes.byref(g), r["ws"], r["ws_bytes"])


BOTH = [
    (dict(), OK), (dict(lengths=None, h0=None), OK), (dict(io=0), OK), (dict(reverse=1), OK), (dict(x=None), ENULL),
    (dict(g=None), ENULL), (dict(batch=-1), ESHAPE), (dict(len=-1), ESHAPE), (dict(dim=-1), ESHAPE),
    (dict(len=(1 << 30) + 1), ESHAPE), (dict(dim=(1 << 24) + 1), ESHAPE), (dict(batch=1 << 40, len=1), ESHAPE),
    (dict(batch=1 << 25, len=1, dim=1), ESHAPE), (dict(io_dtype=7), EUNSUP), (dict(reverse=2), EUNSUP),
    (dict(c=float("nan")), EUNSUP), (dict(c=float("inf")), EUNSUP), (dict(c=-1.0), EUNSUP),
    (dict(x=(1 << 40) + 1), EALIGN), (dict(lam=(1 << 40) + 2), EALIGN), (dict(h0=(1 << 41) + 2), EALIGN),
    (dict(batch=1 << 22, len=1, dim=64), ESHAPE), (dict(b=(1 << 22) - 1, L=1, d=1), OK),
    (dict(z_stride=I2(0, 1 << 26)), EUNSUP), (dict(z=1 << 50, z_stride=I2(0, (1 << 26) - 1)), OK),
    (dict(L=1, len=1, z_stride=I2(0, 1 << 40)), OK),
    (dict(lengths=(1 << 41) + 2), EALIGN), (dict(x_stride=I2(-1, 96)), ESHAPE), (dict(z_stride=I2(1 << 60, 96)), ESHAPE),
]


@pytest.mark.parametrize("over,status", BOTH)
def test_validate(lib, over, status):  # noqa: F811
    assert fwd(lib, **over) == status
    assert bwd(lib, **over) == status


def test_validate_workspace(lib):  # noqa: F811
    for back, call in ((0, fwd), (1, bwd)):
        f = lib.sscan_rec_bwd_workspace_bytes if back else lib.sscan_rec_workspace_bytes
        n = f(8, 5000, 96, 1)
        many = dict(b=8, L=5000)
        assert call(lib, ws_bytes=n, **many) == OK
        if n:
            assert call(lib, ws_bytes=n - 1, **many) == EWS and call(lib, ws=None, **many) == EWS
            assert call(lib, ws=(1 << 50) + 16, **many) == EALIGN
        assert f(-1, 5, 5, 1) == f(1, 5, 5, 9) == f(0, 5, 5, 1) == f(5, 5, 0, 1) == f(1 << 40, 5, 5, 1) == 0


def test_validate_outputs(lib):  # noqa: F811
    p, r = rec()
    assert fwd(lib, out=None) == ENULL and fwd(lib, last=None) == ENULL
    assert fwd(lib, last=p.h0) == OK  # the state in place
    assert fwd(lib, last=p.h0 + 4) == EALIAS and fwd(lib, last=p.lam) == EALIAS
    for at in (p.x, p.z + 64, p.lam, p.h0, p.lengths, r["last"]):
        assert fwd(lib, out=at) == EALIAS
    assert fwd(lib, out=p.x + 1) == EALIGN and fwd(lib, last=p.h0 + 2) == EALIGN
    assert bwd(lib, dout=None) == ENULL and bwd(lib, dx=None) == ENULL and bwd(lib, di=None) == ENULL
    assert bwd(lib, dz=None) == ENULL and bwd(lib, dlam=None, dh0=None, dh=None) == OK
    assert bwd(lib, lam=None) == ENULL and bwd(lib, lam=None, dlam=None) == OK
    assert bwd(lib, i=None) == EUNSUP and bwd(lib, i=None, di=None) == OK and bwd(lib, z=None, dz=None) == OK
    for at in (p.x, r["dg"], r["dout"], p.lam, r["dh"]):
        assert bwd(lib, dx=at) == EALIAS
    assert bwd(lib, dh0=r["dh"]) == EALIAS and bwd(lib, dlam=r["dh0"]) == EALIAS
    assert lib.sscan_validate_rec_fwd(None, 0, 0, None, 0, 0) == ENULL
    assert lib.sscan_validate_rec_bwd(ctypes.byref(p), None, r["dout"], None, None, r["ws"], 1 << 34) == ENULL


def test_validate_kept(lib):  # noqa: F811
    p, r = rec()
    assert fwd(lib, kept=True) == OK and bwd(lib, kept=True) == OK
    for name in KEPT:
        assert fwd(lib, kept=True, **{name: None}) == ENULL
        assert fwd(lib, kept=True, **{name: r["out"]}) == EALIAS
        assert bwd(lib, kept=True, **{name: r["dx"]}) == EALIAS
    assert fwd(lib, kept=True, kx=r["kg"]) == EALIAS and fwd(lib, kept=True, sg=p.lam) == EALIAS
    assert fwd(lib, kept=True, sx=r["sx"] + 2) == EALIGN
    assert fwd(lib, kept=True, i=None) == EUNSUP and fwd(lib, kept=True, i=None, ki=None, si=None) == OK
    assert bwd(lib, kept=True, kx=None) == ENULL and bwd(lib, kept=True, sz=None) == ENULL
    assert bwd(lib, kept=True, kz=None, sz=None) == EUNSUP  # dz without a z
    assert bwd(lib, kept=True, kz=None, sz=None, dz=None) == OK
    g = sscan.RecGrads(*(r[k] for k in ("dx", "dg", "di", "dz", "dlam", "dh0")))
    assert lib.sscan_validate_rec_bwd(ctypes.byref(p), ctypes.byref(kept_of(r)), r["dout"], None, ctypes.byref(g),
                                      r["ws"], 1 << 34) == EUNSUP  # the inputs twice


def test_validate_empty(lib):  # noqa: F811
    none = dict(x=None, g=None, i=None, z=None, out=None, dout=None, dx=None, dg=None, di=None, dz=None)
    assert fwd(lib, b=0, last=None, h0=None, ws=None, **none) == OK
    assert fwd(lib, d=0, last=None, h0=None, ws=None, **none) == OK
    assert fwd(lib, L=0, **none) == OK and fwd(lib, L=0, last=None, **none) == ENULL
    for size in (dict(b=0), dict(L=0), dict(d=0)):
        assert bwd(lib, **size, **none) == OK


def test_validate_step(lib):  # noqa: F811
    def step(state=None, out=None, **over):
        p, r = rec(**dict(dict(L=1, h0=None), **over))
        return lib.sscan_validate_rec_step(ctypes.byref(p), state or r["last"], out or r["out"])

    assert step() == OK and step(b=0) == OK
    assert step(L=2) == ESHAPE and step(reverse=1) == EUNSUP and step(h0=1 << 44) == EUNSUP
    assert step(state=(1 << 50) + 2) == EALIGN and step(x=None) == ENULL
    p, r = rec(L=1, h0=None)
    for state, out in ((p.x, r["out"]), (r["last"], p.g), (r["last"], r["last"])):
        assert lib.sscan_validate_rec_step(ctypes.byref(p), state, out) == EALIAS
    assert lib.sscan_validate_rec_step(ctypes.byref(p), None, r["out"]) == ENULL
    assert lib.sscan_validate_rec_step(None, 0, 0) == ENULL


def test_validate_pack8(lib):  # noqa: F811
    f = Fake()
    x, q, s = f(4 * 5 * 130), f(5 * 130), f(4 * 5 * 3)

    def pack(x=x, stride=130, rows=5, size=130, io=0, q=q, s=s):
        return lib.sscan_validate_pack8(x, stride, rows, size, io, q, s)

    def unpack(q=q, s=s, rows=5, size=130, io=0, out=x):
        return lib.sscan_validate_unpack8(q, s, rows, size, io, out)

    for call in (pack, unpack):
        assert call() == OK and call(io=1) == OK and call(rows=0, q=None, s=None) == OK and call(size=0, q=None) == OK
        assert call(rows=-1) == ESHAPE and call(size=-1) == ESHAPE and call(rows=1 << 40, size=1 << 40) == ESHAPE
        assert call(io=2) == EUNSUP and call(q=None) == ENULL and call(s=None) == ENULL
        assert call(q=x + 4) == EALIAS and call(s=x) == EALIAS and call(s=s + 2) == EALIGN
    assert pack(x=None) == ENULL and pack(x=x + 2) == EALIGN and pack(stride=0) == OK and pack(stride=-1) == ESHAPE
    assert pack(stride=1 << 60) == ESHAPE and pack(s=q) == EALIAS and unpack(out=None) == ENULL
    assert unpack(out=x + 2) == EALIGN


def layer(n=10, size=96, io=1, res=0, **over):
    f, e, r = Fake(), 2 if io == 1 else 4, 2 if res == 1 else 4
    a = dict(x=f(n * size * 4), residual=f(n * size * r), weight=f(size * 4), bias=f(size * 4), x_stride=size, rows=n,
             size=size, eps=1e-5, io_dtype=io, residual_dtype=res)
    rest = dict(out=f(n * size * e), total=f(n * size * r), dout=f(n * size * e), dtotal=f(n * size * r),
                dx=f(n * size * e), dres=f(n * size * r), dw=f(size * 4), db=f(size * 4), ws=f(1 << 30), ws_bytes=1 << 30)
    for key, v in over.items():
        (a if key in a else rest)[key] = v
    return sscan.LayerNormParams(**a), rest


def lfwd(lib, **over):  # noqa: F811
    p, r = layer(**over)
    return lib.sscan_validate_layer_norm(ctypes.byref(p), r["out"], r["total"])


def lbwd(lib, **over):  # noqa: F811
    p, r = layer(**over)
    return lib.sscan_validate_layer_norm_bwd(ctypes.byref(p), *(r[k] for k in ("dout", "dtotal", "dx", "dres", "dw", "db",
                                                                               "ws", "ws_bytes")))


@pytest.mark.parametrize("over,status", [
    (dict(), OK), (dict(weight=None, bias=None, dw=None, db=None), OK), (dict(x=None), ENULL), (dict(rows=-1), ESHAPE),
    (dict(size=0), EUNSUP), (dict(size=8193), EUNSUP), (dict(eps=-1.0), EUNSUP), (dict(eps=float("nan")), EUNSUP),
    (dict(io_dtype=3), EUNSUP), (dict(residual_dtype=3), EUNSUP), (dict(x=(1 << 40) + 1), EALIGN),
    (dict(weight=(1 << 40) + 2), EALIGN), (dict(x_stride=-1), ESHAPE), (dict(x_stride=1 << 60), ESHAPE),
    (dict(x_stride=0), OK), (dict(rows=0, x=None), OK), (dict(rows=1 << 45, size=64), ESHAPE)])
def test_validate_layer_norm(lib, over, status):  # noqa: F811
    assert lfwd(lib, **over) == status
    assert lbwd(lib, **over) == status


def test_validate_layer_norm_outputs(lib):  # noqa: F811
    p, r = layer()
    assert lfwd(lib, out=None) == ENULL and lfwd(lib, total=None) == ENULL and lfwd(lib, total=None, residual=None) == OK
    assert lfwd(lib, residual=None) == OK and lfwd(lib, total=p.residual) == OK
    assert lfwd(lib, total=p.residual + 4) == EALIAS
    for at in (p.x, p.residual, p.weight, p.bias, r["total"]):
        assert lfwd(lib, out=at) == EALIAS
    assert lbwd(lib, dout=None) == ENULL and lbwd(lib, dx=None) == ENULL and lbwd(lib, dtotal=None, dres=None) == OK
    assert lbwd(lib, weight=None) == ENULL and lbwd(lib, bias=None) == ENULL
    assert lbwd(lib, dres=r["dtotal"]) == OK and lbwd(lib, dx=r["dtotal"]) == EALIAS
    for at in (p.x, r["dout"], p.weight, r["dres"], r["dw"]):
        assert lbwd(lib, dx=at) == EALIAS
    assert lbwd(lib, ws=None) == EWS and lbwd(lib, ws_bytes=8) == EWS and lbwd(lib, ws=(1 << 50) + 4) == EALIGN
    assert lib.sscan_validate_layer_norm(None, 0, 0) == ENULL
    for n, size in ((0, 5), (5, 0), (5, 8193), (-1, 5)):
        assert lib.sscan_layer_norm_bwd_workspace_bytes(n, size) == 0


def test_validate_workspace_apart_from_inputs(lib):  # noqa: F811
    """A workspace over an input would be emptied before the input is read."""
    many = dict(b=8, L=5000)
    p, r = rec(**many)
    for call in (fwd, bwd):
        for at in (p.x, p.g, p.i, p.z, p.lam, p.lengths, p.h0):
            assert call(lib, ws=at, **many) == EALIAS
        assert call(lib, **many) == OK
    n = lib.sscan_rec_workspace_bytes(8, 5000, D, 1)
    assert fwd(lib, ws=p.x - n, **many) == OK and fwd(lib, ws=p.x - n + 256, **many) == EALIAS
    for at in (r["dout"], r["dh"]):
        assert bwd(lib, ws=at, **many) == EALIAS
    p, r = rec()
    for name in KEPT:
        assert bwd(lib, kept=True, ws=r[name]) == EALIAS
    p, r = layer(n=3000)
    for at in (p.x, p.weight, p.bias, r["dout"], r["dtotal"]):
        assert lbwd(lib, n=3000, ws=at) == EALIAS
