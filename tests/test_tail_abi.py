"""Host-side checks (CPU) of the residual add between norms and of the gated feed-forward product: bad arguments are
refused before anything is launched, with the status that include/na.h gives, and the binding's own checks raise.  Only
calls that fail validation are made: a valid one would launch a kernel."""
import ctypes
import math

import pytest
import torch

import neighborhood_attention_fwd_gb300 as na
from neighborhood_attention_fwd_gb300 import build as nabuild

INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 6
BF16, FP32, FP16 = 0, 1, 2
NONE, LAYER, RMS = 0, 1, 2
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    nabuild.build()
    return na.load()


def P(x):
    return ctypes.c_void_p(x * MB if isinstance(x, int) else int(x)) if x is not None else None


def at(mb, more):
    return float(mb * MB + more)   # a place inside a megabyte


def add(lib, x=1, y=2, s=3, h=4, w=5, b=6, gate=7, pw=8, pb=9, mean=10, rstd=11, pmean=12, prstd=13, rows=8, C=32, wg=1, gg=1,
        norm=LAYER, post=LAYER, scale=1.0, residual=1.0, eps=1e-5, dtype=BF16):
    return lib.na_addnorm(*map(P, (x, y, s, h, w, b, gate, pw, pb, mean, rstd, pmean, prstd)), rows, C, wg, gg, norm, post, scale, residual,
                          eps, dtype, None)


def test_addnorm_refusals(lib):
    for kw in (dict(x=None), dict(y=None), dict(h=None), dict(s=None, h=None), dict(rows=0), dict(rows=-1), dict(C=0), dict(wg=0),
               dict(gg=-1), dict(wg=3), dict(gg=3), dict(wg=2, gg=4), dict(norm=3), dict(post=-1), dict(scale=math.nan),
               dict(residual=math.inf), dict(eps=-1.0), dict(eps=math.nan), dict(dtype=5),
               dict(norm=NONE), dict(norm=NONE, h=None), dict(norm=NONE, h=None, w=None, b=None),   # statistics left
               dict(post=NONE), dict(post=NONE, pmean=None, prstd=None),                              # weights left
               dict(mean=None), dict(rstd=None), dict(pmean=None), dict(prstd=None), dict(norm=RMS), dict(post=RMS),
               dict(w=None, b=None, wg=2), dict(gate=None, gg=2),
               dict(s=4), dict(s=at(1, 16)), dict(h=at(2, 16)), dict(s=5), dict(h=7), dict(s=10), dict(mean=11), dict(mean=1),
               dict(rstd=13), dict(pmean=8), dict(prstd=2), dict(h=9)):
        assert add(lib, **kw) == INVALID, kw
    for kw in (dict(C=8193), dict(rows=1 << 38), dict(rows=1 << 17, wg=1 << 17), dict(rows=65536, gg=65536)):
        assert add(lib, **kw) == UNSUPPORTED, kw
    for name in ("x", "y", "s", "h", "w", "b", "gate", "pw", "pb"):
        assert add(lib, **{name: at(20, 8)}) == ALIGNMENT, name
    for name in ("mean", "rstd", "pmean", "prstd"):
        assert add(lib, **{name: at(20, 2)}) == ALIGNMENT, name


def add_bwd(lib, dh=1, ds=2, s=3, y=4, w=5, gate=6, pw=7, pb=8, mean=9, rstd=10, pmean=11, prstd=12, dx=13, dy=14, dw=15, db=16, dgate=17,
            dpw=18, dpb=19, rows=8, C=32, wg=1, gg=1, norm=LAYER, post=LAYER, scale=1.0, residual=1.0, dtype=BF16, ws=20, nbytes=MB):
    return lib.na_addnorm_bwd(*map(P, (dh, ds, s, y, w, gate, pw, pb, mean, rstd, pmean, prstd, dx, dy, dw, db, dgate, dpw, dpb)), rows, C, wg,
                              gg, norm, post, scale, residual, dtype, P(ws), nbytes, None)


def test_addnorm_bwd_refusals(lib):
    for kw in (dict(dh=None), dict(s=None), dict(y=None), dict(dx=None), dict(dy=None), dict(mean=None), dict(rstd=None), dict(pmean=None),
               dict(prstd=None), dict(rows=0), dict(C=-1), dict(rows=9, wg=2), dict(wg=4, gg=2), dict(norm=NONE), dict(post=NONE), dict(norm=RMS),
               dict(post=RMS), dict(scale=math.inf), dict(gate=None), dict(dtype=-1),
               dict(norm=NONE, dh=None, s=None, ds=None, w=None, dw=None, db=None, mean=None, rstd=None),
               dict(norm=NONE, dh=None, s=None, w=None, dw=None, mean=None, rstd=None),
               dict(post=NONE, pw=None, pb=None, pmean=None, prstd=None),
               dict(dx=4), dict(dx=14), dict(dy=13), dict(dx=at(1, 16)), dict(dy=at(4, 32)), dict(dx=5), dict(dy=12), dict(dw=16), dict(dw=5),
               dict(dgate=6), dict(dpw=13), dict(dpb=3), dict(db=10), dict(ws=13), dict(ws=15), dict(ws=6), dict(ws=4)):
        assert add_bwd(lib, **kw) == INVALID, kw
    assert add_bwd(lib, C=10000) == UNSUPPORTED
    assert add_bwd(lib, rows=1 << 40) == UNSUPPORTED
    for name in ("dh", "ds", "s", "y", "w", "gate", "pw", "pb", "dx", "dy", "ws"):
        assert add_bwd(lib, **{name: at(30, 8)}) == ALIGNMENT, name
    for name in ("mean", "rstd", "pmean", "prstd", "dw", "db", "dgate", "dpw", "dpb"):
        assert add_bwd(lib, **{name: at(30, 1)}) == ALIGNMENT, name
    need = lib.na_addnorm_bwd_workspace_size(8, 32, 1, 1, BF16)
    assert need > 0 and add_bwd(lib, nbytes=need - 1) == WORKSPACE
    for bad in ((0, 32, 1, 1, 0), (8, 0, 1, 1, 0), (8, 32, 3, 1, 0), (8, 32, 1, 0, 0), (8, 32, 1, 1, 7), (8, 8193, 1, 1, 0)):
        assert lib.na_addnorm_bwd_workspace_size(*bad) == 0, bad


def glu(lib, x=1, wg=2, wu=3, bg=4, bu=5, h=6, rows=8, D=32, F=16, act=0, dtype=BF16):
    return lib.na_glu(*map(P, (x, wg, wu, bg, bu, h)), rows, D, F, act, dtype, None)


def test_glu_refusals(lib):
    for kw in (dict(x=None), dict(wg=None), dict(wu=None), dict(h=None), dict(rows=0), dict(D=0), dict(F=-1), dict(act=5), dict(act=-1),
               dict(dtype=4), dict(h=1), dict(h=at(2, 16)), dict(h=3), dict(h=4), dict(h=5)):
        assert glu(lib, **kw) == INVALID, kw
    for kw in (dict(D=(1 << 20) + 1), dict(F=(1 << 20) + 1), dict(rows=1 << 31), dict(rows=1 << 30, D=1 << 14), dict(rows=1 << 30, F=1 << 14)):
        assert glu(lib, **kw) == UNSUPPORTED, kw
    for name in ("x", "wg", "wu", "bg", "bu", "h"):
        assert glu(lib, **{name: at(20, 8)}) == ALIGNMENT, name


def glu_bwd(lib, dh=1, x=2, wg=3, wu=4, bg=5, bu=6, dx=7, dwg=8, dwu=9, dbg=10, dbu=11, rows=8, D=32, F=16, act=0, dtype=BF16, ws=12, nbytes=MB):
    return lib.na_glu_bwd(*map(P, (dh, x, wg, wu, bg, bu, dx, dwg, dwu, dbg, dbu)), rows, D, F, act, dtype, P(ws), nbytes, None)


def test_glu_bwd_refusals(lib):
    for kw in (dict(dh=None), dict(x=None), dict(wg=None), dict(wu=None), dict(dwg=None), dict(dwu=None), dict(bg=None), dict(bu=None),
               dict(dx=None, dwg=None, dwu=None, dbg=None, dbu=None), dict(rows=0), dict(D=0), dict(F=0), dict(act=9), dict(dtype=3),
               dict(dx=2), dict(dx=1), dict(dwg=3), dict(dwg=9), dict(dwu=at(7, 16)), dict(dbg=11), dict(dbu=6), dict(ws=1), dict(ws=8), dict(ws=11)):
        assert glu_bwd(lib, **kw) == INVALID, kw
    assert glu_bwd(lib, F=1 << 21) == UNSUPPORTED
    for name in ("dh", "x", "wg", "wu", "bg", "bu", "dx", "dwg", "dwu", "dbg", "dbu", "ws"):
        assert glu_bwd(lib, **{name: at(30, 8)}) == ALIGNMENT, name
    need = lib.na_glu_bwd_workspace_size(8, 32, 16, BF16)
    assert need >= 2 * 8 * 16 * 2 and glu_bwd(lib, nbytes=need - 1) == WORKSPACE
    assert lib.na_glu_bwd_workspace_size(0, 32, 16, BF16) == 0 and lib.na_glu_bwd_workspace_size(8, 32, 16, 9) == 0


def test_binding_refusals(lib):
    """The binding's checks come before the library: wrong shapes, types and combinations raise on CPU tensors too."""
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)
    f = lambda *s: torch.zeros(s)
    x = z(2, 6, 32)
    n = dict(norm="layer")
    for call in (
        lambda: na.na_addnorm(x, z(2, 6, 31), x, x, **n),
        lambda: na.na_addnorm(x, f(2, 6, 32), x, x, **n),
        lambda: na.na_addnorm(x, x, x, None, **n),
        lambda: na.na_addnorm(x, x, None, None, norm="none"),
        lambda: na.na_addnorm(x, x, x, x, norm="batch"),
        lambda: na.na_addnorm(x, x, x, x, post="group"),
        lambda: na.na_addnorm(x, x, x, x, gate=z(32)),                 # not fp32
        lambda: na.na_addnorm(x, x, x, x, gate=f(3, 32)),              # no leading axes of x
        lambda: na.na_addnorm(x, x, x, x, gate=f(6, 32)),
        lambda: na.na_addnorm(x, x, x, x, w=f(2, 32), b=f(32)),
        lambda: na.na_addnorm(x, x, x, x, gate=f(2, 6, 32, 32)),
        lambda: na.na_addnorm(x, x, x, x, gate=f(32, 2).t()),          # not contiguous
        lambda: na.na_addnorm(x, x, x, x, post_w=f(32)),               # no post norm
        lambda: na.na_addnorm(x, x, x, x, post="rms", post_w=f(2, 32)),
        lambda: na.na_addnorm(x, x, x, x, mean=f(2, 6)),
        lambda: na.na_addnorm(x, x, x, x, norm="rms", mean=f(2, 6), rstd=f(2, 6)),
        lambda: na.na_addnorm(x, x, x, x, post_rstd=f(2, 6)),
        lambda: na.na_addnorm(x, x, x, x, mean=f(12), rstd=f(12)),
        lambda: na.na_addnorm(x, x, x, x),                             # CPU tensors
        lambda: na.na_addnorm_bwd(x, x, x, x, x, x),                   # no statistics
        lambda: na.na_addnorm_bwd(None, x, x, x, x, x, mean=f(2, 6), rstd=f(2, 6)),
        lambda: na.na_addnorm_bwd(None, None, None, x, x, x, norm="none"),
        lambda: na.na_addnorm_bwd(x, x, x, x, x, x, mean=f(2, 6), rstd=f(2, 6), dgate=f(32)),
        lambda: na.na_addnorm_bwd(x, x, x, x, x, x, mean=f(2, 6), rstd=f(2, 6), w=f(32), dw=f(2, 32)),
        lambda: na.na_addnorm_bwd(x, x, x, x, x, x, mean=f(2, 6), rstd=f(2, 6), dpost_w=f(32)),
        lambda: na.na_addnorm_bwd(x, x, x, x, x, x, mean=f(2, 6), rstd=f(2, 6)),
    ):
        with pytest.raises((ValueError, TypeError)):
            call()
    w, h = z(16, 32), z(2, 6, 16)
    for call in (
        lambda: na.na_glu(x, w, z(17, 32), h), lambda: na.na_glu(x, z(16, 31), w, h), lambda: na.na_glu(x, w, w, z(2, 6, 15)),
        lambda: na.na_glu(x, w, w, f(2, 6, 16)), lambda: na.na_glu(x, z(32, 16).t(), w, h), lambda: na.na_glu(x, z(0, 32), z(0, 32), z(2, 6, 0)),
        lambda: na.na_glu(x, w, w, h, bg=f(16)), lambda: na.na_glu(x, w, w, h, bu=z(32)), lambda: na.na_glu(x, w, w, h, act="tanh"),
        lambda: na.na_glu(x, z(16), w, h), lambda: na.na_glu(x, w, w, h),
        lambda: na.na_glu_bwd(h, x, w, w), lambda: na.na_glu_bwd(h, x, w, w, x, w), lambda: na.na_glu_bwd(h, x, w, w, x, dbg=z(16)),
        lambda: na.na_glu_bwd(h, x, w, w, z(2, 6, 31)), lambda: na.na_glu_bwd(h, x, w, w, None, w, z(16, 31)),
        lambda: na.na_glu_bwd(h, x, w, w, x),
    ):
        with pytest.raises((ValueError, TypeError)):
            call()
