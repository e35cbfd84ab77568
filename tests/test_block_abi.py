"""Host-side checks (CPU) of the operators around the attention: bad arguments are refused before anything is
launched, with the status that include/na.h gives, and the binding's own checks raise.  Only calls that
fail validation are made: a valid one would launch a kernel."""
import ctypes
import math

import pytest
import torch

import neighborhood_attention_fwd_gb300 as na
from neighborhood_attention_fwd_gb300 import build as nabuild

INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 6
BF16, FP32, FP16 = 0, 1, 2
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    nabuild.build()
    return na.load()


def P(x):
    return ctypes.c_void_p(x) if x is not None else None


def I(v):
    return (ctypes.c_int * len(v))(*v)


def rope(lib, q=1 * MB, k=2 * MB, qo=3 * MB, ko=4 * MB, B=1, spatial=(4, 4), hq=2, hk=2, D=32, rot=(16, 16), freq=0.5,
         origin=None, amp=1.0, layout=0, dtype=BF16, bwd=False):
    f = (ctypes.c_double * 64)(*([freq] * 64))
    call = lib.na_rope_bwd if bwd else lib.na_rope
    return call(P(q), P(k), P(qo), P(ko), B, len(spatial), I(spatial), hq, hk, D, I(rot), f, origin, amp, layout, dtype, None)


@pytest.mark.parametrize("bwd", [False, True])
def test_rope_refusals(lib, bwd):
    call = lambda **kw: rope(lib, bwd=bwd, **kw)
    for kw in (dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(hk=0), dict(hk=-1), dict(B=0), dict(hq=0),
               dict(spatial=(0, 4)), dict(rot=(15, 16)), dict(rot=(18, 16)), dict(rot=(-2, 16)), dict(rot=(0, 0)),
               dict(freq=math.nan), dict(freq=math.inf), dict(freq=1e7), dict(amp=math.nan), dict(layout=2), dict(dtype=9),
               dict(spatial=(1, 1, 1, 1), rot=(4, 4, 4, 4)),
               dict(qo=2 * MB),                   # q_out over k
               dict(qo=1 * MB + 64),              # q_out over a part of q
               dict(ko=3 * MB), dict(ko=1 * MB)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(D=48, rot=(8, 8)), dict(D=256, rot=(8, 8)), dict(spatial=(1 << 16, 1 << 16)),
               dict(B=1 << 20, spatial=(1 << 10, 1 << 10))):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(q=MB + 8), dict(k=2 * MB + 4), dict(qo=3 * MB + 2), dict(ko=4 * MB + 8)):
        assert call(**kw) == ALIGNMENT, kw


def norm(lib, x=1 * MB, w=2 * MB, b=3 * MB, y=4 * MB, mean=5 * MB, rstd=6 * MB, rows=8, C=32, eps=1e-5, dtype=BF16):
    return lib.na_layernorm(P(x), P(w), P(b), P(y), P(mean), P(rstd), rows, C, eps, dtype, None)


def norm_bwd(lib, dy=1 * MB, x=2 * MB, w=3 * MB, mean=4 * MB, rstd=5 * MB, dx=6 * MB, dw=7 * MB, db=8 * MB, rows=8, C=32,
             dtype=BF16, ws=9 * MB, nbytes=MB):
    return lib.na_layernorm_bwd(P(dy), P(x), P(w), P(mean), P(rstd), P(dx), P(dw), P(db), rows, C, dtype, P(ws), nbytes, None)


def test_layernorm_refusals(lib):
    for kw in (dict(x=None), dict(y=None), dict(mean=None), dict(rstd=None), dict(rows=0), dict(rows=-1), dict(C=0),
               dict(eps=-1.0), dict(eps=math.nan), dict(dtype=5), dict(y=MB + 16), dict(y=2 * MB), dict(mean=1 * MB),
               dict(mean=6 * MB), dict(rstd=4 * MB)):
        assert norm(lib, **kw) == INVALID, kw
    assert norm(lib, C=8193) == UNSUPPORTED
    assert norm(lib, rows=1 << 40, C=8) == UNSUPPORTED
    for kw in (dict(x=MB + 8), dict(w=2 * MB + 4), dict(b=3 * MB + 8), dict(y=4 * MB + 2), dict(mean=5 * MB + 2)):
        assert norm(lib, **kw) == ALIGNMENT, kw


def test_layernorm_bwd_refusals(lib):
    for kw in (dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(dx=None), dict(dw=None), dict(db=None),
               dict(rows=0), dict(C=0), dict(dtype=3), dict(dx=2 * MB + 16), dict(dw=8 * MB), dict(dw=6 * MB),
               dict(db=1 * MB), dict(dx=4 * MB), dict(ws=6 * MB)):
        assert norm_bwd(lib, **kw) == INVALID, kw
    assert norm_bwd(lib, C=8200) == UNSUPPORTED
    for kw in (dict(dx=6 * MB + 8), dict(dw=7 * MB + 1), dict(ws=9 * MB + 4)):
        assert norm_bwd(lib, **kw) == ALIGNMENT, kw
    need = na.na_layernorm_bwd_workspace_size(8, 32)
    assert need > 0 and norm_bwd(lib, nbytes=need - 1) == WORKSPACE
    assert na.na_layernorm_bwd_workspace_size(0, 32) == 0
    assert na.na_layernorm_bwd_workspace_size(8, 9000) == 0


def test_dropout_refusals(lib):
    call = lambda x=MB, y=2 * MB, n=64, p=0.1, rng=3 * MB, dtype=BF16: lib.na_dropout(P(x), P(y), n, p, P(rng), dtype, None)
    for kw in (dict(x=None), dict(y=None), dict(n=0), dict(n=-5), dict(p=-0.1), dict(p=1.1), dict(p=math.nan),
               dict(rng=None), dict(dtype=4), dict(y=MB + 16), dict(rng=2 * MB)):
        assert call(**kw) == INVALID, kw
    assert call(n=(1 << 40) + 1) == UNSUPPORTED
    for kw in (dict(x=MB + 2), dict(y=2 * MB + 4), dict(rng=3 * MB + 4)):
        assert call(**kw) == ALIGNMENT, kw


def soft(lib, x=1 * MB, y=2 * MB, B=1, spatial=(8, 8), heads=2, kernel=(3, 3), p=0.1, rng=9 * MB, dtype=BF16, dy=None):
    head = (P(x), P(y)) if dy is None else (P(x), P(dy), P(y))
    call = lib.na_softmax_dropout if dy is None else lib.na_softmax_dropout_bwd
    return call(*head, B, len(spatial), I(spatial), heads, I(kernel), p, P(rng), dtype, None)


@pytest.mark.parametrize("dy", [None, 3 * MB])
def test_softmax_dropout_refusals(lib, dy):
    call = lambda **kw: soft(lib, **{"dy": dy, **kw})
    for kw in (dict(x=None), dict(y=None), dict(B=0), dict(heads=0), dict(kernel=(3, 4)), dict(kernel=(3, 9)),
               dict(kernel=(0, 3)), dict(p=2.0), dict(rng=None), dict(dtype=8), dict(y=MB + 32), dict(rng=2 * MB)):
        assert call(**kw) == INVALID, kw
    assert call(B=1 << 20, spatial=(1 << 10, 1 << 10)) == UNSUPPORTED
    assert call(x=MB + 2) == ALIGNMENT
    assert call(rng=9 * MB + 4) == ALIGNMENT


def diff(lib, x1=1 * MB, x2=2 * MB, lam=3 * MB, rows=0, y=4 * MB, B=1, spatial=(8, 8), heads=2, kernel=(3, 3), p=0.0,
         rng=None, dtype=BF16):
    return lib.na_diff_softmax(P(x1), P(x2), P(lam), rows, P(y), B, len(spatial), I(spatial), heads, I(kernel), p, P(rng), dtype,
                               None)


def diff_bwd(lib, x1=1 * MB, x2=2 * MB, lam=3 * MB, rows=0, dy=4 * MB, dx1=5 * MB, dx2=6 * MB, dlam=7 * MB, B=1,
             spatial=(8, 8), heads=2, kernel=(3, 3), p=0.0, rng=None, dtype=BF16, ws=8 * MB, nbytes=MB):
    return lib.na_diff_softmax_bwd(P(x1), P(x2), P(lam), rows, P(dy), P(dx1), P(dx2), P(dlam), B, len(spatial), I(spatial),
                                   heads, I(kernel), p, P(rng), dtype, P(ws), nbytes, None)


def test_diff_softmax_refusals(lib):
    for kw in (dict(x1=None), dict(x2=None), dict(lam=None), dict(y=None), dict(rows=2), dict(p=0.1), dict(kernel=(2, 3)),
               dict(y=3 * MB), dict(y=2 * MB + 16), dict(dtype=3)):
        assert diff(lib, **kw) == INVALID, kw
    for kw in (dict(x2=2 * MB + 4), dict(lam=3 * MB + 2)):
        assert diff(lib, **kw) == ALIGNMENT, kw
    for kw in (dict(dx1=None), dict(dx2=None), dict(dlam=None), dict(dy=None), dict(dx2=5 * MB), dict(dlam=5 * MB),
               dict(dlam=3 * MB), dict(dx1=1 * MB + 16), dict(ws=5 * MB)):
        assert diff_bwd(lib, **kw) == INVALID, kw
    need = na.na_diff_softmax_bwd_workspace_size(1, (8, 8), 2, (3, 3))
    assert need >= 8 * 8 * 2 * 4 and diff_bwd(lib, nbytes=need - 1) == WORKSPACE
    assert diff_bwd(lib, ws=8 * MB + 8) == ALIGNMENT
    assert diff_bwd(lib, dlam=7 * MB + 2) == ALIGNMENT
    assert na.na_diff_softmax_bwd_workspace_size(1, (8, 8), 2, (3, 4)) == 0


def test_binding_checks():
    q = torch.zeros(1, 4, 4, 2, 32)
    f = na.RopeFreqs.scaled((16, 16))
    with pytest.raises(ValueError):
        na.na_rope(q, None, q, None, f)                                   # not on a CUDA device
    with pytest.raises(ValueError):
        na.RopeFreqs([[1.0]], layout="other")
    with pytest.raises(ValueError):
        na.RopeFreqs.scaled((15,))
    with pytest.raises(ValueError):
        na.RopeFreqs.scaled((16,), scaling="yarn", factor=4.0)            # no trained length
    with pytest.raises(ValueError):
        na.RopeFreqs.scaled((16,), scaling="other")


def test_tensors_of_another_device_are_refused(monkeypatch):
    """A tensor of a device other than the current one, or of two devices, raises before the library is called."""
    class Fake:
        def __init__(self, at):
            self.at, self.device = at, f"cuda:{at}"

        def get_device(self):
            return self.at

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda at: 77 + at, raising=False)
    assert na._launch_stream(None, Fake(0), None, Fake(0)) == 77
    for tensors in ((Fake(1),), (Fake(0), Fake(1)), (Fake(0), Fake(-1))):
        with pytest.raises(ValueError):
            na._launch_stream(None, *tensors)


def test_scaled_frequencies():
    plain = na.RopeFreqs.scaled((32, 8)).freqs
    assert plain[0][0] == 1.0 and len(plain[0]) == 16 and len(plain[1]) == 4
    assert plain[0][8] == pytest.approx(0.01)
    lin = na.RopeFreqs.scaled((32,), scaling="linear", factor=4.0).freqs[0]
    assert all(a == pytest.approx(b / 4) for a, b in zip(lin, plain[0]))
    ntk = na.RopeFreqs.scaled((32,), scaling="ntk", factor=4.0).freqs[0]
    assert ntk[0] == 1.0 and ntk[-1] == pytest.approx(plain[0][-1] / 4)
    y = na.RopeFreqs.scaled((32,), scaling="yarn", factor=4.0, trained=4096)
    assert y.amplitude == pytest.approx(0.1 * math.log(4) + 1)
    assert y.freqs[0][0] == 1.0 and y.freqs[0][-1] == pytest.approx(plain[0][-1] / 4)
    turns = [4096 * v / (2 * math.pi) for v in plain[0]]
    for v, base, t in zip(y.freqs[0], plain[0], turns):
        if t > 32:
            assert v == base
        elif t < 1:
            assert v == pytest.approx(base / 4)
        else:
            assert base / 4 < v < base
