"""Pins of the reference of the residual add between norms and of the gated feed-forward product (CPU): finite
differences of every gradient, and the properties that define them."""
import math

import numpy as np
import pytest

import oracle.tail as ot
from test_oracle_block import fd


@pytest.mark.parametrize("how", ot.ACTS)
def test_activations(how):
    v = np.concatenate([np.linspace(-9, 9, 401), [-40.0, 40.0]])
    if how != "relu":
        assert np.allclose((ot.act(v + 1e-6, how) - ot.act(v - 1e-6, how)) / 2e-6, ot.slope(v, how), atol=1e-8)
    limit = 1.0 if how == "sigmoid" else 40.0
    assert abs(ot.act(40.0, how) - limit) < 1e-9 and abs(ot.act(-40.0, how)) < 1e-9
    assert ot.act(0.0, how) == (0.5 if how == "sigmoid" else 0.0)
    assert ot.slope(0.0, how) == {"sigmoid": 0.25, "relu": 0.0}.get(how, 0.5)
    # values known in closed form: sigmoid(ln 3) = 3/4, Phi(sqrt 2 erfinv) through erf(1)
    if how in ("sigmoid", "silu"):
        assert abs(ot.act(math.log(3.0), how) - (0.75 if how == "sigmoid" else 0.75 * math.log(3.0))) < 1e-15
    if how == "gelu":
        assert abs(ot.act(math.sqrt(2.0), how) - math.sqrt(2.0) * 0.5 * (1 + 0.8427007929497149)) < 1e-15
    if how == "gelu_tanh":
        assert np.abs(ot.act(v, how) - ot.act(v, "gelu")).max() < 5e-4   # it approximates gelu


@pytest.mark.parametrize("how", ot.ACTS)
def test_glu_gradients(how):
    r = np.random.default_rng(3)
    x, wg, wu = r.standard_normal((4, 5)), r.standard_normal((6, 5)), r.standard_normal((6, 5))
    bg, bu, dh = r.standard_normal(6), r.standard_normal(6), r.standard_normal((4, 6))
    args = [x, wg, wu, bg, bu]
    grads = ot.glu_bwd(dh, *args, how)
    for i, g in enumerate(grads):
        fn = lambda v: ot.glu(*args[:i], v, *args[i + 1:], how)[0]
        assert np.allclose(fd(fn, args[i], dh), g, atol=1e-7), i
    assert np.allclose(ot.glu(x, wg, wu, None, None, how)[0], ot.glu(x, wg, wu, 0 * bg, 0 * bu, how)[0])


@pytest.mark.parametrize("norm", ["none", "layer", "rms"])
@pytest.mark.parametrize("post", ["none", "layer", "rms"])
@pytest.mark.parametrize("groups", [1, 3])
def test_addnorm_gradients(norm, post, groups):
    r = np.random.default_rng(4)
    rows, C = 6, 5
    N = lambda *s: r.standard_normal(s)
    v = dict(x=N(rows, C), y=N(rows, C), gate=N(groups, C))
    if norm != "none":
        v.update(w=N(groups, C), b=N(groups, C))
    if post != "none":
        v.update(post_w=N(C), post_b=N(C))
    how = dict(norm=norm, post=post, scale=0.7, residual=1.3, eps=1e-3)
    dh, ds = N(rows, C), N(rows, C)
    f = ot.addnorm(**v, **how)

    def loss(out):
        return out["s"] * ds + (0.0 if norm == "none" else out["h"] * dh)

    del how["eps"]
    stats = {k: f[k] for k in ("mean", "rstd", "post_mean", "post_rstd")}
    g = ot.addnorm_bwd(dh, ds, f["s"], v["y"], **{k: v[k] for k in ("w", "b", "gate", "post_w", "post_b") if k in v}, **how, **stats)
    how["eps"] = 1e-3
    for name in v:
        fn = lambda t: loss(ot.addnorm(**{**v, name: t}, **how))
        assert np.allclose(fd(fn, v[name], np.ones((rows, C))), g["d" + name], atol=1e-6), name


def test_addnorm_norms():
    r = np.random.default_rng(5)
    x, y = r.standard_normal((7, 64)), 3 + 2 * r.standard_normal((7, 64))
    f = ot.addnorm(x, y, norm="layer", post="rms", eps=0.0)
    z = f["s"] - x
    assert np.allclose((z ** 2).mean(-1), 1) and np.allclose(z / y, (z / y)[:, :1])
    assert np.allclose(f["h"].mean(-1), 0) and np.allclose((f["h"] ** 2).mean(-1), 1)
    plain = ot.addnorm(x, y, norm="none", scale=0.5, residual=2.0)
    assert np.allclose(plain["s"], 2 * x + 0.5 * y) and plain["h"] is None
    gate = r.standard_normal((7, 64))
    assert np.allclose(ot.addnorm(x, y, gate=gate, norm="none")["s"], x + gate * y)
