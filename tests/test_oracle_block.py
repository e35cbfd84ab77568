"""Pins of the reference of the operators around the attention (CPU): known answers of the generator, finite
differences of every gradient, and the properties that define the rotation and the norm."""
import math

import numpy as np
import pytest

import oracle.block as ob


def test_generator_known_answers():
    """The published known answers of Philox4x32 at seven and at ten rounds."""
    f = 0xFFFFFFFF
    z, o = [[0, 0, 0, 0]], [[f, f, f, f]]
    assert [hex(int(v)) for v in ob.philox(z, (0, 0), 7)[0]] == ["0x5f6fb709", "0xd893f64", "0x4f121f81", "0x4f730a48"]
    assert [hex(int(v)) for v in ob.philox(o, (f, f), 7)[0]] == ["0x5207ddc2", "0x45165e59", "0x4d8ee751", "0x8c52f662"]
    assert [hex(int(v)) for v in ob.philox(z, (0, 0), 10)[0]] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]
    pi = [[0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344]]
    assert [hex(int(v)) for v in ob.philox(pi, (0xA4093822, 0x299F31D0), 10)[0]] == [
        "0xd16cfe09", "0x94fdcceb", "0x5001e420", "0x24126ea1"]


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9, 1.0])
def test_dropout_factor_keeps_the_mean(p):
    n = 200_000
    f = ob.dropout_factor(n, p, 1234567890123, 42)
    assert set(np.unique(f == 0)) <= {True, False}
    zero = float((f == 0).mean())
    assert abs(zero - p) < 6 * math.sqrt(max(p * (1 - p), 1e-12) / n) + 2.0 ** -17
    if p < 1:
        assert abs(f.max() * (1 - p) - 1) < 2.0 ** -16 / (1 - p)
    assert np.array_equal(f[:1001], ob.dropout_factor(1001, p, 1234567890123, 42))


def test_dropout_depends_on_seed_offset_and_place():
    a = ob.dropout_factor(4096, 0.5, 1, 2)
    for other in (ob.dropout_factor(4096, 0.5, 2, 2), ob.dropout_factor(4096, 0.5, 1, 3),
                  ob.dropout_factor(4096, 0.5, 1 + (1 << 32), 2), ob.dropout_factor(4096, 0.5, 1, 2 + (1 << 32))):
        assert 0.4 < float((a == other).mean()) < 0.6
    assert 0.4 < float((a[8:] == a[:-8]).mean()) < 0.6


def fd(fn, x, dy, h=1e-6):
    """Central differences of <dy, fn(x)> along every element of x."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        g[i] = ((fn(up) - fn(down)) * dy).sum() / (2 * h)
    return g


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_turns_pairs_and_its_gradient_turns_back(layout):
    r = np.random.default_rng(1)
    x = r.standard_normal((2, 3, 4, 2, 16))
    freqs = [[1.0, 0.3, 0.01], [0.7, 0.05]]
    y = ob.rope(x, freqs, [5, -2], 1.3, layout)
    assert np.array_equal(y[..., 10:], x[..., 10:])                       # channels past the blocks
    assert np.allclose((y[..., :10] ** 2).sum(-1), 1.69 * (x[..., :10] ** 2).sum(-1))
    # a complex number per pair, turned by position times frequency
    lo, hi = (0, 3) if layout == "half" else (0, 1)
    z = (x[1, 2, 3, 1, lo] + 1j * x[1, 2, 3, 1, hi]) * 1.3 * np.exp(1j * 7 * 1.0)
    assert np.allclose([y[1, 2, 3, 1, lo], y[1, 2, 3, 1, hi]], [z.real, z.imag])
    # products of rotated q and k depend on the positions' difference alone
    q, k = r.standard_normal((1, 6, 1, 16)), r.standard_normal((1, 6, 1, 16))
    q[:], k[:] = q[:, :1], k[:, :1]
    a, b = ob.rope(q, [[0.9, 0.2]], [0], 1.0, layout), ob.rope(k, [[0.9, 0.2]], [11], 1.0, layout)
    dots = (a[0, :, 0, None] * b[0, None, :, 0]).sum(-1)
    assert np.allclose(dots[1:, 1:], dots[:-1, :-1])
    dy = r.standard_normal(x.shape)
    back = ob.rope(dy, freqs, [5, -2], 1.3, layout, inverse=True)
    assert np.allclose((back * x).sum(), (dy * y).sum())                  # adjoint


def test_layernorm_against_differences():
    r = np.random.default_rng(2)
    x, w, b = r.standard_normal((3, 7)) + 2, r.standard_normal(7), r.standard_normal(7)
    dy = r.standard_normal(x.shape)
    y, mean, rstd = ob.layernorm(x, w, b, 1e-3)
    h = (y - b) / w
    assert np.allclose(h.mean(-1), 0) and np.allclose((h * h).mean(-1), 1 - 1e-3 * rstd ** 2)
    dx, dw, db = ob.layernorm_bwd(dy, x, w, mean, rstd)
    assert np.allclose(dx, fd(lambda t: ob.layernorm(t, w, b, 1e-3)[0], x, dy), atol=1e-7)
    assert np.allclose(dw, fd(lambda t: ob.layernorm(x, t, b, 1e-3)[0], w, dy), atol=1e-7)
    assert np.allclose(db, fd(lambda t: ob.layernorm(x, w, t, 1e-3)[0], b, dy), atol=1e-7)


@pytest.mark.parametrize("per_row", [False, True])
def test_window_softmax_gradients_against_differences(per_row):
    r = np.random.default_rng(3)
    shape = (1, 2, 2, 5)
    x1, x2, dy = (r.standard_normal(shape) for _ in range(3))
    x1[0, 0, 1, 3:] = -np.inf
    x2[0, 1, 0] = -np.inf                                                 # an empty row
    lam = r.standard_normal(shape[:-1] if per_row else (2,))
    f = ob.dropout_factor(x1.size, 0.4, 9, 9).reshape(shape)
    dx1, dx2, dlam = ob.diff_softmax_bwd(x1, x2, lam, dy, f)
    with np.errstate(invalid="ignore"):
        n1 = fd(lambda t: ob.diff_softmax(t, x2, lam, f), x1, dy)
        n2 = fd(lambda t: ob.diff_softmax(x1, t, lam, f), x2, dy)
    assert np.allclose(dx1, n1, atol=1e-7) and np.allclose(dx2, n2, atol=1e-7)
    assert np.allclose(dlam, fd(lambda t: ob.diff_softmax(x1, x2, t, f), lam, dy), atol=1e-7)
    assert np.array_equal(ob.diff_softmax(x1, x2, 0 * lam, f), ob.softmax_dropout(x1, f))
    assert np.array_equal(dx2[0, 1, 0], np.zeros(5)) and np.array_equal(dx1[0, 0, 1, 3:], np.zeros(2))


def test_softmax_of_masked_rows():
    low = float(np.finfo(np.float32).min)
    x = np.array([[low, low, low], [low, 0.0, low], [-np.inf, 1.0, -np.inf], [-np.inf] * 3])
    s = ob.softmax(x)
    assert np.allclose(s, [[1 / 3] * 3, [0, 1, 0], [0, 1, 0], [0, 0, 0]])
