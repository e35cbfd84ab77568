"""GPU tests of the operators around the attention against the fp64 reference, element by element.

Tolerances.  Every bound below is derived from the arithmetic the kernels do in fp32, e = 2^-24 being half a step of
fp32, and one rounding to the tensors' type at the end, u = finfo(type).eps / 2 relative to the value, plus
half the smallest subnormal.  A sum of n terms in a tree or in a thread's run of d terms is off by at most
d e times the sum of the terms' sizes, d its longest path; DEPTH = 64 covers every row's sum here (at most 33
words or elements per thread, then five to ten tree steps).  An approximate exponential is off by 2 steps.
"""
import math

import numpy as np
import pytest
import torch

import oracle.block as ob
import oracle.unfused as un
from neighborhood_attention_fwd_gb300 import inputs as nain

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E = 2.0 ** -24
DEPTH = 64


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(TYPES[dtype])


def close(name, got, ref, slack, dtype=torch.float32):
    """|got - ref| <= u (|ref| + slack) + slack + half the type's smallest step, element by element."""
    info = torch.finfo(dtype)
    ref = np.asarray(ref, dtype=np.float64)
    got = f64(got)
    assert got.shape == ref.shape, f"{name}: {got.shape} against {ref.shape}"
    bound = info.eps / 2 * (np.abs(ref) + slack) + slack + info.smallest_normal * info.eps / 2
    off = np.abs(got - ref)
    bad = ~(off <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(np.isnan(off), np.inf, off / bound)), off.shape)
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} outside, worst at {i}: got {got[i]!r}, want {ref[i]!r}, "
                             f"bound {np.broadcast_to(bound, off.shape)[i]:.3e}")


def status_ok(na):
    st, raw = na.na_device_status()
    assert st == 0, f"device status {st} raw {raw:#x}"


# ---------------------------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------------------------

ROPE = [
    # dtype, B, grid, heads_q, heads_k, D, rot, layout, origin
    ("fp32", 1, (16, 16), 2, 2, 16, (8, 8), "half", None),
    ("bf16", 2, (13, 18), 2, 2, 32, (16, 16), "half", None),
    ("bf16", 2, (13, 18), 2, 2, 32, (16, 16), "interleaved", None),
    ("fp16", 1, (1001,), 4, 1, 128, (64,), "interleaved", (1_000_000,)),
    ("fp16", 1, (1001,), 4, 1, 128, (64,), "half", (1 << 40,)),
    ("bf16", 1, (5, 7, 9), 3, 3, 64, (32, 16, 16), "half", (-3, 100, 7)),
    ("bf16", 1, (5, 7, 9), 3, 0, 64, (20, 22, 22), "half", None),           # halves that are not whole chunks
    ("fp32", 2, (6, 11), 5, 2, 128, (6, 10), "half", (2, 9)),
    ("fp16", 1, (9, 10), 3, 5, 16, (2, 6), "half", None),
    ("bf16", 1, (9, 10), 3, 5, 16, (2, 6), "interleaved", None),            # a chunk turned in part
    ("fp32", 1, (1,), 1, 0, 16, (2,), "interleaved", (3,)),                 # one token
    ("bf16", 1, (1,), 1, 1, 16, (16,), "half", None),
    ("bf16", 1, (3, 4), 2, 2, 32, (0, 32), "half", (5, 5)),                 # an axis without channels
    ("bf16", 1, (70, 33), 16, 16, 128, (64, 64), "half", None),             # several passes per block
    ("fp32", 1, (40, 33), 16, 7, 128, (64, 62), "interleaved", None),
    ("bf16", 1, (9, 31), 3, 2, 32, (8, 12), "half", None),                  # even halves, some channels copied
    ("fp16", 2, (5, 7, 9), 2, 5, 64, (20, 20, 24), "half", (1, 2, 3)),
    ("bf16", 1, (300,), 40, 1, 128, (44,), "half", None),                   # several turns of a block
    ("fp16", 1, (300,), 40, 3, 128, (46,), "half", None),
]


def rope_case(case):
    dtype, B, grid, hq, hk, D, rot, layout, origin = case
    q = randn((B, *grid, hq, D), dtype, 1)
    k = randn((B, *grid, hk, D), dtype, 2) if hk else None
    return q, k


def rope_slack(x, amp, pairs_of):
    # cos and sin: phase cut at 2^-32 turns and rounded to fp32 (2^-25 half turns), two steps of sincospi; amplitude,
    # two products and a sum: 8 e of |u| + |v|
    return 8 * E * amp * pairs_of(np.abs(f64(x)))


@pytest.mark.parametrize("case", ROPE, ids=[str(c) for c in ROPE])
def test_rope_and_its_gradient(case, cuda_lib):
    na = cuda_lib
    dtype, B, grid, hq, hk, D, rot, layout, origin = case
    q, k = rope_case(case)
    freqs = na.RopeFreqs.scaled(rot, scaling="yarn", factor=4.0, trained=2048, layout=layout)
    org = [0] * len(grid) if origin is None else list(origin)

    def partner_sum(a):   # |u| + |v| at both places of every pair
        s, base = a.copy(), 0
        for r in rot:
            i = np.arange(r // 2)
            lo, hi = (base + i, base + r // 2 + i) if layout == "half" else (base + 2 * i, base + 2 * i + 1)
            t = a[..., lo] + a[..., hi]
            s[..., lo], s[..., hi] = t, t
            base += r
        s[..., base:] = 0
        return s

    for call, inverse in ((na.na_rope, False), (na.na_rope_bwd, True)):
        qd, kd = q.cuda(), None if k is None else k.cuda()
        qo, ko = torch.full_like(qd, 7.0), None if k is None else torch.full_like(kd, 7.0)
        call(qd, kd, qo, ko, freqs, origin=origin)
        status_ok(na)
        for name, x, y in (("q", q, qo), ("k", k, ko)):
            if x is None:
                continue
            ref = rope_exact(f64(x), freqs, org, inverse)
            close(name, y, ref, rope_slack(x, freqs.amplitude, partner_sum), TYPES[dtype])
            assert torch.equal(y[..., sum(rot):].cpu(), x[..., sum(rot):])          # channels past the blocks: copied
        call(qd, kd, qd, kd, freqs, origin=origin)                                    # in place
        assert torch.equal(qd, qo) and (k is None or torch.equal(kd, ko))


def rope_exact(x, freqs, origin, inverse):
    """The reference, with the angles of far positions reduced in exact integers (the product of a position above
    2^20 and a frequency keeps too few digits of the angle in fp64)."""
    from fractions import Fraction

    two_pi = Fraction(2 * 314159265358979323846264338327950288419716939937510, 10 ** 50)
    if max(abs(o) for o in origin) < 1 << 12:
        return ob.rope(x, freqs.freqs, origin, freqs.amplitude, freqs.layout, inverse)
    n = x.ndim - 3
    y, base = x.copy(), 0
    for a in range(n):
        f = freqs.freqs[a]
        half = len(f)
        theta = np.array([[float((Fraction(origin[a] + i) * Fraction(v)) % two_pi) for v in f] for i in range(x.shape[1 + a])])
        theta = -theta if inverse else theta
        shape = [1] * x.ndim
        shape[1 + a], shape[-1] = x.shape[1 + a], half
        c, s = np.cos(theta).reshape(shape), np.sin(theta).reshape(shape)
        i = np.arange(half)
        lo, hi = (base + i, base + half + i) if freqs.layout == "half" else (base + 2 * i, base + 2 * i + 1)
        u, v = x[..., lo], x[..., hi]
        y[..., lo], y[..., hi] = freqs.amplitude * (u * c - v * s), freqs.amplitude * (u * s + v * c)
        base += 2 * half
    return y


def test_rope_leaves_unturned_channels_alone(cuda_lib):
    """Infinities and NaN in channels past the blocks do not reach the others, and are copied as they are."""
    na = cuda_lib
    for rot, layout in (((6, 4), "half"), ((8, 8), "half"), ((6, 4), "interleaved")):
        q = randn((1, 3, 5, 2, 32), "bf16", 5)
        q[..., sum(rot)::2] = float("inf")
        q[..., sum(rot) + 1::2] = float("nan")
        out = torch.empty_like(q).cuda()
        na.na_rope(q.cuda(), None, out, None, na.RopeFreqs.scaled(rot, layout=layout))
        status_ok(na)
        out = out.cpu()
        assert torch.isfinite(out[..., :sum(rot)].float()).all()
        assert torch.equal(out[..., sum(rot):].view(torch.int16), q[..., sum(rot):].view(torch.int16))


# ---------------------------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------------------------

NORM = [
    # dtype, rows, C
    ("bf16", 1, 1), ("fp32", 3, 1), ("bf16", 700, 16), ("fp16", 333, 32), ("fp32", 333, 32), ("bf16", 1, 64), ("bf16", 77, 128),
    ("fp32", 77, 128), ("bf16", 1000, 256), ("bf16", 101, 264), ("fp16", 65, 512), ("bf16", 33, 520), ("fp32", 21, 768),
    ("bf16", 17, 1024), ("fp16", 17, 1032), ("fp32", 333, 2048), ("bf16", 1300, 2048), ("bf16", 5, 8192), ("fp32", 5, 8192),
    ("bf16", 19, 7), ("fp16", 130, 33), ("fp32", 57, 63), ("bf16", 57, 65), ("fp32", 13, 129), ("bf16", 9, 1001), ("fp32", 9, 4099),
    ("fp16", 3, 8191), ("bf16", 40000, 24),
    # wide rows around the fewest that take the gradients' general kernels
    ("bf16", 1536, 264), ("bf16", 1537, 264), ("fp32", 1536, 296), ("fp32", 1100, 4096), ("fp32", 1, 8192), ("fp16", 65, 4104), ("fp32", 63, 4100),
]


@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("case", NORM, ids=[str(c) for c in NORM])
def test_layernorm_and_its_gradients(case, affine, cuda_lib):
    na = cuda_lib
    dtype, rows, C = case
    x = (randn((rows, C), "fp32", 1) * 1.5 + randn((rows, 1), "fp32", 2)).to(TYPES[dtype])
    w = 1 + 0.3 * randn((C,), "fp32", 3) if affine else None
    b = randn((C,), "fp32", 4) if affine else None
    dy = randn((rows, C), dtype, 5)
    dev = lambda t: None if t is None else t.cuda()
    xd, wd, bd, dyd = dev(x), dev(w), dev(b), dev(dy)
    y, mean, rstd = torch.empty_like(xd), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    na.na_layernorm(xd, wd, bd, y, mean, rstd, eps=1e-5)
    status_ok(na)
    X = f64(x)
    ry, rm, rr = ob.layernorm(X, None if w is None else f64(w), None if b is None else f64(b), float(np.float32(1e-5)))
    em = DEPTH * E * np.abs(X).mean(-1)                       # the mean
    er = (DEPTH + 8) * E + (em * rr) ** 2                     # rstd, relative: half the variance's
    close("mean", mean, rm, em)
    close("rstd", rstd, rr, rr * er)
    h = (X - rm[:, None]) * rr[:, None]
    W = np.ones(C) if w is None else np.abs(f64(w))
    Bv = np.zeros(C) if b is None else np.abs(f64(b))
    close("y", y, ry, W * (rr * em)[:, None] + np.abs(h) * W * (er[:, None] + 8 * E) + 2 * E * Bv, TYPES[dtype])
    # the gradients at the statistics that the library saved
    dx, dw, db = torch.empty_like(xd), torch.full((C,), 9.0, device="cuda"), torch.full((C,), 9.0, device="cuda")
    na.na_layernorm_bwd(dyd, xd, wd, mean, rstd, dx, dw, db)
    status_ok(na)
    m, r = f64(mean)[:, None], f64(rstd)[:, None]
    rdx, rdw, rdb = ob.layernorm_bwd(f64(dy), X, None if w is None else f64(w), f64(mean), f64(rstd))
    h, g = (X - m) * r, f64(dy) * (1 if w is None else f64(w))
    c1, c2 = np.abs(g.mean(-1, keepdims=True)), np.abs((g * h).mean(-1, keepdims=True))
    slack = r * E * (8 * (np.abs(g) + c1 + np.abs(h) * c2) + (DEPTH + 8) * (
        np.abs(g).mean(-1, keepdims=True) + np.abs(h) * np.abs(g * h).mean(-1, keepdims=True)))
    close("dx", dx, rdx, slack, TYPES[dtype])
    # a column's sum: a thread's run of rows (at most rows / 8 here), shuffles, warps, blocks
    path = rows / 8 + 150
    close("dw", dw, rdw, path * E * np.abs(f64(dy) * h).sum(0))
    close("db", db, rdb, path * E * np.abs(f64(dy)).sum(0))
    # in place, with a workspace, without the weights' gradients: the same values
    ws = torch.empty(na.na_layernorm_bwd_workspace_size(rows, C, TYPES[dtype]), dtype=torch.uint8, device="cuda")
    dw2, db2, dx2 = torch.empty_like(dw), torch.empty_like(db), dyd.clone()
    na.na_layernorm_bwd(dx2, xd, wd, mean, rstd, dx2, dw2, db2, workspace=ws)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
    na.na_layernorm_bwd(dyd, xd, wd, mean, rstd, dx2)
    assert torch.equal(dx2, dx)
    y2 = xd.clone()
    na.na_layernorm(y2, wd, bd, y2)
    assert torch.equal(y2, y)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_layernorm_gradients_of_few_wide_rows_over_their_inputs(dtype, cuda_lib):
    """Few wide rows need no workspace; dx over x or dy gives what a separate dx gives, also without dw and db, and in a
    captured graph."""
    na = cuda_lib
    for rows, C in ((1, 520), (130, 2048), (500, 6000)):
        x, dy = randn((rows, C), dtype, 1).cuda(), randn((rows, C), dtype, 2).cuda()
        w = torch.rand(C, device="cuda")
        y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        na.na_layernorm(x, w, None, y, mean, rstd)
        assert na.na_layernorm_bwd_workspace_size(rows, C, TYPES[dtype]) == 0

        def grads(over=None, sums=True):
            a, b = x.clone(), dy.clone()
            dx = {None: torch.empty_like(x), "x": a, "dy": b}[over]
            dw, db = (torch.full((C,), 9.0, device="cuda") for _ in range(2))
            na.na_layernorm_bwd(b, a, w, mean, rstd, dx, *((dw, db) if sums else ()))
            return (dx, dw, db) if sums else (dx,)

        ref = grads()
        for over in ("x", "dy"):
            assert all(torch.equal(g, r) for g, r in zip(grads(over), ref))
            assert torch.equal(grads(over, False)[0], ref[0])
        assert torch.equal(grads(None, False)[0], ref[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = grads("x")
        for t in out:
            t.zero_()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
    status_ok(na)


def test_layernorm_keeps_its_digits_far_from_zero(cuda_lib):
    """A mean a thousand times the spread, rows of one value, and zeros."""
    na = cuda_lib
    x = (randn((64, 256), "fp32", 7) + 1000.0).cuda()
    x[5] = 3.25
    x[6] = 0.0
    y, mean, rstd = torch.empty_like(x), torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    na.na_layernorm(x, None, None, y, mean, rstd)
    status_ok(na)
    X = f64(x)
    ry, rm, rr = ob.layernorm(X, None, None, float(np.float32(1e-5)))
    em = DEPTH * E * np.abs(X).mean(-1)
    close("mean", mean, rm, em)
    er = (DEPTH + 8) * E + (em * rr) ** 2
    close("y", y, ry, (rr * em)[:, None] + np.abs(ry) * (er[:, None] + 8 * E))
    assert torch.equal(y[6], torch.zeros(256, device="cuda"))


# ---------------------------------------------------------------------------------------------
# Dropout, the window softmax with dropout, the differential softmax
# ---------------------------------------------------------------------------------------------

SEED, OFFSET = 0x1234_5678_9ABC_DEF1, 0x0FED_CBA9_8765_4321


def rng_state():
    return torch.tensor([SEED, OFFSET], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 1000, 8192 * 3 + 5, 1 << 20])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout(dtype, n, p, cuda_lib):
    na = cuda_lib
    x = randn((n,), dtype, 11)
    y = torch.full_like(x, 3.0).cuda()
    na.na_dropout(x.cuda(), y, p, rng_state())
    status_ok(na)
    f = ob.dropout_factor(n, p, SEED, OFFSET)
    ref = f64(x) * f
    close("y", y, ref, 2 * E * np.abs(ref), TYPES[dtype])
    assert np.array_equal(f64(y) == 0, (f == 0) | (f64(x) == 0))
    z = x.cuda()
    na.na_dropout(z, z, p, rng_state())
    assert torch.equal(z, y)
    if p == 0.0:
        na.na_dropout(x.cuda(), y, p, None)
        assert torch.equal(y.cpu(), x)


def factor_at(first, n, p):
    """dropout_factor's values of elements first .. first + n - 1 (first a multiple of 8)."""
    i = np.arange(first // 8, (first + n + 7) // 8, dtype=np.uint64)
    low, shift = np.uint64(0xFFFFFFFF), np.uint64(32)
    full = lambda v: np.full(len(i), v, np.uint64)
    words = ob.philox(np.stack([i & low, i >> shift, full(OFFSET & 0xFFFFFFFF), full(OFFSET >> 32)], 1),
                      (SEED & 0xFFFFFFFF, SEED >> 32), 7)
    fields = np.empty((len(i), 8), dtype=np.uint64)
    fields[:, 0::2], fields[:, 1::2] = words & np.uint64(0xFFFF), words >> np.uint64(16)
    steps = int(math.floor((1 - p) * 65536 + 0.5))
    return np.where(fields.reshape(-1)[:n] < steps, 65536.0 / steps, 0.0)


@pytest.mark.slow
@pytest.mark.parametrize("n", [(1 << 32) + 1003, (1 << 35) + 12347])
def test_dropout_past_32_bits(n, cuda_lib):
    """Element indices past 2^32, and generator blocks past 2^32, in place."""
    na = cuda_lib
    if torch.cuda.mem_get_info()[0] < 2 * n + (8 << 30):
        pytest.skip("not enough free device memory")
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    na.na_dropout(x, x, 0.3, rng_state())
    status_ok(na)
    for at in (0, (1 << 32) - 64, (n - 4096) // 8 * 8):
        got = x[at:at + 4096]
        ref = factor_at(at, got.numel(), 0.3)
        close("y", got, ref, 2 * E * ref, torch.bfloat16)
        assert np.array_equal(f64(got) == 0, ref == 0)


@pytest.mark.slow
def test_rows_past_32_bits(cuda_lib):
    """Weights and channels at offsets past 2^32 elements: the first rows, those around the border and the last ones."""
    na = cuda_lib
    K, heads = 81, 8
    L = (1 << 32) // (K * heads) + 1001
    rows = (0, (1 << 32) // (K * heads) - 1, L - 3)
    x = torch.full((1, L, heads, K), 0.5, dtype=torch.bfloat16, device="cuda")
    for r in rows:
        x[0, r:r + 3].normal_()
    before = [f64(x[0, r:r + 3]) for r in rows]
    na.na_softmax_dropout(x, x, (K,), 0.3, rng_state())
    status_ok(na)
    for r, b in zip(rows, before):
        first = r * heads * K // 8 * 8
        f = factor_at(first, 3 * heads * K + 8, 0.3)[r * heads * K - first:][:3 * heads * K].reshape(3, heads, K)
        s = ob.softmax(b)
        ref = ob.softmax_dropout(b, f)
        close("y", x[0, r:r + 3], ref, np.abs(ref) * map_error(b, s), torch.bfloat16)
    C = 256
    x = x.view(-1)[:(1 << 32) + 3 * C].view(-1, C)
    n = x.shape[0]
    x.normal_()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd, db, dw = (torch.empty(m, device="cuda") for m in (n, n, C, C))
    na.na_layernorm(x, None, None, y, mean, rstd)
    na.na_layernorm_bwd(y, x, None, mean, rstd, dx, dw, db)
    status_ok(na)
    for r in (0, (1 << 32) // C - 1, n - 3):
        X = f64(x[r:r + 3])
        ry, _, rr = ob.layernorm(X, None, None, float(np.float32(1e-5)))
        slack = 2 * DEPTH * E * (1 + np.abs(ry)) * (1 + rr[:, None])
        close("y", y[r:r + 3], ry, slack, torch.bfloat16)
        dy = f64(y[r:r + 3])
        rdx = ob.layernorm_bwd(dy, X, None, f64(mean[r:r + 3]), f64(rstd[r:r + 3]))[0]
        close("dx", dx[r:r + 3], rdx, 4 * DEPTH * E * (1 + rr[:, None]) * (1 + np.abs(dy)) * (1 + np.abs(ry)), torch.bfloat16)


def test_dropout_drops_what_is_not_a_number(cuda_lib):
    na = cuda_lib
    x = torch.full((4096,), float("nan"), device="cuda")
    x[::2] = float("inf")
    y = torch.empty_like(x)
    na.na_dropout(x, y, 0.5, rng_state())
    f = torch.from_numpy(ob.dropout_factor(4096, 0.5, SEED, OFFSET)).cuda()
    assert torch.equal(y[f == 0], torch.zeros_like(y[f == 0])) and not torch.isfinite(y[f != 0]).any()


WIN = [
    # dtype, B, grid, heads, kernel
    ("fp32", 1, (16, 16), 2, (5, 5)), ("bf16", 2, (13, 18), 2, (5, 7)), ("fp16", 1, (6, 9, 10), 1, (3, 5, 5)),
    ("bf16", 1, (1,), 1, (1,)), ("bf16", 1, (3,), 1, (3,)), ("fp16", 1, (3, 3), 1, (3, 3)), ("fp32", 1, (3,), 3, (1,)),
    ("bf16", 1, (20, 24), 3, (9, 9)), ("fp32", 1, (20, 24), 3, (9, 9)), ("bf16", 1, (16, 15), 8, (13, 13)),
    ("fp16", 1, (8, 8, 9), 2, (5, 7, 7)), ("bf16", 1, (7, 8, 7), 1, (7, 7, 7)), ("fp16", 1, (40, 31), 5, (3, 3)),
    ("bf16", 1, (101,), 7, (5,)), ("bf16", 1, (37,), 3, (15,)), ("fp16", 1, (31,), 5, (23,)), ("bf16", 1, (9, 9, 9), 1, (9, 9, 9)),
    ("fp32", 1, (7, 7, 8), 1, (7, 7, 7)), ("bf16", 1, (767,), 1, (767,)), ("bf16", 1, (765,), 1, (765,)),
    ("bf16", 1, (1031,), 2, (1001,)), ("fp32", 1, (400,), 3, (399,)), ("fp32", 1, (383,), 1, (383,)), ("fp32", 1, (385,), 1, (385,)),
    ("fp16", 1, (5001,), 1, (4999,)), ("bf16", 3, (50, 41), 300, (1, 3)),
    ("fp32", 1, (9, 9, 9), 1, (9, 9, 9)), ("fp32", 1, (767,), 1, (767,)), ("fp32", 1, (770,), 1, (769,)),
    ("fp16", 1, (9, 41), 3, (9, 9)), ("fp32", 1, (45,), 5, (11,)), ("bf16", 1, (1200,), 2, (33,)), ("fp16", 1, (700,), 3, (121,)),
]
WIN_IDS = [str(c) for c in WIN]


def logits(shape, dtype, seed, masked):
    x = randn(shape, dtype, seed, 2.0)
    if masked:
        g = torch.Generator().manual_seed(seed + 100)
        x[torch.rand(shape, generator=g) < 0.3] = float("-inf")
        flat = x.view(-1, shape[-1])
        flat[::7] = float("-inf")                               # rows that the mask leaves empty
        flat[3::11, :] = torch.finfo(x.dtype).min               # rows masked by the lowest finite value
        flat[4::13, : (shape[-1] + 1) // 2] = torch.finfo(x.dtype).min
    return x


def map_error(x, s):
    """Relative error bound of a row's weights: an exponential's argument is off by e of its size (and the
    constant's half step), two steps of the exponential, the sum, the inverse and the products."""
    d = np.where(s > 0, np.abs(np.where(np.isneginf(x), 0, x) - np.max(np.where(np.isneginf(x), -np.inf, x), -1, keepdims=True,
                                                                       initial=-1e300)), 0.0)
    d = np.minimum(d, 200.0)
    return E * (2 * (d + (s * d).sum(-1, keepdims=True)) + DEPTH + 10)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("p", [0.0, 0.2])
@pytest.mark.parametrize("case", WIN, ids=WIN_IDS)
def test_softmax_dropout_and_its_gradient(case, p, masked, cuda_lib):
    na = cuda_lib
    dtype, B, grid, heads, kernel = case
    shape = (B, *grid, heads, math.prod(kernel))
    x, dy = logits(shape, dtype, 21, masked), randn(shape, dtype, 22)
    xd, dyd = x.cuda(), dy.cuda()
    y, dx = torch.full_like(xd, 5.0), torch.full_like(xd, 5.0)
    na.na_softmax_dropout(xd, y, kernel, p, rng_state())
    na.na_softmax_dropout_bwd(xd, dyd, dx, kernel, p, rng_state())
    status_ok(na)
    f = ob.dropout_factor(x.numel(), p, SEED, OFFSET).reshape(shape)
    X = f64(x)
    s = ob.softmax(X)
    es = map_error(X, s)
    ref = ob.softmax_dropout(X, f)
    close("y", y, ref, np.abs(ref) * es + 2.0 ** -120, TYPES[dtype])
    assert np.array_equal(f64(y) == 0, ref == 0) or dtype != "fp32" or np.abs(ref[(f64(y) == 0) & (ref != 0)]).max() < 2.0 ** -120
    slack, _ = grad_slack(s, es, f64(dy), f)
    close("dx", dx, ob.softmax_dropout_bwd(X, f64(dy), f), slack, TYPES[dtype])
    z = xd.clone()
    na.na_softmax_dropout(z, z, kernel, p, rng_state())
    assert torch.equal(z, y)
    a, b = xd.clone(), dyd.clone()
    na.na_softmax_dropout_bwd(a, dyd, a, kernel, p, rng_state())
    na.na_softmax_dropout_bwd(xd, b, b, kernel, p, rng_state())
    assert torch.equal(a, dx) and torch.equal(b, dx)
    status_ok(na)


def grad_slack(s, es, dy, f):
    """Error bounds of s (g - r) and of r = sum s g, g = f dy."""
    g = np.abs(np.where(s == 0, 0.0, dy * f))
    er = (s * g * (es + (DEPTH + 4) * E)).sum(-1, keepdims=True)
    r = (s * g).sum(-1, keepdims=True)
    return s * ((g + r) * (es + 8 * E) + er) + 2.0 ** -120, er[..., 0] + 4 * E * r[..., 0]


@pytest.mark.parametrize("lam_kind", ["head", "row"])
@pytest.mark.parametrize("p,masked", [(0.0, False), (0.0, True), (0.2, True)])
@pytest.mark.parametrize("case", WIN, ids=WIN_IDS)
def test_diff_softmax_and_its_gradients(case, p, masked, lam_kind, cuda_lib):
    na = cuda_lib
    dtype, B, grid, heads, kernel = case
    shape = (B, *grid, heads, math.prod(kernel))
    x1, x2, dy = logits(shape, dtype, 31, masked), logits(shape, dtype, 32, masked), randn(shape, dtype, 33)
    lam = randn(shape[:-1] if lam_kind == "row" else (heads,), "fp32", 34)
    d1, d2, dd, dl = x1.cuda(), x2.cuda(), dy.cuda(), lam.cuda()
    rng = rng_state() if p else None
    y, g1, g2, gl = torch.full_like(d1, 5.0), torch.full_like(d1, 5.0), torch.full_like(d1, 5.0), torch.full_like(dl, 5.0)
    na.na_diff_softmax(d1, d2, dl, y, kernel, p, rng)
    na.na_diff_softmax_bwd(d1, d2, dl, dd, g1, g2, gl, kernel, p, rng)
    status_ok(na)
    f = ob.dropout_factor(x1.numel(), p, SEED, OFFSET).reshape(shape)
    X1, X2, L, D = f64(x1), f64(x2), f64(lam), f64(dy)
    s1, s2 = ob.softmax(X1), ob.softmax(X2)
    e1, e2 = map_error(X1, s1), map_error(X2, s2)
    lr = np.abs(L)[..., None]
    close("y", y, ob.diff_softmax(X1, X2, L, f), f * (s1 * e1 + lr * s2 * (e2 + 4 * E)) + 2.0 ** -120, TYPES[dtype])
    r1, r2, rl = ob.diff_softmax_bwd(X1, X2, L, D, f)
    k1, _ = grad_slack(s1, e1, D, f)
    k2, row = grad_slack(s2, e2, D, f)
    close("dx1", g1, r1, k1, TYPES[dtype])
    close("dx2", g2, r2, lr * (k2 + 4 * E * np.abs(r2)), TYPES[dtype])
    if lam_kind == "row":
        close("dlam", gl, rl, row)
    else:   # rows' values summed: a thread's run of rows and a tree, at most rows / 8 + 300 long
        each = np.abs(np.where(s2 == 0, 0, s2 * D * f).sum(-1)).reshape(-1, heads).sum(0)
        close("dlam", gl, rl, row.reshape(-1, heads).sum(0) + (math.prod(shape[:-2]) / 8 + 300) * E * each)
    # a workspace of the caller's, and outputs over the inputs: the same values
    nbytes = na.na_diff_softmax_bwd_workspace_size(B, grid, heads, kernel)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    gl2, a1, a2, ad = torch.empty_like(gl), d1.clone(), d2.clone(), dd.clone()
    na.na_diff_softmax_bwd(a1, a2, dl, ad, ad, a1, gl2, kernel, p, rng, workspace=ws)
    assert torch.equal(ad, g1) and torch.equal(a1, g2) and torch.equal(gl2, gl)
    na.na_diff_softmax(d1, a2, dl, a2, kernel, p, rng)
    assert torch.equal(a2, y)
    status_ok(na)


def test_a_map_of_weight_zero_is_the_softmax(cuda_lib):
    """lam = 0 gives na_softmax_dropout's values, and without dropout na_softmax's to a rounding."""
    na = cuda_lib
    shape, kernel = (1, 9, 11, 4, 81), (9, 9)
    x1, x2 = randn(shape, "fp32", 1).cuda(), randn(shape, "fp32", 2).cuda()
    lam = torch.zeros(4, device="cuda")
    y, z, w = torch.empty_like(x1), torch.empty_like(x1), torch.empty_like(x1)
    na.na_diff_softmax(x1, x2, lam, y, kernel, 0.3, rng_state())
    na.na_softmax_dropout(x1, z, kernel, 0.3, rng_state())
    assert torch.equal(y, z)
    na.na_softmax_dropout(x1, z, kernel, 0.0, None)
    na.na_softmax(x1, w, kernel)
    assert torch.allclose(z, w, rtol=1e-6, atol=0)


@pytest.mark.parametrize("K", [5, 81, 1001])
def test_not_a_number_and_infinite_logits(K, cuda_lib):
    """A NaN or +inf makes its own row NaN and no other; dy at masked places takes no part."""
    na = cuda_lib
    x = randn((1, 1024, 1, K), "fp16", 3)
    x[0, 10, 0, 2] = float("nan")
    x[0, 20, 0, 1] = float("inf")
    x[0, 30, 0, :] = float("-inf")
    x[0, 30, 0, 3] = 1.0
    dy = randn(x.shape, "fp16", 4)
    dy[0, 30, 0, 0], dy[0, 30, 0, 1] = float("nan"), float("inf")
    xd = x.cuda()
    y, dx = torch.empty_like(xd), torch.empty_like(xd)
    kernel = (K,)
    na.na_softmax_dropout(xd, y, kernel, 0.0, None)
    na.na_softmax_dropout_bwd(xd, dy.cuda(), dx, kernel, 0.0, None)
    bad = torch.isnan(y).any(-1).flatten().nonzero().flatten().tolist()
    assert bad == [10, 20] and torch.isnan(y[0, 10]).all() and torch.isnan(y[0, 20]).all()
    assert torch.isnan(dx).any(-1).flatten().nonzero().flatten().tolist() == [10, 20]
    assert y[0, 30, 0, 3] == 1 and torch.equal(dx[0, 30], torch.zeros_like(dx[0, 30]))


# ---------------------------------------------------------------------------------------------
# Streams, graphs, devices, and the whole chain
# ---------------------------------------------------------------------------------------------

def test_on_another_stream(cuda_lib):
    na = cuda_lib
    s = torch.cuda.Stream()
    x = randn((1, 64, 64, 4, 81), "bf16", 1).cuda()
    rng, lam = rng_state(), torch.full((4,), 0.5, device="cuda")
    ref = torch.empty_like(x)
    na.na_diff_softmax(x, x, lam, ref, (9, 9), 0.1, rng)
    y, tmp = torch.empty_like(x), torch.empty_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        tmp.copy_(x)
        na.na_diff_softmax(tmp, x, lam, y, (9, 9), 0.1, rng)          # the current stream
    na.na_diff_softmax(tmp, x, lam, tmp, (9, 9), 0.1, rng, stream=s)  # a given stream, after the call before it
    s.synchronize()
    assert torch.equal(y, ref) and torch.equal(tmp, ref)


def test_everything_dropped(cuda_lib):
    """p = 1: zeros everywhere, also where the logits or the gradient are not numbers."""
    na = cuda_lib
    x = randn((1, 40, 3, 25), "bf16", 1).cuda()
    x[0, 3, 1, 2] = float("nan")
    y, dx, d2 = (torch.full_like(x, 5.0) for _ in range(3))
    lam, dl = torch.rand(3, device="cuda"), torch.full((3,), 5.0, device="cuda")
    na.na_softmax_dropout(x, y, (25,), 1.0, rng_state())
    assert torch.equal(y, torch.zeros_like(y))
    na.na_diff_softmax(x, x, lam, y, (25,), 1.0, rng_state())
    assert torch.equal(y, torch.zeros_like(y))
    x[0, 3, 1, 2] = 1.0
    dy = torch.full_like(x, float("inf"))
    na.na_softmax_dropout_bwd(x, dy, dx, (25,), 1.0, rng_state())
    na.na_diff_softmax_bwd(x, x, lam, dy, y, d2, dl, (25,), 1.0, rng_state())
    for t in (dx, y, d2, dl):
        assert torch.equal(t, torch.zeros_like(t))
    status_ok(na)


def test_calls_on_two_streams_at_once(cuda_lib):
    na = cuda_lib
    x = [randn((1, 96, 96, 8, 49), "bf16", i).cuda() for i in range(4)]
    q = [randn((1, 96, 96, 8, 64), "bf16", 9 + i).cuda() for i in range(4)]
    lam, rng, f = torch.rand(8, device="cuda"), rng_state(), na.RopeFreqs.scaled((20, 22))

    def work(i, **kw):
        o = [torch.empty_like(x[i]), torch.empty_like(x[i]), torch.empty_like(lam), torch.empty_like(q[i]), torch.empty_like(q[i])]
        st = torch.empty(q[i].shape[:-1], device="cuda"), torch.empty(q[i].shape[:-1], device="cuda")
        for _ in range(5):
            na.na_diff_softmax_bwd(x[i], x[(i + 1) % 4], lam, x[(i + 2) % 4], o[0], o[1], o[2], (7, 7), 0.2, rng)
            na.na_rope(q[i], None, o[3], None, f)
            na.na_layernorm(o[3], None, None, o[4], *st)
            na.na_layernorm_bwd(q[(i + 1) % 4], o[3], None, *st, o[4])
        return o

    ref = [work(i) for i in range(4)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            got.append(work(i))
    torch.cuda.synchronize()
    status_ok(na)
    for r, g in zip(ref, got):
        assert all(torch.equal(a, b) for a, b in zip(r, g))


def test_the_binding_refuses_other_layouts(cuda_lib):
    na = cuda_lib
    x = torch.zeros(1, 8, 8, 2, 32, device="cuda")
    f = na.RopeFreqs.scaled((16, 16))
    bad = [
        lambda: na.na_rope(x.transpose(1, 2), None, x, None, f),                          # strided
        lambda: na.na_rope(x, x.double(), x, x, f),                                       # another type
        lambda: na.na_rope(x, None, x, x, f),                                             # k_out without k
        lambda: na.na_rope(x, None, x, None, na.RopeFreqs.scaled((16,))),                 # frequencies of one axis
        lambda: na.na_rope(x, x[:, :4].contiguous(), x, x[:, :4].contiguous(), f),        # another grid
        lambda: na.na_rope(x, None, x, None, f, origin=(1, 2, 3)),
        lambda: na.na_layernorm(x, torch.zeros(31, device="cuda"), None, x),
        lambda: na.na_layernorm(x, torch.zeros(32, device="cuda", dtype=torch.bfloat16), None, x),
        lambda: na.na_layernorm(x, None, None, x, torch.zeros(1, 8, 8, 2, device="cuda")),
        lambda: na.na_layernorm(x[..., :0], None, None, x[..., :0]),
        lambda: na.na_dropout(x, x, 0.1, torch.zeros(2, device="cuda")),                  # the state's type
        lambda: na.na_dropout(x, x, 0.1, torch.zeros(2, dtype=torch.int64)),              # on the host
        lambda: na.na_softmax_dropout(x, x, (5, 5), 0.1, rng_state()),                    # not 32 weights
        lambda: na.na_diff_softmax(x, x, torch.zeros(3, device="cuda"), x, (32,)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {i} was taken")
    for call in (lambda: na.na_dropout(x, x, 0.1, None), lambda: na.na_dropout(x, x, 1.5, rng_state()),
                 lambda: na.na_rope(x, None, x, None, na.RopeFreqs.scaled((32, 32))),
                 lambda: na.na_rope(x[..., 1:17].contiguous().view(-1)[1:-15].view(-1, 1, 1, 16)[:8].view(1, 8, 1, 16), None,
                                    torch.zeros(1, 8, 1, 16, device="cuda"), None, na.RopeFreqs.scaled((16,)))):
        with pytest.raises(na.NAError):
            call()
    status_ok(na)


def test_workspaces_on_another_stream(cuda_lib):
    """The gradients that sum over rows, on a given stream (the library allocates there) and with the caller's
    workspace, give what the current stream gives."""
    na = cuda_lib
    x1, x2, dy = (randn((2, 30, 41, 8, 45), "bf16", i).cuda() for i in range(3))
    lam, w = torch.rand(8, device="cuda"), torch.rand(360, device="cuda")
    rows = x1.view(-1, 360)
    mean, rstd = torch.empty(rows.shape[0], device="cuda"), torch.empty(rows.shape[0], device="cuda")
    y = torch.empty_like(rows)
    na.na_layernorm(rows, w, None, y, mean, rstd)

    def both(**kw):
        o = [torch.empty_like(x1), torch.empty_like(x1), torch.empty_like(lam), torch.empty_like(rows), torch.empty_like(w),
             torch.empty_like(w)]
        torch.cuda.synchronize()
        na.na_diff_softmax_bwd(x1, x2, lam, dy, o[0], o[1], o[2], (5, 9), 0.1, rng, **kw)
        na.na_layernorm_bwd(dy.view(-1, 360), rows, w, mean, rstd, o[3], o[4], o[5], **kw)
        torch.cuda.synchronize()
        return o

    rng = rng_state()
    ref = both()
    s = torch.cuda.Stream()
    for o in (both(stream=s), both(stream=s.cuda_stream)):
        assert all(torch.equal(a, b) for a, b in zip(o, ref))


def test_captured_calls_read_the_generator_anew(cuda_lib):
    """Every operator captured into one graph, replayed with new inputs and a new generator state, gives what the
    eager calls give; two graphs with workspaces of their own do not disturb one another."""
    na = cuda_lib
    kernel, shape = (5, 7), (1, 14, 15, 3, 35)
    f = na.RopeFreqs.scaled((16, 16))
    t = {n: randn(shape, "bf16", i).cuda() for i, n in enumerate(("x1", "x2", "dy"))}
    q = randn((1, 14, 15, 3, 32), "bf16", 9).cuda()
    lam, rng = torch.rand(3, device="cuda"), rng_state()
    w = torch.rand(32, device="cuda")

    def outputs():
        e = lambda a: torch.empty_like(a)
        return dict(y=e(t["x1"]), d1=e(t["x1"]), d2=e(t["x1"]), dl=e(lam), s=e(t["x1"]), ds=e(t["x1"]), q=e(q), dr=e(q), n=e(q),
                    dn=e(q), m=torch.empty(q.shape[:-1], device="cuda"), r=torch.empty(q.shape[:-1], device="cuda"), dw=e(w), db=e(w))

    def step(o):
        na.na_rope(q, None, o["q"], None, f)
        na.na_layernorm(o["q"], w, None, o["n"], o["m"], o["r"])
        na.na_layernorm_bwd(q, o["q"], w, o["m"], o["r"], o["dn"], o["dw"], o["db"])
        na.na_dropout(o["n"], o["dr"], 0.3, rng)
        na.na_diff_softmax(t["x1"], t["x2"], lam, o["y"], kernel, 0.2, rng)
        na.na_diff_softmax_bwd(t["x1"], t["x2"], lam, t["dy"], o["d1"], o["d2"], o["dl"], kernel, 0.2, rng)
        na.na_softmax_dropout(t["x1"], o["s"], kernel, 0.2, rng)
        na.na_softmax_dropout_bwd(t["x1"], t["dy"], o["ds"], kernel, 0.2, rng)

    side = torch.cuda.Stream()
    step(outputs())
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        o = outputs()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(o)
        graphs.append((g, o))
    for turn in range(3):
        for v in t.values():
            v.normal_()
        rng[1] += 1
        ref = outputs()
        step(ref)
        torch.cuda.synchronize()
        for g, o in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, o in graphs:
            for name in ref:
                assert torch.equal(o[name], ref[name]), (turn, name)
    status_ok(na)


@pytest.mark.parametrize("which", ["soft", "soft_bwd", "diff", "diff_bwd", "norm_bwd"])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_a_copy_that_never_lands_is_reported(which, p, cuda_lib):
    """The test hook leaves out one tile's copy: the wait for it runs out after 2 ms, the kernel ends and reports it
    (sites 9 and 10), and the next launch is clean."""
    na = cuda_lib
    shape, kernel = (1, 64, 64, 4, 25), (5, 5)
    x1, x2, dy = (randn(shape, "bf16", i).cuda() for i in range(3))
    lam, w = torch.rand(4, device="cuda"), torch.rand(100, device="cuda")
    rows = randn((4096, 96), "bf16", 5).cuda()
    g = randn((4096, 96), "bf16", 6).cuda()
    mean, rstd = torch.zeros(4096, device="cuda"), torch.ones(4096, device="cuda")
    rng = rng_state()

    def call():
        e = torch.empty_like
        if which == "soft":
            o = [e(x1)]
            na.na_softmax_dropout(x1, o[0], kernel, p, rng)
        elif which == "soft_bwd":
            o = [e(x1)]
            na.na_softmax_dropout_bwd(x1, dy, o[0], kernel, p, rng)
        elif which == "diff":
            o = [e(x1)]
            na.na_diff_softmax(x1, x2, lam, o[0], kernel, p, rng)
        elif which == "diff_bwd":
            o = [e(x1), e(x1), e(lam)]
            na.na_diff_softmax_bwd(x1, x2, lam, dy, *o, kernel, p, rng)
        else:
            o = [e(rows), e(w[:96]), e(w[:96])]
            na.na_layernorm_bwd(g, rows, None, mean, rstd, *o)
        return o

    ref = call()
    status_ok(na)
    na.na_debug_wait_hook(2_000_000, True)
    try:
        call()
        st, raw = na.na_device_status()
    finally:
        na.na_debug_wait_hook(0, False)
    assert st == 5 and raw in (0x5009, 0x500A), (st, hex(raw))
    assert all(torch.equal(a, b) for a, b in zip(call(), ref))
    status_ok(na)


def test_results_do_not_depend_on_the_run(cuda_lib):
    na = cuda_lib
    shape, kernel = (2, 50, 41, 8, 45), (5, 9)
    x1, x2, dy = (randn(shape, "bf16", i).cuda() for i in range(3))
    lam = torch.rand(8, device="cuda")
    runs = []
    for _ in range(3):
        o = [torch.empty_like(x1), torch.empty_like(x1), torch.empty_like(lam)]
        na.na_diff_softmax_bwd(x1, x2, lam, dy, *o, kernel, 0.1, rng_state())
        runs.append(o)
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def chain(na, t, w, freqs, rng, p):
    """Differential neighborhood attention in training: norm of q and k per head, rotation, two maps, dropout,
    weighted sum, norm per head; then its gradients."""
    kern, dil, scale = w.kernel, w.dilation, w.scale
    e = torch.empty_like
    st = lambda: (torch.empty(t["q1"].shape[:-1], device="cuda"), torch.empty(t["q1"].shape[:-1], device="cuda"))
    keep, o = {}, {}
    for n in ("q1", "k1", "q2", "k2"):
        keep[n] = (e(t[n]), *st())
        na.na_layernorm(t[n], t["w"], t["b"], *keep[n])
    for m in "12":
        na.na_rope(keep["q" + m][0], keep["k" + m][0], keep["q" + m][0], keep["k" + m][0], freqs)   # in place
    attn = []
    for m in "12":
        a = torch.empty(t["q1"].shape[:-1] + (w.keys_per_query,), dtype=t["q1"].dtype, device="cuda")
        na.na_qk(keep["q" + m][0], keep["k" + m][0], a, kern, dil, scale)
        attn.append(a)
    y = e(attn[0])
    na.na_diff_softmax(attn[0], attn[1], t["lam"], y, kern, p, rng)
    av = e(t["v"])
    na.na_av(y, t["v"], av, kern, dil)
    out, om, orr = e(av), *st()
    na.na_layernorm(av, t["w"], t["b"], out, om, orr)
    o["out"] = out
    # backward
    dav, o["dw"], o["db"] = e(av), e(t["w"]), e(t["b"])
    na.na_layernorm_bwd(t["dO"], av, t["w"], om, orr, dav, o["dw"], o["db"])
    dy, o["dv"] = e(y), e(t["v"])
    na.na_av_bwd(dav, y, t["v"], dy, o["dv"], kern, dil)
    o["dlam"] = e(t["lam"])
    na.na_diff_softmax_bwd(attn[0], attn[1], t["lam"], dy, attn[0], attn[1], o["dlam"], kern, p, rng)
    for i, m in enumerate("12"):
        dq, dk = e(t["q1"]), e(t["q1"])
        na.na_qk_bwd(attn[i], keep["q" + m][0], keep["k" + m][0], dq, dk, kern, dil, scale)
        na.na_rope_bwd(dq, dk, dq, dk, freqs)
        for n, d in (("q" + m, dq), ("k" + m, dk)):
            o["d" + n] = e(t[n])
            na.na_layernorm_bwd(d, t[n], t["w"], keep[n][1], keep[n][2], o["d" + n])
    status_ok(na)
    return o


def chain_reference(t, w, freqs, factor):
    kern, dil, scale = w.kernel, w.dilation, w.scale
    W, Bv, L = f64(t["w"]), f64(t["b"]), f64(t["lam"])
    x = {n: f64(t[n]) for n in ("q1", "k1", "q2", "k2", "v", "dO")}
    eps = float(np.float32(1e-5))
    n = {k: ob.layernorm(x[k], W, Bv, eps) for k in ("q1", "k1", "q2", "k2")}
    r = {k: ob.rope(n[k][0], freqs.freqs) for k in n}
    a = [un.qk(r["q" + m], r["k" + m], kern, dil, scale) for m in "12"]
    y = ob.diff_softmax(a[0], a[1], L, factor)
    av = un.av(y, x["v"], kern, dil)
    out, om, orr = ob.layernorm(av, W, Bv, eps)
    o = {"out": out}
    dav, o["dw"], o["db"] = ob.layernorm_bwd(x["dO"], av, W, om, orr)
    dy, o["dv"] = un.av_bwd(dav, y, x["v"], kern, dil)
    d1, d2, o["dlam"] = ob.diff_softmax_bwd(a[0], a[1], L, dy, factor)
    for d, m in ((d1, "1"), (d2, "2")):
        dq, dk = un.qk_bwd(d, r["q" + m], r["k" + m], kern, dil, scale)
        for k, g in (("q" + m, dq), ("k" + m, dk)):
            o["d" + k] = ob.layernorm_bwd(ob.rope(g, freqs.freqs, inverse=True), x[k], W, n[k][1], n[k][2])[0]
    return o


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_differential_attention_chain(dtype, cuda_lib):
    """The operators as they are used together, against the reference chain in fp64: relative 2-norm of every output and
    gradient.  Each of the about ten roundings to the type on the longest way adds at most u of what it
    rounds, amplified by the norm (up to 1 / spread of the averaged values: about 3 here) and by the softmax's differences:
    60 u; in fp32 the same count of roundings with sums of DEPTH steps: 60 DEPTH e."""
    na = cuda_lib
    w = nain.small_workload(dtype, (9, 11), 3, 32, (5, 3), (1, 2), B=2, seed=5)
    t = {}
    for i, n in enumerate(("q1", "k1", "q2", "k2", "v", "dO")):
        t[n] = randn(w.shape, dtype, 40 + i).cuda()
    t["w"], t["b"] = (1 + 0.2 * randn((32,), "fp32", 50)).cuda(), (0.1 * randn((32,), "fp32", 51)).cuda()
    t["lam"] = (0.3 + 0.3 * torch.rand(3, generator=torch.Generator().manual_seed(1))).cuda()
    freqs = na.RopeFreqs.scaled((16, 16))
    got = chain(na, t, w, freqs, rng_state(), 0.1)
    n = math.prod(w.shape[:-1]) * w.keys_per_query
    factor = ob.dropout_factor(n, 0.1, SEED, OFFSET).reshape(w.shape[:-1] + (w.keys_per_query,))
    ref = chain_reference(t, w, freqs, factor)
    tol = 60 * DEPTH * E if dtype == "fp32" else 60 * torch.finfo(TYPES[dtype]).eps / 2
    for name in ref:
        g, x = f64(got[name]), ref[name]
        far = np.linalg.norm(g - x) / np.linalg.norm(x)
        assert far <= tol, f"{name}: {far:.3e} > {tol:.3e}"
