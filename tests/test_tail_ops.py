"""GPU tests of the residual add between norms and of the gated feed-forward product against the fp64 reference,
element by element.

Tolerances follow test_block_ops.py: e = 2^-24 half a step of fp32, u = finfo(type).eps / 2 of the rounding to the
tensors' type; a sum whose longest path is d additions is off by at most d e times the sum of its terms' sizes (DEPTH = 64
covers a row's sums).  A product over n terms is a path of at most n + 16 additions, whatever their order; the tensor
cores' additions cut instead of rounding, which is a whole step: 2 e each.  Errors go through each formula to first order,
and where a formula divides or multiplies errors the second order is below the slack of the counts.
"""
import numpy as np
import pytest
import torch

import oracle.tail as ot
import test_block_ops as tb

pytestmark = pytest.mark.gpu

TYPES, E, DEPTH, close, f64, randn, status_ok = tb.TYPES, tb.E, tb.DEPTH, tb.close, tb.f64, tb.randn, tb.status_ok


def dev(t):
    return None if t is None else t.cuda()


def n64(t):
    return None if t is None else f64(t)


def abs_or(t, rows, C, none):
    return np.abs(ot.rows_of(n64(t), rows, C, none))


# ---------------------------------------------------------------------------------------------
# The residual add between norms
# ---------------------------------------------------------------------------------------------

ADD = [
    # dtype, lead, C, norm, post, gate, w, b, post_b, scale, residual    (gate, w: None | channel | batch | row)
    ("fp32", (1, 256), 32, "layer", "none", "channel", "channel", True, False, 1.0, 1.0),
    ("bf16", (2, 130), 64, "rms", "rms", "channel", "channel", False, False, 1.0, 1.0),
    ("bf16", (2, 130), 256, "layer", "layer", "batch", "batch", True, True, 0.5, 1.5),
    ("fp16", (3, 37), 200, "layer", "rms", "batch", "channel", True, True, 1.0, -1.0),
    ("fp16", (3, 37), 256, "rms", "layer", None, "batch", False, True, 1.0, 1.0),
    ("fp32", (3, 37), 256, "rms", "layer", "channel", "batch", True, False, 2.0, 1.0),
    ("fp32", (2, 50), 200, "layer", "layer", "batch", "channel", False, True, 1.0, 0.0),
    ("bf16", (1, 70), 1024, "layer", "rms", "channel", "channel", True, False, 1.0, 1.0),
    ("bf16", (5, 31), 2048, "layer", "layer", "batch", "batch", True, True, 0.25, 1.0),
    ("fp32", (2, 33), 2048, "rms", "rms", "batch", None, True, False, 1.0, 1.0),
    ("fp16", (1, 9), 8192, "layer", "layer", "channel", "channel", True, True, 1.0, 1.0),
    ("fp32", (1, 9), 8192, "layer", "layer", "channel", "channel", True, True, 1.0, 1.0),
    ("bf16", (2, 20), 4104, "rms", "rms", "channel", "batch", False, False, 1.0, 1.0),
    ("fp32", (1, 40), 1001, "layer", "none", "channel", "channel", True, False, 0.5, 1.0),
    ("bf16", (2, 21), 1001, "layer", "layer", "batch", "batch", True, True, 1.0, 1.0),
    ("fp16", (1, 19), 8191, "rms", "layer", "channel", "channel", True, True, 1.0, 1.0),
    ("fp32", (1, 11), 4099, "rms", "rms", "channel", "channel", False, False, 1.0, 1.0),
    ("bf16", (7, 11), 99, "layer", "rms", "batch", "batch", True, True, 1.0, 1.0),
    ("fp16", (4, 3), 8, "layer", "layer", "row", "row", True, True, 1.0, 1.0),
    ("fp32", (4, 3), 4, "rms", "layer", "row", "channel", False, False, 1.0, 1.0),
    ("bf16", (300, 1), 264, "layer", "none", "batch", "batch", True, False, 1.0, 1.0),
    ("bf16", (3, 5, 7), 48, "none", "rms", "batch", None, False, True, 1.0, 1.0),
    ("fp32", (3, 5, 7), 48, "none", "none", "row", None, False, False, 0.5, 2.0),
    ("fp16", (1, 1), 1, "layer", "layer", "channel", "channel", True, True, 1.0, 1.0),
    ("fp32", (1, 1), 1, "rms", "rms", None, None, False, False, 1.0, 1.0),
    ("bf16", (1, 1), 4096, "rms", "none", "channel", "channel", False, False, 1.0, 1.0),
    ("bf16", (1, 5000), 96, "rms", "rms", "channel", "channel", False, False, 1.0, 1.0),
    ("fp32", (2, 2500), 72, "layer", "layer", "batch", "batch", True, True, 1.0, 1.0),
    ("fp16", (1, 3001), 520, "layer", "none", "channel", "channel", True, False, 1.0, 1.0),
    # rows that are not whole 16-byte chunks, over several tiles
    ("bf16", (2, 2501), 11, "layer", "layer", "batch", "batch", True, True, 1.0, 1.0),
    ("fp32", (1, 3), 1, "none", "none", "channel", None, False, False, 1.0, 1.0),
    ("fp16", (3, 1001), 53, "rms", "layer", "channel", "batch", True, True, 1.0, 1.0),
    ("fp32", (1, 777), 165, "layer", "rms", "channel", "channel", True, False, 0.5, 1.0),
    ("bf16", (300, 1), 259, "rms", "none", "batch", "batch", True, False, 1.0, 1.0),
    ("bf16", (1, 401), 2803, "layer", "none", "channel", "channel", True, False, 1.0, 1.0),
    ("bf16", (1, 5000), 2601, "rms", "layer", "channel", "channel", True, True, 1.0, 1.0),
    ("fp16", (1, 400), 8191, "layer", "layer", "channel", "channel", True, True, 1.0, 1.0),
    ("fp32", (2, 5500), 1001, "layer", "rms", "batch", "channel", True, False, 1.0, 1.0),
]


def add_case(case):
    dtype, lead, C, norm, post, gate, w, b, post_b, scale, residual = case

    def vector(kind, mean, seed):
        shape = {None: None, "channel": (C,), "batch": lead[:1] + (C,), "row": lead + (C,)}[kind]
        return None if shape is None else mean + 0.3 * randn(shape, "fp32", seed)

    t = dict(x=(randn(lead + (C,), "fp32", 1) + randn((C,), "fp32", 2)).to(TYPES[dtype]),
             y=(1.5 * randn(lead + (C,), "fp32", 3) + 0.5).to(TYPES[dtype]))
    v = dict(gate=vector(gate, 0.7, 4), w=vector(w, 1.0, 5), b=vector(w if w else "channel", 0.0, 6) if b else None,
             post_w=vector("channel" if post != "none" else None, 1.0, 7), post_b=vector("channel" if post_b else None, 0.0, 8))
    return t, v, dict(norm=norm, post=post, scale=scale, residual=residual)


def moment_error(v, ev, kind, mean, rstd):
    """Errors of the mean, and of the inverse deviation relative to it, of rows v that are off by ev."""
    em = DEPTH * E * np.abs(v).mean(-1) + ev.mean(-1) if kind == "layer" else np.zeros(len(v))
    d = np.abs(v - mean[:, None])
    ed = ev + em[:, None] + E * d
    return em, (DEPTH + 8) * E + ((d * ed).mean(-1) + (ed * ed).mean(-1)) * rstd ** 2


@pytest.mark.parametrize("case", ADD, ids=[str(c) for c in ADD])
def test_addnorm_and_its_gradients(case, cuda_lib):
    na = cuda_lib
    dtype, lead, C = case[:3]
    T = TYPES[dtype]
    rows = int(np.prod(lead))
    t, v, how = add_case(case)
    norm, post, scale, residual = how["norm"], how["post"], how["scale"], how["residual"]
    d = {k: dev(a) for k, a in {**t, **v}.items()}
    stat = lambda wanted: torch.full(lead, 7.0, device="cuda") if wanted else None
    s, h = torch.full_like(d["x"], 7.0), torch.full_like(d["x"], 7.0) if norm != "none" else None
    m = dict(mean=stat(norm == "layer"), rstd=stat(norm != "none"), post_mean=stat(post == "layer"), post_rstd=stat(post != "none"))
    vectors = {k: d[k] for k in v}
    na.na_addnorm(d["x"], d["y"], s, h, **vectors, **how, **m)
    status_ok(na)
    flat = lambda a: None if a is None else f64(a).reshape(rows, -1)
    X, Y = flat(t["x"]), flat(t["y"])
    eps = float(np.float32(1e-5))
    ref = ot.addnorm(X, Y, **{k: n64(a) for k, a in v.items()}, **how, eps=eps)
    A = lambda name, none: abs_or(v[name], rows, C, none)
    # s: the unit rows f, their two products with three factors, and the sums with x
    f, ef = np.abs(Y), np.zeros_like(Y)
    if post != "none":
        pm, pr = ref["post_mean"], ref["post_rstd"]
        em, er = moment_error(Y, np.zeros_like(Y), post, pm, pr)
        if post == "layer":
            close("post_mean", m["post_mean"].flatten(), pm, em)
        close("post_rstd", m["post_rstd"].flatten(), pr, pr * er)
        f = np.abs(Y - pm[:, None]) * pr[:, None]
        ef = pr[:, None] * em[:, None] + f * er[:, None]
    a, c = abs(scale) * A("gate", 1.0) * A("post_w", 1.0), abs(scale) * A("gate", 1.0) * A("post_b", 0.0)
    es = a * (ef + 8 * E * f) + 5 * E * c + 4 * E * np.abs(residual * X)
    close("s", s.view(rows, C), ref["s"], es, T)
    if norm != "none":
        mean, rstd = ref["mean"], ref["rstd"]
        em, er = moment_error(ref["s"], es, norm, mean, rstd)
        if norm == "layer":
            close("mean", m["mean"].flatten(), mean, em)
        close("rstd", m["rstd"].flatten(), rstd, rstd * er)
        unit = np.abs(ref["s"] - mean[:, None]) * rstd[:, None]
        close("h", h.view(rows, C), ref["h"], A("w", 1.0) * (rstd[:, None] * (es + em[:, None]) + unit * (er[:, None] + 8 * E))
              + 2 * E * A("b", 0.0), T)
    # in place, and without what is not wanted: the same bits
    x2, y2 = d["x"].clone(), d["y"].clone()
    na.na_addnorm(x2, y2, x2, None if h is None else y2, **vectors, **how)
    assert torch.equal(x2, s) and (h is None or torch.equal(y2, h))
    if h is not None:
        x2 = d["x"].clone()
        na.na_addnorm(x2, d["y"], None, x2, **vectors, **how)
        assert torch.equal(x2, h)

    # the gradients at what the library saved
    dh = randn(lead + (C,), dtype, 11) if norm != "none" else None
    ds = randn(lead + (C,), dtype, 12) if case[-1] != 1.5 or norm == "none" else None
    S, DH, DS = flat(s), flat(dh), flat(ds)
    grads = {"d" + k: None if a is None else torch.full_like(a, 9.0) for k, a in d.items() if k in v}
    dx, dy = torch.full_like(s, 9.0), torch.full_like(s, 9.0)
    back = {k: a for k, a in vectors.items() if k != "b"}
    normed = lambda a: None if norm == "none" else a
    args = (dev(dh), dev(ds), normed(s), d["y"])
    na.na_addnorm_bwd(*args, dx, dy, **back, **how, **m, **grads)
    status_ok(na)
    M = {k: None if a is None else f64(a).flatten() for k, a in m.items()}
    g = ot.addnorm_bwd(DH, DS, S, Y, **{k: n64(a) for k, a in v.items()}, **how, **M)
    col = lambda a: 0.0 if a is None else a[:, None]
    means = lambda q, k: (np.abs(q).mean(-1, keepdims=True) if k == "layer" else 0.0)

    def through(q, eq, f, r, kind):
        """Error of r (q - sum q / C - f sum (q f) / C) for q off by eq."""
        c1, c2 = means(q, kind), np.abs(q * f).mean(-1, keepdims=True)
        e1, e2 = means(eq, kind), (np.abs(eq) * np.abs(f)).mean(-1, keepdims=True)
        return r * (eq + e1 + np.abs(f) * e2 + 8 * E * (np.abs(q) + c1 + np.abs(f) * c2) + (DEPTH + 8) * E * (c1 + np.abs(f) * c2))

    D, eD = (np.zeros_like(Y), np.zeros_like(Y)) if DS is None else (DS, 4 * E * np.abs(DS))
    path = rows / 8 + 150
    if norm != "none":
        e = (S - col(M["mean"])) * col(M["rstd"])
        q = DH * ot.rows_of(n64(v["w"]), rows, C, 1.0)
        eD = eD + through(q, 2 * E * np.abs(q), e, col(M["rstd"]), norm)
        if v["w"] is not None:
            close("dw", grads["dw"].view(g["dw"].shape), g["dw"], (path + 8) * E * ot.to_vector(np.abs(DH * e), n64(v["w"]), C))
        if v["b"] is not None:
            close("db", grads["db"].view(g["db"].shape), g["db"], path * E * ot.to_vector(np.abs(DH), n64(v["b"]), C))
    D = g["dx"] / residual if residual else None
    close("dx", dx.view(rows, C), g["dx"], abs(residual) * eD + 4 * E * np.abs(g["dx"]), T)
    if D is None:
        D = ot.addnorm_bwd(DH, DS, S, Y, **{k: n64(a) for k, a in v.items()}, **{**how, "residual": 1.0}, **M)["dx"]
    f = Y if post == "none" else (Y - col(M["post_mean"])) * col(M["post_rstd"])
    coef = scale * ot.rows_of(n64(v["gate"]), rows, C, 1.0) * ot.rows_of(n64(v["post_w"]), rows, C, 1.0)
    q, eq = D * coef, np.abs(coef) * (eD + 8 * E * np.abs(D))
    close("dy", dy.view(rows, C), g["dy"], eq if post == "none" else through(q, eq, f, col(M["post_rstd"]), post), T)
    along, plain = eD * np.abs(f) + (path + 12) * E * np.abs(D * f), eD + (path + 8) * E * np.abs(D)
    PW, PB, G = A("post_w", 1.0), A("post_b", 0.0), A("gate", 1.0)
    for name, slack in (("gate", PW * along + PB * plain), ("post_w", G * along), ("post_b", G * plain)):
        if v[name] is not None:
            close("d" + name, grads["d" + name].view(g["d" + name].shape), g["d" + name], abs(scale) * ot.to_vector(slack, n64(v[name]), C))
    # over the inputs, with a workspace, and without the vectors' gradients: the same bits
    groups = [1 if a is None else a.numel() // C for a in (v["w"] if v["w"] is not None else v["b"], v["gate"])]
    ws = torch.empty(na.na_addnorm_bwd_workspace_size(rows, C, *groups, T), dtype=torch.uint8, device="cuda")
    for over in ("ds", "dh", "s"):
        a = dict(zip(("dh", "ds", "s", "y"), (None if b is None else b.clone() for b in args)))
        if a[over] is None:
            continue
        again = {k: None if b is None else torch.full_like(b, 5.0) for k, b in grads.items()}
        na.na_addnorm_bwd(a["dh"], a["ds"], a["s"], a["y"], a[over], a["y"], **back, **how, **m, **again, workspace=ws)
        assert torch.equal(a[over], dx) and torch.equal(a["y"], dy)
        assert all(b is None or torch.equal(b, grads[k]) for k, b in again.items())
    dx2, dy2 = torch.empty_like(dx), torch.empty_like(dy)
    na.na_addnorm_bwd(*args, dx2, dy2, **back, **how, **m)
    assert torch.equal(dx2, dx) and torch.equal(dy2, dy)


def test_addnorm_keeps_its_digits_far_from_zero(cuda_lib):
    """A mean a thousand times the spread, rows of one value, zeros, and a row that is not finite beside them."""
    na = cuda_lib
    C = 256
    for wide in (C, 1024, 1001):
        y = (randn((64, wide), "fp32", 7) + 1000.0).cuda()
        y[5], y[6] = 3.25, 0.0
        x = torch.zeros_like(y)
        s, h, ref = (torch.empty_like(y) for _ in range(3))
        na.na_addnorm(x, y, s, h, norm="layer", post="layer")
        Y = f64(y)
        o = ot.addnorm(Y * 0, Y, norm="layer", post="layer", eps=float(np.float32(1e-5)))
        em = DEPTH * E * np.abs(Y).mean(-1, keepdims=True) * o["post_rstd"][:, None]
        close("s", s, o["s"], em + np.abs(o["s"]) * ((DEPTH + 16) * E + em * em))
        assert torch.equal(s[6], torch.zeros_like(s[6])) and torch.equal(h[6], torch.zeros_like(h[6]))
        ill = y.clone()
        ill[9, 3], ill[10, 4] = float("inf"), float("nan")
        na.na_addnorm(x, ill, ref, h, norm="layer", post="layer")
        keep = torch.ones(64, dtype=torch.bool, device="cuda")
        keep[9:11] = False
        assert torch.equal(ref[keep], s[keep]) and not torch.isfinite(ref[9:11]).all()
    status_ok(na)


@pytest.mark.parametrize("C", [24, 200, 1000, 1001])
def test_addnorm_gradients_of_a_row_do_not_depend_on_its_neighbours(C, cuda_lib):
    na = cuda_lib
    n = 37
    dh, ds, s, y = (randn((n, C), "bf16", i).cuda() for i in range(4))
    stats = {k: (torch.rand(n, device="cuda") + 0.5) for k in ("mean", "rstd", "post_mean", "post_rstd")}
    dx, dy, dx2, dy2 = (torch.empty_like(s) for _ in range(4))
    na.na_addnorm_bwd(dh, ds, s, y, dx, dy, norm="layer", post="layer", **stats)
    ill = dh.clone()
    ill[20, 1] = float("inf")
    na.na_addnorm_bwd(ill, ds, s, y, dx2, dy2, norm="layer", post="layer", **stats)
    keep = torch.arange(n, device="cuda") != 20
    assert torch.equal(dx[keep], dx2[keep]) and torch.equal(dy[keep], dy2[keep])
    status_ok(na)


# ---------------------------------------------------------------------------------------------
# The gated feed-forward product
# ---------------------------------------------------------------------------------------------

GLU = [
    # dtype, T, D, F, act, bias
    ("fp32", 1, 1, 1, "silu", True), ("fp32", 5, 3, 7, "gelu", True), ("fp32", 130, 40, 70, "gelu_tanh", False),
    ("fp32", 253, 96, 255, "gelu", True), ("fp32", 300, 132, 129, "sigmoid", True), ("fp32", 1000, 24, 20, "relu", True),
    ("fp32", 9000, 8, 12, "silu", True),
    ("bf16", 1, 8, 1, "silu", True), ("bf16", 1, 64, 40, "silu", False), ("fp16", 3, 72, 17, "gelu", True),
    ("bf16", 130, 40, 70, "gelu_tanh", True), ("fp16", 127, 256, 96, "sigmoid", True), ("bf16", 128, 128, 128, "silu", False),
    ("bf16", 129, 264, 136, "gelu", False), ("fp16", 300, 520, 333, "silu", True), ("bf16", 1000, 96, 260, "relu", True),
    ("bf16", 700, 200, 1000, "silu", False), ("fp16", 513, 64, 600, "gelu_tanh", True), ("bf16", 2049, 256, 512, "silu", True),
    ("bf16", 20000, 32, 24, "silu", True), ("fp16", 64, 1024, 256, "silu", False), ("bf16", 16, 2048, 304, "gelu", False),
    ("bf16", 7, 1000, 2736, "silu", True), ("fp16", 257, 8, 8, "silu", True), ("bf16", 385, 392, 24, "sigmoid", False),
    # enough tiles for pairs of blocks, forward and for every gradient
    ("bf16", 5200, 136, 1000, "silu", True), ("fp16", 5001, 72, 2001, "relu", True), ("fp16", 2900, 1032, 1304, "silu", False),
    ("bf16", 40000, 264, 88, "sigmoid", False),
    # pairs of pairs, the last one's second beyond the tokens
    ("fp16", 5200, 1000, 1001, "gelu", False), ("bf16", 2900, 1096, 1304, "relu", True),
    # rows that are not whole 16-byte chunks
    ("bf16", 1, 1, 1, "silu", True), ("bf16", 37, 99, 50, "silu", True), ("fp16", 200, 130, 131, "gelu", False),
    ("bf16", 1300, 257, 700, "silu", True), ("fp16", 900, 1001, 260, "gelu", True), ("bf16", 3, 9001, 8000, "relu", False),
    # long sums
    ("fp16", 2, 65544, 9, "silu", True), ("fp16", 5, 65528, 24, "gelu", False), ("bf16", 130, 70000, 40, "sigmoid", True),
]


def glu_inputs(dtype, T, D, F, bias, seed=1):
    x, wg, wu = randn((T, D), dtype, seed), randn((F, D), dtype, seed + 1, D ** -0.5), randn((F, D), dtype, seed + 2, D ** -0.5)
    bg, bu = (randn((F,), dtype, seed + 3 + i, 0.3) if bias else None for i in range(2))
    return x, wg, wu, bg, bu, randn((T, F), dtype, seed + 5)


def act_error(g, how, dtype):
    """Errors of act and of its slope at g: e of a few steps in fp32; 2^-17 with the approximate exponential and quotient, whose
    error grows with |g| but stays below that for |g| < 40."""
    r = 32 * E if dtype == "fp32" else 2.0 ** -17
    return r * np.abs(ot.act(g, how)), r * (1.0 + np.abs(g))


@pytest.mark.parametrize("case", GLU, ids=[str(c) for c in GLU])
def test_glu_and_its_gradients(case, cuda_lib):
    na = cuda_lib
    dtype, T, D, F, how, bias = case
    t = glu_inputs(dtype, T, D, F, bias)
    x, wg, wu, bg, bu, dh = (dev(a) for a in t)
    h = torch.full((T, F), 7.0, dtype=TYPES[dtype], device="cuda")
    na.na_glu(x, wg, wu, h, bg, bu, act=how)
    status_ok(na)
    X, WG, WU, BG, BU, DH = (n64(a) for a in t)
    b = (0.0, 0.0) if BG is None else (np.abs(BG), np.abs(BU))
    ref, g, u = ot.glu(X, WG, WU, BG, BU, how)
    depth = 2 * (D + 16) * E
    eg, eu = (depth * (np.abs(X) @ np.abs(W).T + c) for W, c in ((WG, b[0]), (WU, b[1])))
    a, sl = ot.act(g, how), ot.slope(g, how)
    ea, esl = act_error(g, how, dtype)
    steep = np.maximum(np.abs(sl), 1.2 * (how != "relu")) if how != "relu" else (g > -eg) * 1.0
    ea = ea + steep * eg
    esl = esl + (np.abs(g) <= eg) * 1.0 if how == "relu" else esl + 0.8 * eg   # every second derivative is below 0.8
    close("h", h, ref, ea * np.abs(u) + np.abs(a) * eu + ea * eu + 2 * E * np.abs(ref), TYPES[dtype])

    dx, dwg, dwu = (torch.full_like(v, 9.0) for v in (x, wg, wu))
    dbg, dbu = (None if v is None else torch.full_like(v, 9.0) for v in (bg, bu))
    na.na_glu_bwd(dh, x, wg, wu, dx, dwg, dwu, bg, bu, dbg, dbu, act=how)
    status_ok(na)
    rdx, rdwg, rdwu, rdbg, rdbu = ot.glu_bwd(DH, X, WG, WU, BG, BU, how)
    info = torch.finfo(TYPES[dtype])
    dg, du = DH * u * sl, DH * a
    small = info.smallest_normal * info.eps / 2
    round_ = lambda v, e: info.eps / 2 * (np.abs(v) + e) + e + small
    edg = round_(dg, np.abs(DH) * (np.abs(u) * esl + np.abs(sl) * eu + esl * eu) + 4 * E * np.abs(dg))
    edu = round_(du, np.abs(DH) * ea + 2 * E * np.abs(du))
    dg, du = np.abs(dg) + edg, np.abs(du) + edu
    close("dx", dx, rdx, edg @ np.abs(WG) + edu @ np.abs(WU) + 2 * (2 * F + 16) * E * (dg @ np.abs(WG) + du @ np.abs(WU)), TYPES[dtype])
    for name, got, want, e, v in (("dwg", dwg, rdwg, edg, dg), ("dwu", dwu, rdwu, edu, du)):
        close(name, got, want, e.T @ np.abs(X) + 2 * (T + 16) * E * (v.T @ np.abs(X)), TYPES[dtype])
    if bias:
        for name, got, want, e, v in (("dbg", dbg, rdbg, edg, dg), ("dbu", dbu, rdbu, edu, du)):
            close(name, got, want, e.sum(0) + (T + 16) * E * v.sum(0), TYPES[dtype])
    # with a workspace, each gradient alone: the same bits
    ws = torch.full((na.na_glu_bwd_workspace_size(T, D, F, TYPES[dtype]),), 255, dtype=torch.uint8, device="cuda")
    one = torch.full_like(dx, 5.0)
    na.na_glu_bwd(dh, x, wg, wu, one, bg=bg, bu=bu, act=how, workspace=ws)
    assert torch.equal(one, dx)
    one, two = torch.full_like(dwg, 5.0), torch.full_like(dwu, 5.0)
    na.na_glu_bwd(dh, x, wg, wu, None, one, two, bg, bu, act=how, workspace=ws)
    assert torch.equal(one, dwg) and torch.equal(two, dwu)
    if bias:
        one = torch.full_like(dbu, 5.0)
        na.na_glu_bwd(dh, x, wg, wu, bg=bg, bu=bu, dbu=one, act=how, workspace=ws)
        assert torch.equal(one, dbu)
    status_ok(na)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("how", ot.ACTS)
def test_glu_activations_over_their_range(dtype, how, cuda_lib):
    """x of one channel and weights of one: g takes any value of the type, u is one."""
    na = cuda_lib
    top = 88.0 if dtype != "fp16" else 60.0
    v = torch.cat([torch.linspace(-top, top, 1999), torch.linspace(-3, 3, 2001), torch.tensor([0.0, -0.0, 1e4, -1e4, 3e4, -3e4])]).to(TYPES[dtype])
    D = 8
    x = torch.zeros(len(v), D, dtype=TYPES[dtype])
    x[:, 0], x[:, 1] = v, 1
    wg, wu = torch.zeros(16, D, dtype=TYPES[dtype]), torch.zeros(16, D, dtype=TYPES[dtype])
    wg[:, 0], wu[:, 1] = 1, 1
    h, dh = torch.empty(len(v), 16, dtype=TYPES[dtype], device="cuda"), torch.ones(len(v), 16, dtype=TYPES[dtype], device="cuda")
    na.na_glu(x.cuda(), wg.cuda(), wu.cuda(), h, act=how)
    G = f64(v)
    with np.errstate(over="ignore"):
        ref, sl = ot.act(G, how), ot.slope(G, how)
    r = 32 * E if dtype == "fp32" else 2.0 ** -15   # the approximate exponential at 88
    tiny = 2.0 ** -120                               # what the approximate quotient flushes
    # far below zero the reference's 1 + erf has lost its digits
    rough = 2.0 ** -50 * np.abs(G) * (how in ("gelu", "gelu_tanh", "silu", "sigmoid"))
    close("h", h, np.repeat(ref[:, None], 16, 1), (r * np.abs(ref) + tiny + rough)[:, None], TYPES[dtype])
    dx = torch.empty_like(x).cuda()
    na.na_glu_bwd(dh, x.cuda(), wg.cuda(), wu.cuda(), dx, act=how)
    status_ok(na)
    info = torch.finfo(TYPES[dtype])
    dg = info.eps / 2 * np.abs(sl) + info.smallest_normal + r * (np.abs(sl) + np.abs(G) * np.exp(-np.abs(G)) + 2.0 ** -20 * (np.abs(G) < 20)) + tiny + rough * 4
    close("dx", dx[:, 0], 16 * sl, 16 * dg + 64 * E * np.abs(sl), TYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_glu_rows_do_not_depend_on_their_neighbours(dtype, cuda_lib):
    """Bit for bit: a row that is not finite changes no other, nor does memory behind the tensors' last row."""
    na = cuda_lib
    T, D, F = 200, 72, 104
    x, wg, wu, _, _, dh = (dev(a) for a in glu_inputs(dtype, T, D, F, False))
    h, ref, dx, rdx = (torch.empty(T, n, dtype=TYPES[dtype], device="cuda") for n in (F, F, D, D))
    na.na_glu(x, wg, wu, ref)
    na.na_glu_bwd(dh, x, wg, wu, rdx)
    ill = x.clone()
    ill[77, 3], ill[130, 9] = float("nan"), float("inf")
    na.na_glu(ill, wg, wu, h)
    na.na_glu_bwd(dh, ill, wg, wu, dx)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[77], keep[130] = False, False
    assert torch.equal(h[keep], ref[keep]) and torch.equal(dx[keep], rdx[keep]) and torch.isnan(h[77]).all()
    # a view in the middle of NaN
    pad = torch.full((T + 64, D), float("nan"), dtype=TYPES[dtype], device="cuda")
    pad[32:32 + T] = x
    out = torch.full((T + 64, F), 3.0, dtype=TYPES[dtype], device="cuda")
    na.na_glu(pad[32:32 + T], wg, wu, out[32:32 + T])
    assert torch.equal(out[32:32 + T], ref) and (out[:32] == 3).all() and (out[32 + T:] == 3).all()
    status_ok(na)


@pytest.mark.parametrize("T", [3, 200, 5200])
@pytest.mark.parametrize("how", ot.ACTS)
def test_glu_columns_do_not_depend_on_their_neighbours(how, T, cuda_lib):
    """Bit for bit: weights and biases that are not finite, or far from zero, change their own column alone."""
    na = cuda_lib
    D, F = 72, 333
    x, wg, wu, bg, bu, dh = (dev(a) for a in glu_inputs("bf16", T, D, F, True))
    ill = [v.clone() for v in (wg, wu, bg, bu)]
    ill[0][20, 3], ill[0][37, 0], ill[1][50, 9], ill[2][99], ill[3][130] = float("nan"), float("inf"), float("nan"), float("nan"), float("inf")
    ill[2][201], ill[2][300], ill[2][301], ill[2][332] = -60.0, -1e30, 1e30, float("nan")
    cols = torch.ones(F, dtype=torch.bool, device="cuda")
    cols[[20, 37, 50, 99, 130, 201, 300, 301, 332]] = False

    def run(wg, wu, bg, bu):
        h, g = torch.empty(T, F, dtype=x.dtype, device="cuda"), [torch.empty_like(v) for v in (wg, wu, bg, bu)]
        na.na_glu(x, wg, wu, h, bg, bu, act=how)
        na.na_glu_bwd(dh, x, wg, wu, None, g[0], g[1], bg, bu, g[2], g[3], act=how)
        return [h.T] + g

    good, bad = run(wg, wu, bg, bu), run(*ill)
    for a, b in zip(good, bad):
        assert torch.isfinite(a).all() and torch.equal(a[cols], b[cols])
    # a far bias gives its own value: act(-60) and its limit
    G = f64(x) @ f64(wg[201]) - 60.0
    ref = ot.act(G, how) * (f64(x) @ f64(wu[201]) + f64(bu[201]))
    slack = 2.0 ** -14 * np.abs(ref) + 2.0 ** -50 * 60 * (how in ("gelu", "gelu_tanh", "silu", "sigmoid"))
    if how in ("silu", "sigmoid"):   # the only ones that are not zero there; g is off by its sum's error, and so is its exponential
        slack = slack + np.abs(ref) * 4 * D * E * (60 + (np.abs(f64(x)) @ np.abs(f64(wg[201]))))
    close("far", bad[0][201], ref, slack, torch.bfloat16)
    status_ok(na)


# ---------------------------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------------------------

def test_a_block_of_attention_and_feed_forward(cuda_lib):
    """Neighborhood attention, the add with its norms, the gated product and a second add, captured in a graph and replayed
    on new inputs; the gradients of both new operators back to the attention's output."""
    na = cuda_lib
    B, grid, heads, D, kernel, F = 2, (12, 10), 2, 16, (5, 3), 48
    C = heads * D
    bf = lambda shape, seed, scale=1.0: randn(shape, "bf16", seed, scale).cuda()
    q, k, v = (bf((B, *grid, heads, D), i) for i in range(3))
    x = bf((B, *grid, C), 4)
    wg, wu, wd = bf((F, C), 5, C ** -0.5), bf((F, C), 6, C ** -0.5), bf((C, F), 7, F ** -0.5)
    vec = lambda mean, seed, lead=(): (mean + 0.2 * randn(lead + (C,), "fp32", seed)).cuda()
    gate, w, pw, w2, b2 = vec(0.5, 8, (B,)), vec(1, 9), vec(1, 10), vec(1, 11, (B,)), vec(0, 12, (B,))
    e = torch.empty_like
    o, lse, s1, h1, hid, s2, h2 = e(q), torch.empty(q.shape[:-1], device="cuda"), e(x), e(x), e(x[..., :1]).expand(B, *grid, F).contiguous(), e(x), e(x)
    m = {n: torch.empty(x.shape[:-1], device="cuda") for n in ("rstd", "post_rstd")}
    n2 = {n: torch.empty(x.shape[:-1], device="cuda") for n in ("mean", "rstd")}
    down, dwork = e(x), e(x)
    one = dict(gate=gate, w=w, post_w=pw, norm="rms", post="rms")
    two = dict(norm="layer", w=w2)
    g = {n: e(t) for n, t in (("dwg", wg), ("dwu", wu))}
    gv = {n: e(t) for n, t in (("dgate", gate), ("dw", w), ("dpost_w", pw))}
    g2 = {n: e(t) for n, t in (("dw", w2), ("db", b2))}
    dx, do, dh1, dhid, dmid, ddown, dh2 = e(x), e(x), e(x), e(hid), e(x), e(x), bf(x.shape, 20)

    def step():
        na.na_fwd(q, k, v, o, lse, kernel)
        na.na_addnorm(x, o.view(x.shape), s1, h1, **one, **m)
        na.na_glu(h1, wg, wu, hid)
        torch.matmul(hid, wd.T, out=down)
        na.na_addnorm(s1, down, s2, h2, b=b2, **two, **n2)
        na.na_addnorm_bwd(dh2, None, s2, down, dmid, ddown, **two, **n2, **g2)
        torch.matmul(ddown, wd, out=dhid)
        na.na_glu_bwd(dhid, h1, wg, wu, dh1, **g)
        na.na_addnorm_bwd(dh1, dmid, s1, o.view(x.shape), dx, do, **one, **m, **gv)

    outs = [s1, h1, hid, s2, h2, dmid, ddown, dhid, dh1, dx, do, *g.values(), *gv.values(), *g2.values()]
    step()
    eager = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in outs:
        t.fill_(3.0)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(outs, eager))
    status_ok(na)
    # against the reference, each operator on what the library passed it: one rounding and its slack
    R = B * grid[0] * grid[1]
    flat = lambda t: f64(t).reshape(R, -1)
    eps = float(np.float32(1e-5))
    a = ot.addnorm(flat(x), flat(o), w=f64(w), gate=f64(gate), post_w=f64(pw), norm="rms", post="rms", eps=eps)
    near = lambda name, t, ref: close(name, t.view(ref.shape), ref, 2.0 ** -12 * (1 + np.abs(ref)), torch.bfloat16)
    near("s1", s1, a["s"])
    near("h1", h1, a["h"])
    near("hid", hid, ot.glu(flat(h1), f64(wg), f64(wu))[0])
    a = ot.addnorm(flat(s1), flat(down), w=f64(w2), b=f64(b2), norm="layer", eps=eps)
    near("s2", s2, a["s"])
    near("h2", h2, a["h"])
    r = ot.addnorm_bwd(flat(dh2), None, flat(s2), flat(down), w=f64(w2), norm="layer", mean=f64(n2["mean"]), rstd=f64(n2["rstd"]), b=f64(b2))
    near("dmid", dmid, r["dx"])
    near("ddown", ddown, r["dy"])
    rdx = ot.glu_bwd(flat(dhid), flat(h1), f64(wg), f64(wu))
    for name, t, ref in (("dh1", dh1, rdx[0]), ("dwg", g["dwg"], rdx[1]), ("dwu", g["dwu"], rdx[2])):
        close(name, t.view(ref.shape), ref, 2.0 ** -8 * np.abs(ref).max(), torch.bfloat16)   # dg and du rounded before their sums
    r = ot.addnorm_bwd(flat(dh1), flat(dmid), flat(s1), flat(o), w=f64(w), gate=f64(gate), post_w=f64(pw), norm="rms", post="rms",
                       rstd=f64(m["rstd"]), post_rstd=f64(m["post_rstd"]))
    near("dx", dx, r["dx"])
    near("do", do, r["dy"])
    for n in gv:
        close(n, gv[n], r[n], 2.0 ** -12 * (1 + np.abs(r[n])))


def test_calls_on_several_streams_at_once(cuda_lib):
    """Each stream with its own outputs, without a workspace of the caller's: what one call alone gives."""
    na = cuda_lib
    x, wg, wu, bg, bu, dh = (dev(a) for a in glu_inputs("bf16", 300, 128, 200, True))
    y, ds = randn((300, 128), "bf16", 20).cuda(), randn((300, 128), "bf16", 21).cuda()
    gate, rstd = torch.rand(128, device="cuda"), torch.rand(300, device="cuda") + 0.5

    def buffers():
        return [torch.empty(300, 200, dtype=x.dtype, device="cuda")] + [torch.empty_like(t) for t in (x, wg, wu, bg, bu, x, x, gate)]

    def calls(b, stream):
        na.na_glu(x, wg, wu, b[0], bg, bu, stream=stream)
        na.na_glu_bwd(dh, x, wg, wu, b[1], b[2], b[3], bg, bu, b[4], b[5], stream=stream)
        na.na_addnorm_bwd(x, ds, y, y, b[6], b[7], gate=gate, norm="rms", rstd=rstd, dgate=b[8], stream=stream)

    ref = buffers()
    calls(ref, None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    sets = [buffers() for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, b in zip(streams, sets):
            calls(b, s)
    torch.cuda.synchronize()
    status_ok(na)
    for b in sets:
        assert all(torch.equal(p, q) for p, q in zip(b, ref))


def spread(dtype, *shape):
    """Values over [-1, 1] without a buffer of another type beside them."""
    return torch.empty(shape, dtype=TYPES[dtype], device="cuda").uniform_(-1, 1)


@pytest.mark.parametrize("dtype,T,D,F", [("bf16", 600_000, 16, 7500), ("bf16", 600_001, 16, 7501), ("fp32", 70_000, 4, 62_000)])
def test_glu_of_more_than_32_bits_of_elements(dtype, T, D, F, cuda_lib):
    """T F above 2^32: the rows at both sides of that element and the last ones, and the columns of the weights' gradients
    that the last tokens alone reach."""
    na = cuda_lib
    assert T * F > 1 << 32
    x, wg, wu = spread(dtype, T, D), spread(dtype, F, D), spread(dtype, F, D)
    h, dx = torch.empty(T, F, dtype=TYPES[dtype], device="cuda"), torch.empty_like(x)
    na.na_glu(x, wg, wu, h)
    edge = (1 << 32) // F
    rows = torch.cat([torch.arange(2), torch.arange(edge - 2, edge + 3), torch.arange(T - 5, T)]).cuda()
    X, WG, WU = f64(x[rows]), f64(wg), f64(wu)
    ref, g, u = ot.glu(X, WG, WU, None, None, "silu")
    depth = 2 * (D + 16) * E
    eg, eu = (depth * (np.abs(X) @ np.abs(W).T) for W in (WG, WU))
    a, sl = ot.act(g, "silu"), ot.slope(g, "silu")
    ea, esl = act_error(g, "silu", dtype)
    ea, esl = ea + 1.2 * eg, esl + 0.8 * eg
    close("h", h[rows], ref, ea * np.abs(u) + np.abs(a) * eu + ea * eu + 2 * E * np.abs(ref), TYPES[dtype])
    # dh in h's place; only the rows looked at reach the weights
    h.zero_()
    h[rows] = spread(dtype, len(rows), F)
    DH = f64(h[rows])
    dwg, dwu = torch.empty_like(wg), torch.empty_like(wu)
    na.na_glu_bwd(h, x, wg, wu, dx, dwg, dwu)
    status_ok(na)
    rdx, rdwg, rdwu, _, _ = ot.glu_bwd(DH, X, WG, WU, None, None, "silu")
    info = torch.finfo(TYPES[dtype])
    small = info.smallest_normal * info.eps / 2
    round_ = lambda v, e: info.eps / 2 * (np.abs(v) + e) + e + small
    dg, du = DH * u * sl, DH * a
    edg = round_(dg, np.abs(DH) * (np.abs(u) * esl + np.abs(sl) * eu + esl * eu) + 4 * E * np.abs(dg))
    edu = round_(du, np.abs(DH) * ea + 2 * E * np.abs(du))
    dg, du = np.abs(dg) + edg, np.abs(du) + edu
    close("dx", dx[rows], rdx, edg @ np.abs(WG) + edu @ np.abs(WU) + 2 * (2 * F + 16) * E * (dg @ np.abs(WG) + du @ np.abs(WU)), TYPES[dtype])
    for name, got, want, e, v in (("dwg", dwg, rdwg, edg, dg), ("dwu", dwu, rdwu, edu, du)):
        close(name, got, want, e.T @ np.abs(X) + 2 * (len(rows) + 16) * E * (v.T @ np.abs(X)), TYPES[dtype])
    other = torch.ones(T, dtype=torch.bool, device="cuda")
    other[rows] = False
    assert not dx[other].any()


@pytest.mark.parametrize("C", [4096, 4001])
def test_addnorm_of_more_than_32_bits_of_elements(C, cuda_lib):
    """The rows at both sides of element 2^32 and the last ones are what a call of these rows alone gives."""
    na = cuda_lib
    rows = (1 << 32) // C + 1000
    x, y = spread("bf16", rows, C), spread("bf16", rows, C)
    w = torch.rand(C, device="cuda") + 0.5
    s, h = torch.empty_like(x), torch.empty_like(x)
    st = {k: torch.empty(rows, device="cuda") for k in ("mean", "rstd", "post_rstd")}
    how = dict(norm="layer", post="rms", w=w, gate=w, post_w=w)
    na.na_addnorm(x, y, s, h, **how, **st)
    few = torch.cat([torch.arange(3), torch.arange(rows - 1010, rows - 990), torch.arange(rows - 3, rows)]).cuda()
    pick = lambda t: t[few].clone()
    s1, h1 = torch.empty_like(pick(s)), torch.empty_like(pick(s))
    st1 = {k: torch.empty(len(few), device="cuda") for k in st}
    na.na_addnorm(pick(x), pick(y), s1, h1, **how, **st1)
    assert torch.equal(s[few], s1) and torch.equal(h[few], h1) and all(torch.equal(st[k][few], st1[k]) for k in st)
    dx, dy = x, torch.empty_like(x)
    na.na_addnorm_bwd(h, None, s, y, dx, dy, **how, **st)
    dx1, dy1 = torch.empty_like(s1), torch.empty_like(s1)
    na.na_addnorm_bwd(h1, None, s1, pick(y), dx1, dy1, **how, **st1)
    assert torch.equal(dx[few], dx1) and torch.equal(dy[few], dy1)
    status_ok(na)


@pytest.mark.parametrize("T,D,F", [(300, 257, 331), (9, 1000, 700), (200, 96, 255)])
def test_captured_calls_without_a_workspace(T, D, F, cuda_lib):
    """Two graphs, which allocate for themselves, replayed in turn and at once with other inputs in place: what eager calls give."""
    na = cuda_lib
    sets, graphs = [], []
    for i in range(2):
        x, wg, wu, bg, bu, dh = (dev(a) for a in glu_inputs("bf16", T, D, F, True, seed=30 + i))
        gate, rstd = torch.rand(D, device="cuda"), torch.rand(T, device="cuda") + 0.5
        out = [torch.empty_like(t) for t in (dh, x, wg, wu, bg, bu, x, x, gate)]

        def calls(o, x=x, wg=wg, wu=wu, bg=bg, bu=bu, dh=dh, gate=gate, rstd=rstd):
            na.na_glu(x, wg, wu, o[0], bg, bu)
            na.na_glu_bwd(dh, x, wg, wu, o[1], o[2], o[3], bg, bu, o[4], o[5])
            na.na_addnorm_bwd(x, None, x, o[1], o[6], o[7], gate=gate, norm="rms", rstd=rstd, dgate=o[8])

        calls(out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls(out)
        sets.append((x, dh, out, calls))
        graphs.append(g)
    for turn in range(3):
        for k, (x, dh, out, calls) in enumerate(sets):
            x.copy_(randn((T, D), "bf16", 50 + 2 * turn + k))
            dh.copy_(randn((T, F), "bf16", 60 + 2 * turn + k))
            for o in out:
                o.fill_(3.0)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s if turn else torch.cuda.current_stream()):
                g.replay()
        torch.cuda.synchronize()
        status_ok(na)
        for x, dh, out, calls in sets:
            want = [torch.empty_like(o) for o in out]
            calls(want)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))
