"""Timed cases of the second half of a transformer block around neighborhood attention:

glu      the gated feed-forward product h = act(x Wg^T + bg) * (x Wu^T + bu) of tokens, and its gradients with
         respect to the tokens, both weights and both biases (nothing but the inputs is kept for them);
addnorm  the end of one block and the start of the next: s = residual * x + scale * gate * post(y), the stream with
         the block's output y normalised, gated and added, and h = norm(s), what the next block reads, and the
         gradients of both with those of every vector involved.

With own = False, run() computes each operator from elementary torch operations in 32 bits; with own = True it
makes the library's calls.  exact() evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------------------------------------
# Cases.  op: glu | addnorm; dir: fwd | bwd.
# ---------------------------------------------------------------------------------------------

def _glu(dir, dtype, T, D, F, act="silu", bias=False, **more):
    return {"op": "glu", "dir": dir, "dtype": dtype, "T": T, "D": D, "F": F, "act": act, "bias": bias, **more}


def _add(dir, dtype, B, N, C, norm="layer", post="none", gate="channel", w="channel", b=True, scale=1.0, residual=1.0,
         **more):
    """B batch entries of N rows of C channels.  norm, post: none | layer | rms; gate, w (and b beside it): none |
    channel (one vector) | batch (one for every batch entry)."""
    return {"op": "addnorm", "dir": dir, "dtype": dtype, "B": B, "N": N, "C": C, "norm": norm, "post": post, "gate": gate,
            "w": w, "b": b, "scale": scale, "residual": residual, **more}


def listed():
    return [
        # a single token on its way through a trained block: the weights are read once, latency counts
        _glu("fwd", "bf16", 1, 1024, 2736, name="glu_fwd_token"),
        # the 2D benchmark's tokens, 8 heads of 32 channels, hidden width 8/3 of that: many rows, a short product
        _glu("fwd", "bf16", 1024 * 1024, 256, 688, name="glu_fwd_2d"),
        # a wide block over a sequence of odd length: the largest product
        _glu("fwd", "fp16", 4095, 4096, 11008, "gelu_tanh", name="glu_fwd_wide"),
        # a small grid in full precision with biases, odd sizes throughout
        _glu("fwd", "fp32", 253, 96, 255, "gelu", True, name="glu_fwd_fp32"),
        # the 3D model shape's tokens in training
        _glu("bwd", "bf16", 2 * 8 * 128 * 128, 256, 688, name="glu_bwd_3d"),
        # a wider block with biases on an odd number of tokens
        _glu("bwd", "fp16", 2001, 1536, 4096, "gelu", True, name="glu_bwd_wide"),
        # the smallest grid of the test suite, its 32 channels in full precision
        _add("fwd", "fp32", 1, 16 * 16, 32, name="add_fwd_small"),
        # the 2D benchmark's tokens between two blocks: the attention's output normalised, gated per channel, added,
        # and the next block's norm, all of root mean square
        _add("fwd", "bf16", 1, 1024 * 1024, 256, "rms", "rms", b=False, name="add_fwd_2d"),
        # the 3D model shape with gate, scale and shift that depend on the batch entry (a conditioned block)
        _add("fwd", "fp16", 2, 8 * 128 * 128, 512, "layer", "none", "batch", "batch", name="add_fwd_cond"),
        # the 2D benchmark's tokens in training
        _add("bwd", "bf16", 1, 1024 * 1024, 256, "rms", "rms", b=False, name="add_bwd_2d"),
        # wide rows of an odd count, conditioned, the stream scaled up
        _add("bwd", "fp16", 3, 3333, 2048, "layer", "layer", "batch", "batch", residual=1.5, name="add_bwd_cond"),
        # few rows of an odd length in full precision
        _add("bwd", "fp32", 1, 333, 1001, "layer", "none", "channel", scale=0.5, name="add_bwd_few"),
    ]


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    dir = rng.choice(["fwd", "bwd"])
    if rng.random() < 0.5:
        most = 4095 * 4096 * 11008 / (3 if dir == "bwd" else 1)   # the largest listed product
        while True:
            T = max(1, int(2.0 ** rng.uniform(0, 20)))
            D = 8 * max(1, int(2.0 ** rng.uniform(1, 9)))
            F = int(2.0 ** rng.uniform(4, 13.5))
            if rng.random() < 0.7:
                F = 8 * (F // 8)
            if rng.random() < 0.1:
                D = max(1, D - rng.randint(1, 7))
            if T * D * F <= most and T * F <= 1024 * 1024 * 688 and T * D <= 1 << 28:
                return _glu(dir, dtype, T, D, F, rng.choice(["silu", "gelu", "gelu_tanh", "relu", "sigmoid"]), rng.random() < 0.3)
    size = 2.0 ** rng.uniform(10, 28)   # elements of one tensor
    C = rng.choice([32, 64, 128, 256, 512, 8 * int(2.0 ** rng.uniform(1, 10)), int(2.0 ** rng.uniform(0, 13))])
    B = rng.choice([1, 1, 2, 3, 8])
    norm, post = rng.choice(["layer", "rms"]), rng.choice(["none", "layer", "rms"])
    kinds = ["none", "channel", "channel", "batch"]
    return _add(dir, dtype, B, max(1, int(size / C / B)), C, norm, post, rng.choice(kinds), rng.choice(kinds),
                norm == "layer" and rng.random() < 0.7, rng.choice([1.0, 1.0, 0.5]), rng.choice([1.0, 1.0, 1.5]))


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def _prepare_glu(case, s, normal):
    dtype = DTYPES[case["dtype"]]
    T, D, F = case["T"], case["D"], case["F"]
    s["x"] = normal((T, D)).to(dtype)
    s["wg"], s["wu"] = ((normal((F, D)) / math.sqrt(D)).to(dtype) for _ in range(2))
    s["bg"], s["bu"] = ((0.1 * normal((F,))).to(dtype) if case["bias"] else None for _ in range(2))
    if case["dir"] == "fwd":
        s["h"] = torch.empty((T, F), dtype=dtype, device="cuda")
        return s
    s["dh"] = normal((T, F)).to(dtype)
    for name in ("x", "wg", "wu", "bg", "bu"):
        s["d" + name] = None if s[name] is None else torch.empty_like(s[name])
    return s


def _statistics(v, kind, eps):
    """Mean (None for root mean square) and inverse deviation of the rows, as a forward pass saves them."""
    if kind == "none":
        return None, None
    v = v.float()
    mean = v.mean(-1) if kind == "layer" else None
    if mean is not None:
        v = v - mean[..., None]
    return mean, (v.square_() if mean is not None else v.square()).mean(-1).add_(eps).rsqrt_()


def _prepare_add(case, s, normal):
    dtype = DTYPES[case["dtype"]]
    B, N, C = case["B"], case["N"], case["C"]
    shape = (B, N, C)
    s["eps"] = 1e-5

    def vector(kind, mean, spread):
        return None if kind == "none" else mean + spread * normal((C,) if kind == "channel" else (B, C))

    s["gate"] = vector(case["gate"], 0.5, 0.2)
    s["w"] = vector(case["w"], 1.0, 0.1)
    s["b"] = vector(case["w"], 0.0, 0.1) if case["b"] else None
    s["post_w"] = vector("channel", 1.0, 0.1) if case["post"] != "none" else None
    s["post_b"] = vector("channel", 0.0, 0.1) if case["post"] == "layer" else None
    s["y"] = normal(shape).to(dtype)
    empty = lambda kind: torch.empty((B, N), device="cuda") if kind else None
    if case["dir"] == "fwd":
        s["x"] = (normal(shape) + 0.5 * normal((C,))).to(dtype)
        s["s"], s["h"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        for name, kind in (("", case["norm"]), ("post_", case["post"])):
            s[name + "mean"], s[name + "rstd"] = empty(kind == "layer"), empty(kind != "none")
        return s
    s["s"] = (normal(shape) + 0.5 * normal((C,))).to(dtype)
    s["mean"], s["rstd"] = _statistics(s["s"], case["norm"], s["eps"])
    s["post_mean"], s["post_rstd"] = _statistics(s["y"], case["post"], s["eps"])
    s["dh"], s["ds"] = normal(shape).to(dtype), normal(shape).to(dtype)
    s["dx"], s["dy"] = torch.empty_like(s["s"]), torch.empty_like(s["s"])
    for name in ("w", "b", "gate", "post_w", "post_b"):
        s["d" + name] = None if s[name] is None else torch.empty_like(s[name])
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    s = {"case": case}
    return _prepare_glu(case, s, normal) if case["op"] == "glu" else _prepare_add(case, s, normal)


# ---------------------------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------------------------

def _run_own(s):
    import neighborhood_attention_fwd_gb300 as na

    c = s["case"]
    bwd = c["dir"] == "bwd"
    if c["op"] == "glu":
        if bwd:
            na.na_glu_bwd(s["dh"], s["x"], s["wg"], s["wu"], s["dx"], s["dwg"], s["dwu"], bg=s["bg"], bu=s["bu"], dbg=s["dbg"],
                          dbu=s["dbu"], act=c["act"])
            return [s["dx"], s["dwg"], s["dwu"], s["dbg"], s["dbu"]]
        na.na_glu(s["x"], s["wg"], s["wu"], s["h"], bg=s["bg"], bu=s["bu"], act=c["act"])
        return s["h"]
    how = {"norm": c["norm"], "post": c["post"], "scale": c["scale"], "residual": c["residual"]}
    for name in ("w", "gate", "post_w", "post_b", "mean", "rstd", "post_mean", "post_rstd"):
        how[name] = s[name]
    if bwd:
        for name in ("dw", "db", "dgate", "dpost_w", "dpost_b"):
            how[name] = s[name]
        na.na_addnorm_bwd(s["dh"], s["ds"], s["s"], s["y"], s["dx"], s["dy"], **how)
        return [s["dx"], s["dy"], s["dw"], s["db"], s["dgate"], s["dpost_w"], s["dpost_b"]]
    na.na_addnorm(s["x"], s["y"], s["s"], s["h"], b=s["b"], eps=s["eps"], **how)
    return [s["s"], s["h"], s["mean"], s["rstd"], s["post_mean"], s["post_rstd"]]


# ---------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------

def _act(v, act):
    """act(v) and its derivative."""
    if act == "relu":
        return v.clamp(min=0), (v > 0).float()
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(v * math.sqrt(0.5)))
        return v * cdf, cdf + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (v + 0.044715 * v * v * v))
        return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * k * (1 + 3 * 0.044715 * v * v)
    y = 1 / (1 + torch.exp(-v))
    return (y, y * (1 - y)) if act == "sigmoid" else (v * y, y * (1 + v * (1 - y)))


def _plain_glu(s):
    c = s["case"]
    dtype = DTYPES[c["dtype"]]
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    g, u = x @ wg.T, x @ wu.T
    if c["bias"]:
        g, u = g + s["bg"].float(), u + s["bu"].float()
    a, slope = _act(g, c["act"])
    if c["dir"] == "fwd":
        return (a * u).to(dtype)
    dh = s["dh"].float()
    dg, du = dh * u * slope, dh * a
    db = [dg.sum(0).to(dtype), du.sum(0).to(dtype)] if c["bias"] else [None, None]
    return [(dg @ wg + du @ wu).to(dtype), (dg.T @ x).to(dtype), (du.T @ x).to(dtype)] + db


def _rowwise(v):
    """A vector beside [B, N, C]: [C], or [B, C] as [B, 1, C]."""
    return v if v is None or v.dim() == 1 else v[:, None]


def _like(t, v):
    """t [B, N, C] summed to the shape of the vector v."""
    return None if v is None else t.sum((0, 1)) if v.dim() == 1 else t.sum(1)


def _normed(v, kind, eps, w, b):
    if kind == "none":
        return v, None, None
    mean = v.mean(-1) if kind == "layer" else None
    v = v if mean is None else v - mean[..., None]
    rstd = (v.square().mean(-1) + eps).rsqrt()
    v = v * rstd[..., None]
    v = v if w is None else v * _rowwise(w)
    return (v if b is None else v + _rowwise(b)), mean, rstd


def _unit(v, mean, rstd):
    v = v.float()
    return (v if mean is None else v - mean[..., None]) * rstd[..., None]


def _unnormed(g, unit, kind, rstd):
    """The gradient before a norm of the gradient g of its unit rows."""
    out = g - unit * (g * unit).mean(-1, keepdim=True)
    return (out - g.mean(-1, keepdim=True) if kind == "layer" else out) * rstd[..., None]


def _plain_add(s):
    c = s["case"]
    dtype = DTYPES[c["dtype"]]
    if c["dir"] == "fwd":
        z, post_mean, post_rstd = _normed(s["y"].float(), c["post"], s["eps"], s["post_w"], s["post_b"])
        z = z if s["gate"] is None else z * _rowwise(s["gate"])
        out = c["residual"] * s["x"].float() + c["scale"] * z
        h, mean, rstd = _normed(out, c["norm"], s["eps"], s["w"], s["b"])
        return [out.to(dtype), h.to(dtype), mean, rstd, post_mean, post_rstd]
    dh = s["dh"].float()
    unit = _unit(s["s"], s["mean"], s["rstd"])
    dw, db = _like(dh * unit, s["w"]), _like(dh, s["b"])
    g = dh if s["w"] is None else dh * _rowwise(s["w"])
    d = s["ds"].float() + _unnormed(g, unit, c["norm"], s["rstd"])
    dx = (c["residual"] * d).to(dtype)
    d = c["scale"] * d
    dpost_w = dpost_b = None
    if c["post"] == "none":
        dgate = _like(d * s["y"].float(), s["gate"])
        dy = d if s["gate"] is None else d * _rowwise(s["gate"])
        return [dx, dy.to(dtype), dw, db, dgate, None, None]
    unit = _unit(s["y"], s["post_mean"], s["post_rstd"])
    z = unit * s["post_w"]
    dgate = _like(d * (z if s["post_b"] is None else z + s["post_b"]), s["gate"])
    dz = d if s["gate"] is None else d * _rowwise(s["gate"])
    dpost_w, dpost_b = _like(dz * unit, s["post_w"]), _like(dz, s["post_b"])
    return [dx, _unnormed(dz * s["post_w"], unit, c["post"], s["post_rstd"]).to(dtype), dw, db, dgate, dpost_w, dpost_b]


def run(state):
    if own:
        return _run_own(state)
    return _plain_glu(state) if state["case"]["op"] == "glu" else _plain_add(state)


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------

def work(case):
    size, bwd = SIZES[case["dtype"]], case["dir"] == "bwd"
    if case["op"] == "glu":
        T, D, F = case["T"], case["D"], case["F"]
        bias = 2 * F if case["bias"] else 0
        if bwd:   # both projections again, then the two products that make dx and the two that make the weights' gradients
            return {"bytes": size * (2 * T * D + T * F + 4 * F * D + 2 * bias), "flops": 12 * T * D * F}
        return {"bytes": size * (T * D + T * F + 2 * F * D + bias), "flops": 4 * T * D * F}
    B, N, C = case["B"], case["N"], case["C"]
    n = B * N * C
    vector = {"none": 0, "channel": 4 * C, "batch": 4 * B * C}
    vectors = vector[case["gate"]] + vector[case["w"]] * (1 + (case["b"] and not bwd)) + {"none": 0, "layer": 8, "rms": 4}[case["post"]] * C
    made = vector[case["gate"]] + vector[case["w"]] * (1 + case["b"]) + {"none": 0, "layer": 8, "rms": 4}[case["post"]] * C
    statistics = 4 * B * N * sum({"none": 0, "layer": 2, "rms": 1}[case[k]] for k in ("norm", "post"))
    if bwd:
        return {"bytes": 6 * n * size + vectors + made + statistics, "flops": 30 * n}
    return {"bytes": 4 * n * size + vectors + statistics, "flops": 16 * n}


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_glu(case, s):
    leaves = [None if s[n] is None else s[n].double().requires_grad_(case["dir"] == "bwd") for n in ("x", "wg", "wu", "bg", "bu")]
    x, wg, wu, bg, bu = leaves
    nn = torch.nn.functional
    act = {"relu": nn.relu, "gelu": nn.gelu, "gelu_tanh": lambda v: nn.gelu(v, approximate="tanh"), "silu": nn.silu,
           "sigmoid": torch.sigmoid}[case["act"]]
    h = act(nn.linear(x, wg, bg)) * nn.linear(x, wu, bu)
    if case["dir"] == "fwd":
        return h
    h.backward(s["dh"].double())
    return [None if v is None else v.grad for v in leaves]


def _exact_add(case, s):
    B, C = case["B"], case["C"]

    def per_batch(name, otherwise):   # every vector as [B, C]
        v = s[name]
        if v is None:
            return torch.full((B, C), otherwise, device="cuda", dtype=torch.float64)
        return v.double().expand(B, C)

    gate, w, post_w = per_batch("gate", 1.0), per_batch("w", 1.0), per_batch("post_w", 1.0)
    post_b = per_batch("post_b", 0.0)
    y = s["y"].double()

    def moments(v, kind):
        m = v.sum(-1) / C if kind == "layer" else torch.zeros_like(v[..., 0])
        return m, 1.0 / torch.sqrt(torch.einsum("bnc,bnc->bn", v - m[..., None], v - m[..., None]) / C + s["eps"])

    if case["dir"] == "fwd":
        out = torch.zeros_like(y)
        post = moments(y, case["post"]) if case["post"] != "none" else (None, None)
        z = y if post[0] is None else torch.einsum("bnc,bn,bc->bnc", y - post[0][..., None], post[1], post_w) + post_b[:, None]
        out = s["x"].double() * case["residual"] + torch.einsum("bnc,bc->bnc", z, gate * case["scale"])
        mean, rstd = moments(out, case["norm"])
        h = torch.einsum("bnc,bn,bc->bnc", out - mean[..., None], rstd, w) + per_batch("b", 0.0)[:, None]
        layer = lambda kind, v: v if kind == "layer" else None
        return [out, h, layer(case["norm"], mean), rstd, layer(case["post"], post[0]), post[1]]

    def unit(v, prefix, kind):
        m = s[prefix + "mean"].double()[..., None] if kind == "layer" else 0.0
        return (v - m) * s[prefix + "rstd"].double()[..., None]

    def back(g, e, prefix, kind):   # through the row's Jacobian rstd (I - 1 1^T / C - e e^T / C)
        along = torch.einsum("bnc,bnc->bn", g, e) / C
        ones = g.sum(-1) / C if kind == "layer" else torch.zeros_like(along)
        return (g - ones[..., None] - torch.einsum("bn,bnc->bnc", along, e)) * s[prefix + "rstd"].double()[..., None]

    def summed(name, t):   # t [B, C]: the sum over each batch entry's rows
        return None if s[name] is None else (t if s[name].dim() == 2 else t.sum(0))

    dh = s["dh"].double()
    e = unit(s["s"].double(), "", case["norm"])
    dw, db = torch.einsum("bnc,bnc->bc", dh, e), dh.sum(1)
    d = s["ds"].double() + back(torch.einsum("bnc,bc->bnc", dh, w), e, "", case["norm"])
    dx = d * case["residual"]
    d = d * case["scale"]
    f = y if case["post"] == "none" else unit(y, "post_", case["post"])
    along, plain = torch.einsum("bnc,bnc->bc", d, f), d.sum(1)
    dgate = along * post_w + plain * post_b
    dy = torch.einsum("bnc,bc,bc->bnc", d, gate, post_w)
    if case["post"] != "none":
        dy = back(dy, f, "post_", case["post"])
    return [dx, dy, summed("w", dw), summed("b", db), summed("gate", dgate), summed("post_w", gate * along),
            summed("post_b", gate * plain)]


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_glu(case, s) if case["op"] == "glu" else _exact_add(case, s)
