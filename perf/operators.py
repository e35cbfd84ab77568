"""Timed cases of the operators that stand around neighborhood attention in a transformer block:
rotary positions of queries and keys on a grid, layer norm (per head or per token) with its gradients,
the differential softmax over window weights with its gradients, and dropout from a counter-based
generator whose mask is never stored (on attention weights, fused with the softmax, and on tensors).

With own = False, run() computes each operator from elementary torch operations in 32 bits (the
rotation's angles in 64); with own = True it makes the library's calls.  exact() evaluates the
definitions in 64 bits.
"""
import functools
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}


def _dims(text):
    return tuple(int(x) for x in text.split("x"))


def _prod(values):
    return functools.reduce(lambda a, b: a * b, values, 1)


# ---------------------------------------------------------------------------------------------
# Cases.  op: rope | layernorm | diff_softmax | softmax_dropout | dropout; dir: fwd | bwd.
# ---------------------------------------------------------------------------------------------

def _rope(dir, dtype, B, grid, heads_q, heads_k, D, rot, layout, scaling="none", factor=1.0, origin=0, **more):
    return {"op": "rope", "dir": dir, "dtype": dtype, "B": B, "grid": grid, "heads_q": heads_q, "heads_k": heads_k,
            "D": D, "rot": rot, "layout": layout, "scaling": scaling, "factor": factor, "origin": origin, **more}


def _norm(dir, dtype, rows, C, affine=True, **more):
    return {"op": "layernorm", "dir": dir, "dtype": dtype, "rows": rows, "C": C, "affine": affine, **more}


def _weights(op, dir, dtype, B, grid, heads, kernel, p, **more):
    return {"op": op, "dir": dir, "dtype": dtype, "B": B, "grid": grid, "heads": heads, "kernel": kernel, "p": p, **more}


def listed():
    return [
        # the smallest grid of the test suite: a call whose cost is its launch
        _rope("fwd", "fp32", 1, "16x16", 2, 2, 16, "8x8", "half", name="rope_fwd_small"),
        # the 2D benchmark's queries and keys, all channels rotated, before the fused attention
        _rope("fwd", "bf16", 1, "1024x1024", 8, 8, 32, "16x16", "half", name="rope_fwd_2d"),
        # a long 1D sequence of an odd length that starts far out, half of wide heads rotated, frequencies
        # scaled for a context eight times the trained one; the gradient's way back
        _rope("bwd", "fp16", 1, "131071", 16, 4, 128, "64", "interleaved", "yarn", 8.0, 1000000, name="rope_bwd_long"),
        # queries of the 3D model shape normalised per head before the rotation
        _norm("fwd", "bf16", 2 * 8 * 128 * 128 * 8, 32, name="norm_fwd_head"),
        # the 2D benchmark's tokens, all heads' channels in one row, the block's own norm in training
        _norm("bwd", "bf16", 1024 * 1024, 256, name="norm_bwd_token"),
        # few wide rows of an odd count, in full precision: latency and the weight gradient's reduction
        _norm("bwd", "fp32", 333, 2048, name="norm_bwd_few"),
        # the smallest grid: differential weights of two heads with a weight for every row
        _weights("diff_softmax", "fwd", "fp16", 1, "16x16", 2, "5x5", 0.0, lam="row", masked=False, name="diff_fwd_small"),
        # the profiling shape in training, with attention dropout
        _weights("diff_softmax", "fwd", "bf16", 1, "512x512", 8, "9x9", 0.1, lam="head", masked=False, name="diff_fwd_2d"),
        # the 3D model shape's gradients, the windows of some queries masked to a part
        _weights("diff_softmax", "bwd", "bf16", 2, "8x128x128", 8, "5x7x7", 0.0, lam="head", masked=True, name="diff_bwd_3d"),
        # the 2D benchmark's attention weights in training: softmax and dropout in one pass
        _weights("softmax_dropout", "fwd", "bf16", 1, "1024x1024", 8, "9x9", 0.1, masked=False, name="drop_fwd_2d"),
        # the 3D benchmark's weights on a quarter of its frames, the gradient
        _weights("softmax_dropout", "bwd", "fp16", 1, "4x256x256", 8, "3x5x5", 0.2, masked=False, name="drop_bwd_3d"),
        # the projected output of a small fp32 grid of odd sizes
        {"op": "dropout", "dir": "fwd", "dtype": "fp32", "n": 253 * 255 * 96, "p": 0.1, "name": "dropout_fp32"},
    ]


def draw(rng):
    op = rng.choice(["rope", "layernorm", "diff_softmax", "softmax_dropout", "dropout"])
    dir = rng.choice(["fwd", "bwd"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    size = 2.0 ** rng.uniform(12, 26)  # elements of one tensor
    if op == "dropout":
        return {"op": op, "dir": "fwd", "dtype": dtype, "n": int(size), "p": rng.choice([0.05, 0.1, 0.25, 0.5])}
    if op == "layernorm":
        C = rng.choice([16, 32, 64, 128, 8 * int(2.0 ** rng.uniform(1, 9)), int(2.0 ** rng.uniform(0, 12))])
        return _norm(dir, dtype, max(1, int(size / C)), C, rng.random() < 0.8)
    ndim = rng.choice([1, 2, 3])
    B = rng.choice([1, 1, 2, 3])
    heads = rng.choice([1, 2, 3, 4, 8, 12, 16])

    def grid(tokens, least):
        side = max(1.0, tokens) ** (1.0 / ndim)
        return [max(least[a], int(side * 2.0 ** rng.uniform(-0.7, 0.7))) for a in range(ndim)]

    if op == "rope":
        D = rng.choice([16, 32, 64, 128])
        rot = [2 * rng.randint(1, D // (2 * ndim)) for _ in range(ndim)]
        if rng.random() < 0.5:  # whole heads, shared evenly
            rot = [D // ndim // 2 * 2] * ndim
        heads_k = rng.choice([0, 1, heads, heads])
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        L = grid(size / (B * heads * D), [1] * ndim)
        return _rope(dir, dtype, B, "x".join(map(str, L)), heads, heads_k, D, "x".join(map(str, rot)),
                     rng.choice(["half", "interleaved"]), scaling, 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
                     rng.choice([0, 0, rng.randint(1, 1 << 20)]))
    most = {1: 65, 2: 15, 3: 9}[ndim]
    kernel = [2 * rng.randint(0, most // 2) + 1 for _ in range(ndim)]
    L = grid(size / (B * heads * _prod(kernel)), kernel)
    while B * heads * _prod(kernel) * _prod(L) > 1 << 27:
        a = max(range(ndim), key=lambda i: L[i] / kernel[i])
        L[a] = max(kernel[a], L[a] // 2)
        if all(x == k for x, k in zip(L, kernel)):
            break
    case = _weights(op, dir, dtype, B, "x".join(map(str, L)), heads, "x".join(map(str, kernel)),
                    rng.choice([0.0, 0.1, 0.1, 0.3]) if op == "diff_softmax" else rng.choice([0.1, 0.3, 0.5]),
                    masked=rng.random() < 0.4)
    if op == "diff_softmax":
        case["lam"] = rng.choice(["head", "head", "row"])
    return case


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def _rope_freqs(case):
    """Angular frequencies of each axis (lists of Python floats) and the amplitude, as the case's scaling
    defines them: base 10000; linear: all divided by the factor; ntk: the base grows so that the lowest
    frequency is divided by the factor; yarn: divided where less than one turn fits the trained length
    (8192), kept where more than 32 do, blended in between, amplitude 0.1 ln(factor) + 1."""
    factor, how, base, trained = case["factor"], case["scaling"], 10000.0, 8192
    axes = []
    for r in _dims(case["rot"]):
        b = base * factor ** (r / (r - 2)) if how == "ntk" and r > 2 else base
        f = [b ** (-2.0 * i / r) for i in range(r // 2)]
        if how == "linear":
            f = [x / factor for x in f]
        if how == "yarn":
            turns = [trained * x / (2 * math.pi) for x in f]
            keep = [min(1.0, max(0.0, (t - 1.0) / (32.0 - 1.0))) for t in turns]
            f = [x / factor * (1 - g) + x * g for x, g in zip(f, keep)]
        axes.append(f)
    return axes, (0.1 * math.log(factor) + 1.0 if how == "yarn" else 1.0)


def _logits(case, gen, shape, dtype):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)
    if case["masked"]:
        # some queries keep a part of their window, a few nothing at all
        u = torch.rand(shape[:-1], generator=gen, device="cuda")
        kept = torch.where(u < 0.7, 2.0, torch.where(u < 0.999, u, -1.0))
        t = (torch.arange(shape[-1], device="cuda", dtype=torch.float32) + 0.5) / shape[-1]
        x.masked_fill_(t > kept[..., None], float("-inf"))
    return x


def _rng_state(gen):
    return torch.randint(0, 1 << 62, (2,), generator=gen, device="cuda", dtype=torch.int64)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    op, s = case["op"], {"case": case}

    def normal(shape, kind=dtype):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(kind)

    if op == "rope":
        lead = (case["B"],) + _dims(case["grid"])
        s["q"] = normal(lead + (case["heads_q"], case["D"]))
        s["k"] = normal(lead + (case["heads_k"], case["D"])) if case["heads_k"] else None
        s["q_out"] = torch.empty_like(s["q"])
        s["k_out"] = None if s["k"] is None else torch.empty_like(s["k"])
        axes, amp = _rope_freqs(case)
        s["freqs"], s["amp"] = axes, amp
        s["freq_t"] = [torch.tensor(f, dtype=torch.float64, device="cuda") for f in axes]
        s["handle"] = None  # the library's form of the same frequencies, made on the first pass and kept
        return s
    if op == "layernorm":
        R, C = case["rows"], case["C"]
        s["x"] = (normal((R, C), torch.float32) + 0.5 * normal((C,), torch.float32)).to(dtype)
        s["w"] = 1.0 + 0.1 * normal((C,), torch.float32) if case["affine"] else None
        s["b"] = 0.1 * normal((C,), torch.float32) if case["affine"] else None
        s["eps"] = 1e-5
        s["mean"] = torch.empty(R, device="cuda")
        s["rstd"] = torch.empty(R, device="cuda")
        if case["dir"] == "bwd":
            s["dy"] = normal((R, C))
            x = s["x"].float()  # what the forward pass saved
            torch.mean(x, 1, out=s["mean"])
            s["rstd"].copy_((x.sub_(s["mean"][:, None]).square_().mean(1) + s["eps"]).rsqrt())
            s["dx"] = torch.empty_like(s["x"])
            s["dw"] = torch.empty(C, device="cuda") if case["affine"] else None
            s["db"] = torch.empty(C, device="cuda") if case["affine"] else None
        else:
            s["y"] = torch.empty_like(s["x"])
        return s
    s["rng"] = _rng_state(gen)
    if op == "dropout":
        s["x"] = normal((case["n"],))
        s["y"] = torch.empty_like(s["x"])
        return s
    lead = (case["B"],) + _dims(case["grid"]) + (case["heads"],)
    shape = lead + (_prod(_dims(case["kernel"])),)
    s["kernel"] = _dims(case["kernel"])
    s["x1"] = _logits(case, gen, shape, dtype)
    if op == "diff_softmax":
        s["x2"] = _logits(case, gen, shape, dtype)
        s["lam"] = 0.2 + 0.6 * torch.rand(lead if case["lam"] == "row" else (case["heads"],), generator=gen, device="cuda")
    if case["dir"] == "bwd":
        s["dy"] = normal(shape)
        s["dx1"] = torch.empty_like(s["x1"])
        if op == "diff_softmax":
            s["dx2"] = torch.empty_like(s["x2"])
            s["dlam"] = torch.empty_like(s["lam"])
    else:
        s["y"] = torch.empty_like(s["x1"])
    return s


# ---------------------------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------------------------

def _run_own(s):
    import neighborhood_attention_fwd_gb300 as na

    c = s["case"]
    op, bwd = c["op"], c["dir"] == "bwd"
    if op == "rope":
        if s["handle"] is None:
            s["handle"] = na.RopeFreqs(s["freqs"], s["amp"], layout=c["layout"])
        call = na.na_rope_bwd if bwd else na.na_rope
        call(s["q"], s["k"], s["q_out"], s["k_out"], s["handle"], origin=c["origin"])
        return [s["q_out"], s["k_out"]]
    if op == "layernorm":
        if bwd:
            na.na_layernorm_bwd(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], s["dx"], s["dw"], s["db"])
            return [s["dx"], s["dw"], s["db"]]
        na.na_layernorm(s["x"], s["w"], s["b"], s["y"], s["mean"], s["rstd"], eps=s["eps"])
        return [s["y"], s["mean"], s["rstd"]]
    if op == "dropout":
        na.na_dropout(s["x"], s["y"], c["p"], s["rng"])
        return s["y"]
    if op == "softmax_dropout":
        if bwd:
            na.na_softmax_dropout_bwd(s["x1"], s["dy"], s["dx1"], s["kernel"], c["p"], s["rng"])
            return s["dx1"]
        na.na_softmax_dropout(s["x1"], s["y"], s["kernel"], c["p"], s["rng"])
        return s["y"]
    if bwd:
        na.na_diff_softmax_bwd(s["x1"], s["x2"], s["lam"], s["dy"], s["dx1"], s["dx2"], s["dlam"], s["kernel"],
                               p=c["p"], rng=s["rng"])
        return [s["dx1"], s["dx2"], s["dlam"]]
    na.na_diff_softmax(s["x1"], s["x2"], s["lam"], s["y"], s["kernel"], p=c["p"], rng=s["rng"])
    return s["y"]


# ---------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------

def _low(v):
    return v & 0xFFFFFFFF


def _round(state, _):
    """One round of Philox4x32 (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011) on
    32-bit values held in int64."""
    c0, c1, c2, c3, k0, k1 = state
    a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
    return (_low(b >> 32) ^ c1 ^ k0, _low(b), _low(a >> 32) ^ c3 ^ k1, _low(a), _low(k0 + 0x9E3779B9), _low(k1 + 0xBB67AE85))


def _keep_steps(p):
    return int(math.floor((1.0 - p) * 65536.0 + 0.5))


def _kept(n, p, rng):
    """Truth values of the n elements that dropout keeps: element i takes the 16-bit field i % 8 of the
    seven-round Philox4x32 block at counter (i / 8, offset) and key seed, kept below (1 - p) 2^16."""
    block = torch.arange((n + 7) // 8, device=rng.device, dtype=torch.int64)
    seed, offset = rng[0], rng[1]
    state = (_low(block), block >> 32, _low(offset), _low(offset >> 32), _low(seed), _low(seed >> 32))
    words = functools.reduce(_round, range(7), state)[:4]
    steps = _keep_steps(p)
    fields = torch.stack([f < steps for w in words for f in (w & 0xFFFF, w >> 16)], dim=1)
    return fields.reshape(-1)[:n]


def _gain(p):
    steps = _keep_steps(p)
    return 65536.0 / steps if steps else 0.0


def _softmax(x):
    x = x.float()
    top = x.amax(-1, keepdim=True)
    e = (x - torch.where(top == float("-inf"), 0.0, top)).exp_()
    total = e.sum(-1, keepdim=True)
    return e.div_(torch.where(total == 0, 1.0, total))


def _dropped(v, p, rng):
    return v if p == 0 else torch.where(_kept(v.numel(), p, rng).view(v.shape), v * _gain(p), 0.0)


def _turned(x, cos, sin, case):
    """Rotates the pairs of each axis's channels by the angles whose cosines and sines are given."""
    if x is None:
        return None
    rot = _dims(case["rot"])
    done = sum(rot)
    parts = torch.split(x.float(), list(rot) + [x.shape[-1] - done], dim=-1)
    c, s = torch.split(cos, [r // 2 for r in rot], dim=-1), torch.split(sin, [r // 2 for r in rot], dim=-1)
    if case["layout"] == "half":
        pairs = [(v[..., :r // 2], v[..., r // 2:]) for v, r in zip(parts, rot)]
        made = [torch.cat([a * d - b * e, a * e + b * d], -1) for (a, b), d, e in zip(pairs, c, s)]
    else:
        pairs = [(v[..., 0::2], v[..., 1::2]) for v in parts[:-1]]
        made = [torch.stack([a * d - b * e, a * e + b * d], -1).flatten(-2) for (a, b), d, e in zip(pairs, c, s)]
    return torch.cat(made + [parts[-1]], -1).to(x.dtype)


def _run_plain(s):
    c = s["case"]
    op, bwd = c["op"], c["dir"] == "bwd"
    dtype = DTYPES[c["dtype"]]
    if op == "rope":
        grid = _dims(c["grid"])
        n = len(grid)
        angles = [((torch.arange(L, device="cuda", dtype=torch.float64) + c["origin"])[:, None] * f)
                  .view([L if i == a else 1 for i in range(n)] + [-1]).expand(grid + (len(f),))
                  for a, (L, f) in enumerate(zip(grid, s["freq_t"]))]
        angle = torch.cat(angles, -1)[..., None, :]
        cos, sin = (angle.cos() * s["amp"]).float(), (angle.sin() * s["amp"]).float()
        sin = -sin if bwd else sin
        return [_turned(s["q"], cos, sin, c), _turned(s["k"], cos, sin, c)]
    if op == "layernorm":
        x = s["x"].float()
        if bwd:
            h = (x - s["mean"][:, None]) * s["rstd"][:, None]
            dy = s["dy"].float()
            g = dy * s["w"] if c["affine"] else dy
            dx = (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True)) * s["rstd"][:, None]
            return [dx.to(dtype), (dy * h).sum(0) if c["affine"] else None, dy.sum(0) if c["affine"] else None]
        mean = x.mean(1)
        d = x - mean[:, None]
        rstd = (d.square().mean(1) + s["eps"]).rsqrt()
        y = d * rstd[:, None]
        return [(y * s["w"] + s["b"] if c["affine"] else y).to(dtype), mean, rstd]
    if op == "dropout":
        return _dropped(s["x"].float(), c["p"], s["rng"]).to(dtype)
    if op == "softmax_dropout":
        y = _softmax(s["x1"])
        if bwd:
            g = _dropped(s["dy"].float(), c["p"], s["rng"])
            return (y * (g - (y * g).sum(-1, keepdim=True))).to(dtype)
        return _dropped(y, c["p"], s["rng"]).to(dtype)
    y1, y2 = _softmax(s["x1"]), _softmax(s["x2"])
    lam = s["lam"][..., None]
    if not bwd:
        return _dropped(y1 - lam * y2, c["p"], s["rng"]).to(dtype)
    g = _dropped(s["dy"].float(), c["p"], s["rng"])
    r2 = (y2 * g).sum(-1, keepdim=True)
    dx1 = y1 * (g - (y1 * g).sum(-1, keepdim=True))
    dx2 = -lam * (y2 * (g - r2))
    dlam = -r2[..., 0] if c["lam"] == "row" else -r2.reshape(-1, c["heads"]).sum(0)
    return [dx1.to(dtype), dx2.to(dtype), dlam]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------

def work(case):
    size, op, bwd = SIZES[case["dtype"]], case["op"], case["dir"] == "bwd"
    if op == "rope":
        tokens = case["B"] * _prod(_dims(case["grid"]))
        heads = case["heads_q"] + case["heads_k"]
        return {"bytes": 2 * tokens * heads * case["D"] * size, "flops": 3 * tokens * heads * sum(_dims(case["rot"]))}
    if op == "layernorm":
        n = case["rows"] * case["C"]
        return {"bytes": (3 if bwd else 2) * n * size + 8 * case["rows"] + (8 * case["C"] if case["affine"] else 0)
                + (4 * case["C"] if bwd and case["affine"] else 0),
                "flops": (14 if bwd else 8) * n}
    if op == "dropout":
        return {"bytes": 2 * case["n"] * size + 16, "flops": 2 * case["n"]}
    rows = case["B"] * _prod(_dims(case["grid"])) * case["heads"]
    n = rows * _prod(_dims(case["kernel"]))
    if op == "softmax_dropout":
        return {"bytes": (3 if bwd else 2) * n * size + 16, "flops": (9 if bwd else 6) * n}
    lam = 4 * (rows if case["lam"] == "row" else case["heads"])
    return {"bytes": (5 if bwd else 3) * n * size + (2 if bwd else 1) * lam, "flops": (19 if bwd else 13) * n}


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_field(n, seed, offset, device):
    """The n 16-bit fields, from the generator's published steps with products split into 16-bit limbs."""
    mask16, mask32 = 0xFFFF, 0xFFFFFFFF

    def product(v, m):  # (high, low) 32 bits of v * m
        vl, vh, ml, mh = v & mask16, v >> 16, m & mask16, m >> 16
        ll, mid1, mid2 = vl * ml, vl * mh, vh * ml
        mid = (ll >> 16) + (mid1 & mask16) + (mid2 & mask16)
        return (vh * mh + (mid1 >> 16) + (mid2 >> 16) + (mid >> 16)) & mask32, ((mid & mask16) << 16) | (ll & mask16)

    i = torch.arange((n + 7) // 8, device=device, dtype=torch.int64)
    x = [i & mask32, i >> 32, torch.full_like(i, offset & mask32), torch.full_like(i, offset >> 32 & mask32)]
    key = [seed & mask32, seed >> 32 & mask32]
    for _ in range(7):
        h0, l0 = product(x[0], 0xD2511F53)
        h1, l1 = product(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ key[0], l1, h0 ^ x[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) & mask32, (key[1] + 0xBB67AE85) & mask32]
    out = torch.empty((i.numel(), 8), device=device, dtype=torch.int32)
    for j in range(8):
        out[:, j] = (x[j // 2] >> (16 * (j % 2))) & mask16
    return out.view(-1)[:n]


def _exact_factor(n, p, rng):
    """What dropout multiplies each element by, in 64 bits."""
    kept = round((1.0 - p) * 65536)
    seed, offset = rng.tolist()
    return (_exact_field(n, seed, offset, rng.device) < kept).double() * (65536.0 / kept)


def _exact_weights(x):
    x = x.double()
    z = torch.exp(x - torch.logsumexp(x, -1, keepdim=True))
    return torch.nan_to_num(z, nan=0.0)  # an empty row has no weights


def _exact_turn(x, angles, amp, case, sign):
    if x is None:
        return None
    out, at = x.double().clone(), 0
    n = angles[0].dim() - 1
    for a, r in enumerate(_dims(case["rot"])):
        part = x[..., at:at + r].double()
        z = torch.complex(part[..., :r // 2], part[..., r // 2:]) if case["layout"] == "half" else torch.view_as_complex(
            part.reshape(part.shape[:-1] + (r // 2, 2)))
        z = z * torch.polar(torch.full_like(angles[a], amp), sign * angles[a]).unsqueeze(n)
        out[..., at:at + r] = torch.cat([z.real, z.imag], -1) if case["layout"] == "half" else torch.view_as_real(z).flatten(-2)
        at += r
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, bwd = case["op"], case["dir"] == "bwd"
    if op == "rope":
        grid = _dims(case["grid"])
        angles = []
        for a, f in enumerate(s["freqs"]):
            pos = torch.arange(case["origin"], case["origin"] + grid[a], device="cuda").double()
            t = torch.outer(pos, torch.tensor(f, device="cuda", dtype=torch.float64))
            t = t.reshape((1,) * a + (grid[a],) + (1,) * (len(grid) - 1 - a) + (len(f),))
            angles.append(t)
        sign = -1.0 if bwd else 1.0
        return [_exact_turn(s["q"], angles, s["amp"], case, sign), _exact_turn(s["k"], angles, s["amp"], case, sign)]
    if op == "layernorm":
        x = s["x"].double()
        C = case["C"]
        if not bwd:
            mean = x.sum(1) / C
            var = (x * x).sum(1) / C - mean * mean if C == 1 else x.var(1, correction=0)
            rstd = 1.0 / torch.sqrt(var + s["eps"])
            y = torch.addcmul(s["b"].double(), (x - mean[:, None]) * rstd[:, None], s["w"].double()) if case["affine"] else (
                x - mean[:, None]) * rstd[:, None]
            return [y, mean, rstd]
        # the gradient at the saved statistics, through the matrix of the row's Jacobian
        mean, rstd = s["mean"].double(), s["rstd"].double()
        h = torch.einsum("rc,r->rc", x - mean[:, None], rstd)
        dy = s["dy"].double()
        g = torch.einsum("rc,c->rc", dy, s["w"].double()) if case["affine"] else dy
        dot = torch.einsum("rc,rc->r", g, h) / C
        dx = torch.einsum("rc,r->rc", g - (g.sum(1) / C)[:, None] - torch.einsum("rc,r->rc", h, dot), rstd)
        return [dx, torch.einsum("rc,rc->c", dy, h) if case["affine"] else None, dy.sum(0) if case["affine"] else None]
    if op == "dropout":
        return s["x"].double() * _exact_factor(case["n"], case["p"], s["rng"])
    z1 = _exact_weights(s["x1"])
    d = _exact_factor(z1.numel(), case["p"], s["rng"]).view(z1.shape) if case["p"] else 1.0
    if op == "softmax_dropout":
        if not bwd:
            return z1 * d
        g = s["dy"].double() * d
        return z1 * g - z1 * torch.einsum("...k,...k->...", z1, g)[..., None]
    z2 = _exact_weights(s["x2"])
    lam = s["lam"].double()
    if not bwd:
        return (z1 - z2 * lam[..., None]) * d
    g = s["dy"].double() * d
    t1, t2 = torch.einsum("...k,...k->...", z1, g), torch.einsum("...k,...k->...", z2, g)
    dlam = -t2 if case["lam"] == "row" else -t2.flatten(0, -2).sum(0)
    return [z1 * g - z1 * t1[..., None], (z2 * t2[..., None] - z2 * g) * lam[..., None], dlam]
