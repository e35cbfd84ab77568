"""GPU tests of the gated feed-forward product over long sums: every step of a sum over tokens counts, whatever the way the
sum is cut.  dh is zero but for a few tokens at the ends and at both sides of every place where a sum is cut, so that the
gradients of the weights are sums of few terms with a bound as tight as these."""
import numpy as np
import pytest
import torch

import oracle.tail as ot
import test_block_ops as tb
from test_tail_plan import BF16, FP16, FP32, planner  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu
TYPES, E, close, f64, status_ok = tb.TYPES, tb.E, tb.close, tb.f64, tb.status_ok
CODES = {"bf16": BF16, "fp16": FP16, "fp32": FP32}


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_sums_over_tokens_of_one_value(dtype, cuda_lib):
    """dbg and dbu over 2^25 tokens of one value, 0.1 in the type.  In one sequence of fp32 additions every term is rounded the same way and
    the sum is off by percents; here a tile's tokens are added first (at most 32 in one sequence), then runs of tiles, then the runs."""
    na = cuda_lib
    T, D, F = 1 << 25, 8, 8
    x = torch.zeros(T, D, dtype=TYPES[dtype], device="cuda")
    wg, wu = torch.zeros(F, D, dtype=x.dtype, device="cuda"), torch.zeros(F, D, dtype=x.dtype, device="cuda")
    bg, bu = torch.ones(F, dtype=x.dtype, device="cuda"), torch.ones(F, dtype=x.dtype, device="cuda")
    dh = torch.full((T, F), 0.1, dtype=x.dtype, device="cuda")
    dbg, dbu = torch.empty_like(bg), torch.empty_like(bu)
    na.na_glu_bwd(dh, x, wg, wu, bg=bg, bu=bu, dbg=dbg, dbu=dbu, act="relu")   # g = u = 1: dg = du = dh
    status_ok(na)
    want = np.full(F, T * float(dh[0, 0]))
    close("dbg", dbg, want, (32 + 432 + 8 + 38 + 8) * E * want, TYPES[dtype])   # a tile, a thread's 432 tiles, eight warps, 38 runs of a warp, eight warps
    assert torch.equal(dbg, dbu)


@pytest.mark.parametrize("dtype,T,D,F,tile", [("fp32", 3, (1 << 18) + 5, 9, 32), ("fp32", 1300, 1 << 18, 700, 128), ("bf16", 2, 1 << 20, 5, 32), ("fp32", 200, 8193, 40, 32)])
def test_products_over_many_channels_of_one_value(dtype, T, D, F, tile, planner, cuda_lib):  # noqa: F811
    """g and u over D channels of one product, 0.3 x 0.7 in the type, on FMA units: runs of 8192 are added up, not all in one sequence
    (which was off by 0.3% at 2^18).  A run's path is 8192 additions, then the runs."""
    na = cuda_lib
    (p,) = planner([(T, D, F, CODES[dtype])])
    assert not p["tensor"] and p["forward"]["rows"] == p["slopes"]["rows"] == tile
    x = torch.full((T, D), 0.3, dtype=TYPES[dtype], device="cuda")
    w = torch.full((F, D), 0.7, dtype=TYPES[dtype], device="cuda")
    w2 = w * (1.0 / 1024)   # exact; h stays in range
    h = torch.empty(T, F, dtype=x.dtype, device="cuda")
    na.na_glu(x, w, w2, h, act="relu")
    g = D * float(x[0, 0]) * float(w[0, 0])
    u, path = g / 1024, (8192 + 16 + -(-D // 8192)) * E
    want = np.full((T, F), g * u)
    close("h", h, want, (2 * path + path * path + 2 * E) * want, TYPES[dtype])
    # the gradients' g and u: with dh of one, dbu sums act(g) over the tokens, dbg sums u
    bg, bu = torch.zeros(F, dtype=x.dtype, device="cuda"), torch.zeros(F, dtype=x.dtype, device="cuda")
    dbg, dbu = torch.empty_like(bg), torch.empty_like(bu)
    na.na_glu_bwd(torch.ones_like(h), x, w, w2, bg=bg, bu=bu, dbg=dbg, dbu=dbu, act="relu")
    status_ok(na)
    step = torch.finfo(x.dtype).eps / 2   # dg and du are rounded to the type
    for name, got, one in (("dbg", dbg, u), ("dbu", dbu, g)):
        want = np.full(F, T * one)
        close(name, got, want, (path + (T + 16) * E + step * (1 + path)) * want, TYPES[dtype])


def test_more_splits_than_a_grid_has_places(planner, cuda_lib):  # noqa: F811
    """fp32, over 2^28 tokens: more than 32767 splits of 8192 tokens.  Values are whole numbers and halves: every sum is exact."""
    na = cuda_lib
    T, D, F = (1 << 28) + 20000, 1, 1
    (p,) = planner([(T, D, F, FP32)])
    run, splits = p["weights"]["run"], p["weights"]["splits"]
    assert splits > 32767
    x = torch.full((T, D), 0.5, device="cuda")
    dh = torch.zeros(T, F, device="cuda")
    at = sorted({t for s in (0, 1, 16384, 32766, 32767, 32768, splits - 1) for t in (s * run, s * run + 1, s * run - 1) if 0 <= t < T} | {T - 1})
    at = torch.tensor(at, device="cuda")
    dh[at, 0] = (1 + torch.arange(len(at), device="cuda")).float()
    wg, wu = torch.full((F, D), 4.0, device="cuda"), torch.full((F, D), -2.0, device="cuda")
    bg, bu = torch.zeros(F, device="cuda"), torch.full((F,), 3.0, device="cuda")   # g = 2, u = 2
    dx, dwg, dwu, dbg, dbu = (torch.full_like(t, 9.0) for t in (x, wg, wu, bg, bu))
    na.na_glu_bwd(dh, x, wg, wu, dx, dwg, dwu, bg, bu, dbg, dbu, act="relu")
    status_ok(na)
    total = float(dh.double().sum())   # dg = dh u = 2 dh, du = dh g = 2 dh
    assert float(dwg) == float(dwu) == total and float(dbg) == float(dbu) == 2 * total
    assert torch.equal(dx[at], dh[at] * (2 * 4 - 2 * 2)) and int(torch.count_nonzero(dx)) == len(at)


def cut_tokens(p, T):
    """Tokens on both sides of every kind of place where the sums over tokens are cut: steps, parts side by side, turns of them, ends."""
    w = p["weights"]
    if p["tensor"]:
        edges = {0, 1, w["ways"] - 1, w["ways"], w["ways"] + 1, w["steps"] - 1, w["steps"]}
        edges |= {t * w["run"] * w["ways"] + d for t in range(w["splits"] // w["ways"] + 1) for d in (-1, 0, 1, w["ways"] - 1)}
        edges = {64 * e for e in edges}
    else:
        edges = {s * w["run"] for s in (0, 1, 2, w["splits"] // 2, w["splits"] - 1, w["splits"])} | {16, T // 16 * 16}
    rows = -(-T // p["sum_rows"]) if p["sum_rows"] == 1 else 32 if p["tensor"] else p["slopes"]["rows"]
    edges |= {s * p["column_run"] * rows for s in (0, 1, p["runs"] - 1, p["runs"])} | {rows, (p["sum_rows"] - 1) * rows}
    return sorted({t + d for t in edges for d in (-1, 0) if 0 <= t + d < T} | {0, T - 1})


LONG = [
    # dtype, T, D, F, one launch for dx and the weights' sums
    ("bf16", 40001, 72, 700, True), ("fp16", 70003, 136, 520, True), ("bf16", 262147, 256, 688, True), ("fp16", 60000, 40, 1000, True),
    ("bf16", 60001, 99, 1000, True), ("fp16", 70003, 264, 520, False), ("bf16", 300001, 520, 100, False), ("bf16", 40000, 264, 88, False), ("fp16", 20000, 32, 24, False), ("bf16", 5001, 72, 2001, False), ("fp16", 100003, 8, 8, False),
    ("bf16", 30000, 1032, 1304, False), ("bf16", 9000, 1001, 260, False), ("fp32", 9000, 8, 12, False), ("fp32", 70001, 40, 30, False), ("fp32", 20001, 260, 130, False),
]


@pytest.mark.parametrize("dtype,T,D,F,both", LONG)
def test_every_token_counts(dtype, T, D, F, both, planner, cuda_lib):  # noqa: F811
    na = cuda_lib
    (p,) = planner([(T, D, F, CODES[dtype])])
    assert both == bool(p["tensor"] and p["tokens"]["workers"])
    type_ = TYPES[dtype]
    gen = torch.Generator(device="cuda").manual_seed(T)
    spread = lambda *s: torch.empty(s, dtype=type_, device="cuda").uniform_(-1, 1, generator=gen)
    x, wg, wu, bg, bu = spread(T, D), spread(F, D) * (D ** -0.5), spread(F, D) * (D ** -0.5), spread(F), spread(F)
    wg, wu = wg * 2, wu * 2
    full = spread(T, F)
    at = torch.tensor(cut_tokens(p, T), device="cuda")
    dh = torch.zeros_like(full)
    dh[at] = full[at]
    dx, rest = torch.full_like(x, 9.0), [torch.full_like(t, 9.0) for t in (wg, wu, bg, bu)]
    na.na_glu_bwd(dh, x, wg, wu, dx, rest[0], rest[1], bg, bu, rest[2], rest[3])
    status_ok(na)
    X, WG, WU, BG, BU, DH = (f64(t) for t in (x[at], wg, wu, bg, bu, dh[at]))
    ref = ot.glu_bwd(DH, X, WG, WU, BG, BU, "silu")
    _, g, u = ot.glu(X, WG, WU, BG, BU, "silu")
    depth = 2 * (D + 16) * E
    eg, eu = (depth * (np.abs(X) @ np.abs(W).T + np.abs(b)) for W, b in ((WG, BG), (WU, BU)))
    a, sl = ot.act(g, "silu"), ot.slope(g, "silu")
    r = 32 * E if dtype == "fp32" else 2.0 ** -17
    ea, esl = r * np.abs(a) + 1.2 * eg, r * (1 + np.abs(g)) + 0.8 * eg
    info = torch.finfo(type_)
    round_ = lambda v, e: info.eps / 2 * (np.abs(v) + e) + e + info.smallest_normal * info.eps / 2
    dg, du = DH * u * sl, DH * a
    edg = round_(dg, np.abs(DH) * (np.abs(u) * esl + np.abs(sl) * eu + esl * eu) + 4 * E * np.abs(dg))
    edu = round_(du, np.abs(DH) * ea + 2 * E * np.abs(du))
    dg, du = np.abs(dg) + edg, np.abs(du) + edu
    n = 2 * (len(at) + 16) * E   # the other terms are zeros
    slack = [edg @ np.abs(WG) + edu @ np.abs(WU) + 2 * (2 * F + 16) * E * (dg @ np.abs(WG) + du @ np.abs(WU)),
             edg.T @ np.abs(X) + n * (dg.T @ np.abs(X)), edu.T @ np.abs(X) + n * (du.T @ np.abs(X)), edg.sum(0) + n * dg.sum(0), edu.sum(0) + n * du.sum(0)]
    for name, got, want, e in zip(("dx", "dwg", "dwu", "dbg", "dbu"), [dx[at]] + rest, ref, slack):
        close(name, got, want, e, type_)
    dx[at] = 0
    assert not dx.any()
    # a token that were left out would show: the oracle without any one of them is outside the bounds
    for k in range(len(at)):
        missing = np.abs((DH[k] * u[k] * sl[k])[:, None] * X[k])
        assert (missing > slack[1] + info.eps * np.abs(ref[1])).any(), int(at[k])
    # dh of all tokens: dx of rows at both sides of tiles, and each gradient alone gives the same bits
    na.na_glu_bwd(full, x, wg, wu, dx, rest[0], rest[1], bg, bu, rest[2], rest[3])
    rows = torch.tensor(sorted({t + d for t in range(0, T, max(256, T // 2048 * 256)) for d in (-1, 0, 1, 127, 128) if 0 <= t + d < T} | set(range(T - 3, T)))[:400], device="cuda")
    X, DH = f64(x[rows]), f64(full[rows])
    want, _, _, _, _ = ot.glu_bwd(DH, X, WG, WU, BG, BU, "silu")
    _, g, u = ot.glu(X, WG, WU, BG, BU, "silu")
    eg, eu = (depth * (np.abs(X) @ np.abs(W).T + np.abs(b)) for W, b in ((WG, BG), (WU, BU)))
    a, sl = ot.act(g, "silu"), ot.slope(g, "silu")
    ea, esl = r * np.abs(a) + 1.2 * eg, r * (1 + np.abs(g)) + 0.8 * eg
    dg, du = DH * u * sl, DH * a
    edg = round_(dg, np.abs(DH) * (np.abs(u) * esl + np.abs(sl) * eu + esl * eu) + 4 * E * np.abs(dg))
    edu = round_(du, np.abs(DH) * ea + 2 * E * np.abs(du))
    dg, du = np.abs(dg) + edg, np.abs(du) + edu
    close("dx", dx[rows], want, edg @ np.abs(WG) + edu @ np.abs(WU) + 2 * (2 * F + 16) * E * (dg @ np.abs(WG) + du @ np.abs(WU)), type_)
    alone = [torch.full_like(t, 5.0) for t in [dx] + rest]
    na.na_glu_bwd(full, x, wg, wu, alone[0], None, None, bg, bu)
    na.na_glu_bwd(full, x, wg, wu, None, alone[1], alone[2], bg, bu)
    na.na_glu_bwd(full, x, wg, wu, None, None, None, bg, bu, alone[3])
    na.na_glu_bwd(full, x, wg, wu, None, None, None, bg, bu, None, alone[4])
    status_ok(na)
    assert all(torch.equal(one, all_) for one, all_ in zip(alone, [dx] + rest))


def test_the_shared_launch_gives_up_a_copy_that_never_lands(planner, cuda_lib):  # noqa: F811
    """As test_tail_wait.py, at a size whose dx and weights' sums share a launch."""
    na = cuda_lib
    T, D, F = 40001, 72, 700
    (p,) = planner([(T, D, F, BF16)])
    assert p["tokens"]["workers"]
    x, wg, wu, dh = (tb.randn(s, "bf16", i).cuda() for i, s in enumerate(((T, D), (F, D), (F, D), (T, F))))
    out = [torch.empty_like(t) for t in (x, wg, wu)]
    run = lambda: na.na_glu_bwd(dh, x, wg, wu, *out)
    run()
    status_ok(na)
    ref = [t.clone() for t in out]
    na.na_debug_wait_hook(2_000_000, True)
    try:
        run()
        st, raw = na.na_device_status()
    finally:
        na.na_debug_wait_hook(0, False)
    assert st == 5 and raw & 0xF000 == 0x5000, (st, hex(raw))
    run()
    status_ok(na)
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
