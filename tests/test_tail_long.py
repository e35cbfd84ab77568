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
    the sum is off by percents; here a sum takes at most 8192 terms, then the runs (4096) are added eight warps a block."""
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
    close("dbg", dbg, want, (1024 + 8 + 512 + 8) * E * want, TYPES[dtype])   # a thread's 1024 tokens, eight warps, 512 runs of a warp, eight warps
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
