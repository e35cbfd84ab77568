"""GPU tests of the biases' gradients of the gated feed-forward product: sums over tokens of dg and du in fp32, not of what the
products take of them, which is rounded to the tensors' type."""
import numpy as np
import pytest
import torch

import oracle.tail as ot
import test_block_ops as tb

pytestmark = pytest.mark.gpu
TYPES, E, close, f64, randn, status_ok = tb.TYPES, tb.E, tb.close, tb.f64, tb.randn, tb.status_ok

CASES = [
    # dtype, T, D, F, act: few tokens (alone, in a cluster), single blocks, pairs, the rows' operand kept, FMA units; ragged ends of all
    ("bf16", 1, 64, 40, "silu"), ("fp16", 16, 2048, 33, "gelu"), ("bf16", 65, 72, 100, "gelu_tanh"), ("fp16", 128, 1000, 130, "sigmoid"),
    ("bf16", 129, 72, 333, "silu"), ("fp16", 271, 64, 1, "sigmoid"), ("bf16", 1000, 520, 96, "relu"), ("fp16", 5001, 136, 1000, "gelu"),
    ("bf16", 40001, 72, 700, "silu"), ("bf16", 2900, 1096, 1305, "gelu_tanh"), ("fp16", 271, 5, 1, "sigmoid"), ("bf16", 900, 257, 260, "silu"),
    ("bf16", 40, 33, 50, "gelu"), ("fp16", 3001, 7, 70, "silu"), ("fp32", 1, 3, 5, "silu"), ("fp32", 253, 96, 255, "gelu"), ("fp32", 5000, 132, 129, "sigmoid"),
    ("fp32", 9001, 8, 12, "gelu_tanh"),
]


@pytest.mark.parametrize("dtype,T,D,F,how", CASES)
def test_no_rounding_before_the_sum(dtype, T, D, F, how, cuda_lib):
    """Pairs of tokens whose dg and du cancel but for what dh's last bit makes: rounding them before the sum would leave its error alone."""
    na = cuda_lib
    type_ = TYPES[dtype]
    x, wg, wu, dh = randn((T, D), dtype, 1), randn((F, D), dtype, 2, D ** -0.5), randn((F, D), dtype, 3, D ** -0.5), randn((T, F), dtype, 4)
    bg, bu = randn((F,), dtype, 5, 0.3), randn((F,), dtype, 6, 0.3)
    n = T // 2
    x[n:2 * n] = x[:n]
    dh[n:2 * n] = (-dh[:n].float() * (1 + torch.finfo(type_).eps)).to(type_)
    if T % 2:
        dh[-1] *= 0.01
    X, WG, WU, BG, BU, DH = (f64(t) for t in (x, wg, wu, bg, bu, dh))
    _, _, _, rbg, rbu = ot.glu_bwd(DH, X, WG, WU, BG, BU, how)
    _, g, u = ot.glu(X, WG, WU, BG, BU, how)
    eg, eu = (2 * (D + 16) * E * (np.abs(X) @ np.abs(W).T + np.abs(b)) for W, b in ((WG, BG), (WU, BU)))
    a, sl = ot.act(g, how), ot.slope(g, how)
    # A token and its twin have the same g and u: the errors of these, and of the activation, enter with dh + its twin's dh only.
    # What each rounds by itself: three products and the sums' path
    DP = DH.copy()
    DP[:n] += DH[n:2 * n]
    DP[n:2 * n] = 0
    r = 32 * E if dtype == "fp32" else 2.0 ** -17
    ea = r * np.abs(a) + (1.2 * eg if how != "relu" else (g > -eg) * eg)
    esl = r * (1 + np.abs(g)) + (0.8 * eg if how != "relu" else (np.abs(g) <= eg) * 1.0)
    path = 4 + 32 + T / 8 + 16
    slack_g = (np.abs(DP) * (np.abs(u) * esl + np.abs(sl) * eu + esl * eu) + path * E * np.abs(DH * u * sl)).sum(0)
    slack_u = (np.abs(DP) * ea + path * E * np.abs(DH * a)).sum(0)
    d = [t.cuda() for t in (dh, x, wg, wu)]
    b = [t.cuda() for t in (bg, bu)]
    dbg, dbu = (torch.full_like(t, 9.0) for t in b)
    na.na_glu_bwd(*d, bg=b[0], bu=b[1], dbg=dbg, dbu=dbu, act=how)
    status_ok(na)
    close("dbg", dbg, rbg, slack_g, type_)
    close("dbu", dbu, rbu, slack_u, type_)
    # beside the other gradients, with a workspace: the same bits, and nothing behind the workspace is touched
    need = na.na_glu_bwd_workspace_size(T, D, F, type_)
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    out = [torch.full_like(t, 5.0) for t in d[1:] + b]
    na.na_glu_bwd(*d, *out[:3], bg=b[0], bu=b[1], dbg=out[3], dbu=out[4], act=how, workspace=ws[:need])
    status_ok(na)
    assert torch.equal(out[3], dbg) and torch.equal(out[4], dbu) and (ws[need:] == 255).all()


@pytest.mark.parametrize("dtype,T,D,F", [("bf16", 5, 64, 40), ("bf16", 300, 72, 130), ("fp16", 5201, 136, 1000), ("fp32", 130, 40, 70), ("bf16", 40, 33, 50)])
def test_columns_that_are_not_finite_stay_alone(dtype, T, D, F, cuda_lib):
    """A bias that is infinite or NaN makes g so in every row of a tile, also in those past the last token, whose dh is not there."""
    na = cuda_lib
    x, wg, wu, dh = (t.cuda() for t in (randn((T, D), dtype, 1), randn((F, D), dtype, 2, D ** -0.5), randn((F, D), dtype, 3, D ** -0.5), randn((T, F), dtype, 4)))
    bg, bu = randn((F,), dtype, 5, 0.3).cuda(), randn((F,), dtype, 6, 0.3).cuda()

    def run(bg, bu):
        o = [torch.empty_like(bg), torch.empty_like(bu)]
        na.na_glu_bwd(dh, x, wg, wu, bg=bg, bu=bu, dbg=o[0], dbu=o[1], act="relu")
        return o

    good = run(bg, bu)
    ill, ilu = bg.clone(), bu.clone()
    ill[3], ill[20], ilu[31], ilu[7] = float("nan"), float("inf"), float("-inf"), float("nan")
    bad = run(ill, ilu)
    keep = torch.ones(F, dtype=torch.bool, device="cuda")
    keep[[3, 20, 31, 7]] = False
    assert all(torch.equal(a[keep], b[keep]) and torch.isfinite(a).all() for a, b in zip(good, bad))
    assert torch.isnan(bad[0][7]) and torch.isnan(bad[1][3])   # relu's slope at NaN is zero: dbg[3] is one
    # g = infinity leaves u alone, and dbg = sum dh u where g > 0
    want = (dh[:, 20].double() * (x.double() @ wu[20].double() + bu[20].double())).sum()
    size = (dh[:, 20].double() * (x.double().abs() @ wu[20].double().abs() + bu[20].double().abs())).abs().sum()
    assert abs(float(bad[0][20]) - float(want)) <= torch.finfo(x.dtype).eps / 2 * abs(float(want)) + (2 * D + T + 64) * E * float(size)
    status_ok(na)


@pytest.mark.parametrize("dtype,T,D,F", [("bf16", 5, 64, 40), ("bf16", 300, 72, 130), ("fp16", 5201, 136, 1000), ("fp32", 130, 40, 70), ("bf16", 40, 33, 50)])
def test_rows_past_the_last_token_add_nothing(dtype, T, D, F, cuda_lib):
    """With g infinite by its bias and positive dh, dbu is infinite; what a tile holds past the last token (0 times infinity) would make it NaN."""
    na = cuda_lib
    x, wg, wu, dh = (t.cuda() for t in (randn((T, D), dtype, 1), randn((F, D), dtype, 2, D ** -0.5), randn((F, D), dtype, 3, D ** -0.5), randn((T, F), dtype, 4).abs() + 0.1))
    bg, bu = torch.full((F,), float("inf"), dtype=x.dtype, device="cuda"), torch.zeros(F, dtype=x.dtype, device="cuda")
    dbg, dbu = torch.empty_like(bg), torch.empty_like(bu)
    for how in ("relu", "silu"):
        na.na_glu_bwd(dh, x, wg, wu, bg=bg, bu=bu, dbg=dbg, dbu=dbu, act=how)
        assert (dbu == float("inf")).all() and (how != "relu" or torch.isfinite(dbg).all())
    status_ok(na)


def test_sums_past_the_types_range_of_a_token(cuda_lib):
    """fp16: a token's dg of 80000 is infinite as an operand of the products; the sum of it and of another one of -79000 is not."""
    na = cuda_lib
    for T in (4, 300):
        D, F = 64, 8
        x = torch.zeros(T, D).half().cuda()
        x[:2, 0] = 1
        wg, wu = torch.zeros(F, D).half().cuda(), torch.zeros(F, D).half().cuda()
        wg[:, 0], wu[:, 0] = 1, 2
        bg, bu = torch.zeros(F).half().cuda(), torch.zeros(F).half().cuda()
        dh = torch.zeros(T, F).half().cuda()
        dh[0], dh[1] = 40000, -39488
        dbg, dbu = torch.empty_like(bg), torch.empty_like(bu)
        na.na_glu_bwd(dh, x, wg, wu, bg=bg, bu=bu, dbg=dbg, dbu=dbu, act="relu")
        status_ok(na)
        assert (dbg == 1024).all() and (dbu == 512).all()
