"""GPU tests of the residual add between norms and of the gated feed-forward product: the ends of fp16's range, sums over F, one bias alone,
one tensor as two arguments, and host threads of the program's own.  Tolerances as in test_tail_ops.py."""
import threading

import numpy as np
import pytest
import torch

import oracle.tail as ot
import test_block_ops as tb
from test_tail_plan import BF16, FP16, FP32, planner  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu
TYPES, E, close, f64, randn, status_ok = tb.TYPES, tb.E, tb.close, tb.f64, tb.randn, tb.status_ok
CODES = {"bf16": BF16, "fp16": FP16, "fp32": FP32}


def n64(t):
    return None if t is None else f64(t)


def glu_grads(dtype, X, WG, WU, BG, BU, DH, how="silu"):
    """The gradients, and what they may be off by: dg and du with their errors in fp32 and their rounding to the type, then the products."""
    D, F, T = X.shape[1], WG.shape[0], len(X)
    ref = ot.glu_bwd(DH, X, WG, WU, BG, BU, how)
    _, g, u = ot.glu(X, WG, WU, BG, BU, how)
    b = [0.0 if v is None else np.abs(v) for v in (BG, BU)]
    eg, eu = (2 * (D + 16) * E * (np.abs(X) @ np.abs(W).T + c) for W, c in ((WG, b[0]), (WU, b[1])))
    a, sl = ot.act(g, how), ot.slope(g, how)
    r = 32 * E if dtype == "fp32" else 2.0 ** -17
    ea, esl = r * np.abs(a) + 1.2 * eg, r * (1 + np.abs(g)) + 0.8 * eg
    info = torch.finfo(TYPES[dtype])
    round_ = lambda v, e: info.eps / 2 * (np.abs(v) + e) + e + info.smallest_normal * info.eps / 2
    dg, du = DH * u * sl, DH * a
    edg = round_(dg, np.abs(DH) * (np.abs(u) * esl + np.abs(sl) * eu + esl * eu) + 4 * E * np.abs(dg))
    edu = round_(du, np.abs(DH) * ea + 2 * E * np.abs(du))
    dg, du = np.abs(dg) + edg, np.abs(du) + edu
    n, m = 2 * (T + 16) * E, 2 * (2 * F + 16) * E
    slack = [edg @ np.abs(WG) + edu @ np.abs(WU) + m * (dg @ np.abs(WG) + du @ np.abs(WU)), edg.T @ np.abs(X) + n * (dg.T @ np.abs(X)),
             edu.T @ np.abs(X) + n * (du.T @ np.abs(X)), edg.sum(0) + n * dg.sum(0), edu.sum(0) + n * du.sum(0)]
    return ref, slack


@pytest.mark.parametrize("power", [12, -14, -20])
@pytest.mark.parametrize("T,D,F", [(12, 64, 40), (300, 72, 130), (300, 33, 50), (5200, 136, 1000)])
def test_fp16_gradients_of_scaled_dh(T, D, F, power, cuda_lib):
    """dh as a loss scaled up makes it, and a very small one.  dg and du are rounded to fp16: half a step, of 2^-24 below 2^-14.
    Few tokens have dh, so that the weights' gradients stay within the type."""
    na = cuda_lib
    dtype = "fp16"
    x, wg, wu = randn((T, D), dtype, 1), randn((F, D), dtype, 2, D ** -0.5), randn((F, D), dtype, 3, D ** -0.5)
    bg, bu = randn((F,), dtype, 4, 0.3), randn((F,), dtype, 5, 0.3)
    dh = (torch.rand((T, F), generator=torch.Generator().manual_seed(6)) * 2 - 1) * 2.0 ** power
    keep = torch.linspace(0, T - 1, 6).long()
    only = torch.zeros(T, 1)
    only[keep] = 1
    dh = (dh * only).half()
    d = [t.cuda() for t in (dh, x, wg, wu)]
    out = [torch.full_like(t, 9.0).cuda() for t in (x, wg, wu, bg, bu)]
    na.na_glu_bwd(*d, out[0], out[1], out[2], bg.cuda(), bu.cuda(), out[3], out[4])
    status_ok(na)
    ref, slack = glu_grads(dtype, *(f64(t) for t in (x[keep], wg, wu, bg, bu, dh[keep])))
    assert all(np.abs(r).max() < 60000 for r in ref)
    for name, got, want, e in zip(("dx", "dwg", "dwu", "dbg", "dbu"), [out[0][keep.cuda()]] + out[1:], ref, slack):
        close(name, got, want, e, torch.float16)


@pytest.mark.parametrize("T", [5, 300, 5200])
def test_fp16_dg_beyond_the_type_is_infinite(T, cuda_lib):
    """dg = dh u act'(g) and du = dh act(g) past 65504 are infinite, as any fp16 value past it: so are their token's dx and their columns of
    dwg or dwu, and no others."""
    na = cuda_lib
    D, F = 64, 72
    x, wg, wu, dh = randn((T, D), "fp16", 1), randn((F, D), "fp16", 2, 0.1), randn((F, D), "fp16", 3, 0.1), randn((T, F), "fp16", 4)
    bu = torch.zeros(F).half()
    run = lambda dh, bu: (lambda o: (na.na_glu_bwd(dh.cuda(), x.cuda(), wg.cuda(), wu.cuda(), *o, bu=bu.cuda(), act="relu"), o)[1])(
        [torch.empty_like(t).cuda() for t in (x, wg, wu)])
    g = (x.double() @ wg.double().T)
    row, col = T - 2, int(torch.argmax(g[T - 2]))   # g > 0 there: the slope is one
    assert g[row, col] > 0.01
    near = run(dh, bu)
    dh[row, col] = 40000.0
    bu[col] = 3.0
    far = run(dh, bu)
    status_ok(na)
    rows, cols = torch.arange(T) != row, torch.arange(F) != col
    u = x[row].double() @ wu[col].double() + 3.0
    over = [abs(float(v)) * 40000 for v in (u, g[row, col])]   # dg, du: neither is within their errors of the type's end
    assert max(over) > 66000 and all(v > 66000 or v < 65000 for v in over)
    assert not torch.isfinite(far[0][row]).any()
    assert all(v < 66000 or not torch.isfinite(far[1 + i][col]).any() for i, v in enumerate(over))
    assert torch.isfinite(far[0][rows.cuda()]).all() and torch.equal(far[1][cols.cuda()], near[1][cols.cuda()]) and torch.equal(far[2][cols.cuda()], near[2][cols.cuda()])


COLUMNS = [("bf16", 200, 16, 400001), ("fp16", 700, 520, 5000), ("bf16", 2000, 40, 30000), ("bf16", 20, 1000, 9001), ("fp32", 300, 40, 20001), ("fp32", 40, 33, 300),
           ("bf16", 3000, 333, 2000), ("bf16", 40001, 72, 700)]


@pytest.mark.parametrize("dtype,T,D,F", COLUMNS)
def test_every_column_counts_in_dx(dtype, T, D, F, planner, cuda_lib):  # noqa: F811
    """dx = dg Wg + du Wu is a sum over the columns of dg, then of du.  dh is zero but in a few columns, at both sides of every
    kind of place where that sum is cut: a sum of few terms, with a bound as tight."""
    na = cuda_lib
    (p,) = planner([(T, D, F, CODES[dtype])])
    t = p["tokens"]
    if p["tensor"]:
        half = t["steps"] // 2
        turns = t["splits"] // t["ways"]
        edges = {0, 1, t["ways"], half - 1, half} | {k * t["run"] * t["ways"] + d for k in range(turns + 1) for d in (-1, 0, 1, t["ways"] - 1)}
        edges = {64 * (e - h) for e in edges for h in (0, half)}
    else:
        pieces = -(-F // 16)
        edges = {16 * (e - h) for k in range(t["splits"] + 1) for e in (k * t["run"],) for h in (0, pieces)} | {F // 16 * 16}
    at = sorted({e + d for e in edges for d in (-1, 0) if 0 <= e + d < F} | {0, F - 1})
    at = torch.tensor(at[:: max(1, len(at) // 60)] + at[-1:]).unique().cuda()
    gen = torch.Generator(device="cuda").manual_seed(T)
    spread = lambda *s: torch.empty(s, dtype=TYPES[dtype], device="cuda").uniform_(-1, 1, generator=gen)
    x, wg, wu = spread(T, D), spread(F, D), spread(F, D)
    dh = torch.zeros(T, F, dtype=x.dtype, device="cuda")
    dh[:, at] = spread(T, len(at))
    dx = torch.full_like(x, 9.0)
    na.na_glu_bwd(dh, x, wg, wu, dx)
    status_ok(na)
    rows = torch.linspace(0, T - 1, min(T, 200), device="cuda").long()
    ref, slack = glu_grads(dtype, *(f64(v) for v in (x[rows], wg[at], wu[at])), None, None, f64(dh[rows][:, at]))
    close("dx", dx[rows], ref[0], slack[0], TYPES[dtype])


@pytest.mark.parametrize("dtype,T,D,F", [("bf16", 3, 64, 40), ("fp16", 200, 72, 100), ("bf16", 5200, 136, 1000), ("fp32", 130, 40, 70), ("bf16", 37, 33, 50)])
@pytest.mark.parametrize("which", ["bg", "bu"])
def test_one_bias_alone(which, dtype, T, D, F, cuda_lib):
    """The other one is as zeros: the same bits."""
    na = cuda_lib
    x, wg, wu, dh = (t.cuda() for t in (randn((T, D), dtype, 1), randn((F, D), dtype, 2, 0.1), randn((F, D), dtype, 3, 0.1), randn((T, F), dtype, 4)))
    b = {which: randn((F,), dtype, 5).cuda()}
    zeros = {"bg": torch.zeros_like(b[which]), "bu": torch.zeros_like(b[which]), **b}

    def run(biases):
        h, o = torch.empty_like(dh), [torch.empty_like(t) for t in (x, wg, wu, b[which])]
        na.na_glu(x, wg, wu, h, **biases)
        na.na_glu_bwd(dh, x, wg, wu, *o[:3], **biases, **{"d" + which: o[3]})
        return [h] + o

    assert all(torch.equal(a, c) for a, c in zip(run(b), run(zeros)))
    status_ok(na)


@pytest.mark.parametrize("dtype,C", [("bf16", 256), ("fp32", 33), ("fp16", 2048)])
def test_one_tensor_as_two_arguments(dtype, C, cuda_lib):
    """The stream as the block's output, dh as ds, one matrix as both weights, and the outputs over them: what copies give."""
    na = cuda_lib
    x, d = randn((70, C), dtype, 1).cuda(), randn((70, C), dtype, 2).cuda()
    e = torch.empty_like
    s, h, r, pr = e(x), e(x), torch.empty(70, device="cuda"), torch.empty(70, device="cuda")
    how = dict(norm="rms", post="rms")
    na.na_addnorm(x, x.clone(), s, h, **how, rstd=r, post_rstd=pr)
    both = x.clone()
    out = e(x)
    na.na_addnorm(both, both, both, out, **how)
    assert torch.equal(both, s) and torch.equal(out, h)
    dx, dy = e(x), e(x)
    na.na_addnorm_bwd(d, d.clone(), s, x, dx, dy, **how, rstd=r, post_rstd=pr)
    both, out = d.clone(), e(x)
    na.na_addnorm_bwd(both, both, s, x, both, out, **how, rstd=r, post_rstd=pr)
    assert torch.equal(both, dx) and torch.equal(out, dy)
    w = randn((40, C), dtype, 3).cuda()
    a, b = (torch.empty(70, 40, dtype=x.dtype, device="cuda") for _ in range(2))
    na.na_glu(x, w, w.clone(), a)
    na.na_glu(x, w, w, b)
    assert torch.equal(a, b)
    status_ok(na)


def test_the_first_calls_of_a_thread(cuda_lib):
    """A host thread that has made no CUDA call yet gets what the main thread gets, bit for bit, and several at once do."""
    na = cuda_lib
    sizes = [(3, 64, 40), (300, 72, 130), (5200, 136, 1000), (40001, 72, 700)]
    stream = torch.cuda.current_stream().cuda_stream
    work, want, failed = [], [], []
    for T, D, F in sizes:
        x, wg, wu, dh = (t.cuda() for t in (randn((T, D), "bf16", 1), randn((F, D), "bf16", 2, 0.1), randn((F, D), "bf16", 3, 0.1), randn((T, F), "bf16", 4)))
        gate, r = torch.rand(D, device="cuda"), torch.rand(T, device="cuda") + 0.5
        ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (na.na_glu_bwd_workspace_size(T, D, F), na.na_addnorm_bwd_workspace_size(T, D))]

        def calls(o, x=x, wg=wg, wu=wu, dh=dh, gate=gate, r=r, ws=ws):
            na.na_glu(x, wg, wu, o[0])
            na.na_glu_bwd(dh, x, wg, wu, *o[1:4], workspace=ws[0])
            na.na_addnorm(x, x, o[4], o[5], gate=gate)
            na.na_addnorm_bwd(x, None, x, x, o[6], o[7], gate=gate, norm="rms", rstd=r, dgate=o[8], workspace=ws[1])

        sets = [[torch.zeros_like(t) for t in (dh, x, wg, wu, x, x, x, x, gate)] for _ in range(2)]
        calls(sets[0])
        want.append(sets[0])
        work.append((calls, sets[1]))
    torch.cuda.synchronize()
    assert stream == torch.cuda.current_stream().cuda_stream

    def run(calls, out):
        try:
            for _ in range(20):
                calls(out)
        except Exception as ex:   # noqa: BLE001  (handed to the test's own thread)
            failed.append(ex)

    for together in (False, True):
        threads = [threading.Thread(target=run, args=w) for w in work]
        for t in threads:
            t.start()
            if not together:
                t.join()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert not failed, failed
        status_ok(na)
        for (_, out), ref in zip(work, want):
            assert all(torch.equal(a, b) for a, b in zip(out, ref))
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
