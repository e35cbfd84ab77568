"""Edges of the operators around the attention that a call's documentation allows: logits far from zero, statistics
near the ends of fp32, rows that share a warp with rows of other kinds, host threads at once, sizes past 32 bits.
Tolerances are those of test_block_ops.py, derived there.
"""
import math
import threading

import numpy as np
import pytest
import torch

import neighborhood_attention_fwd_gb300 as nab
import oracle.block as ob
import test_block_ops as tb
from neighborhood_attention_fwd_gb300 import build as nabuild

TYPES, E, DEPTH, close, f64, randn = tb.TYPES, tb.E, tb.DEPTH, tb.close, tb.f64, tb.randn


def bits(t):
    """A tensor's bit patterns: 0 and -0 differ, as do NaNs."""
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)


# ---------------------------------------------------------------------------------------------
# Window softmax
# ---------------------------------------------------------------------------------------------

FAR = [1e10, 1e12, 1e20, 1e30, 1e36, 1e37, 2e9, 1.5e8, 3e6, 2.0 ** 20, 2.0 ** 20 - 1, 65504.0]


def far_logits(shape, dtype, seed):
    """Rows around +-FAR and the type's extremes: of one value, of one value but for a few places (some of them masked),
    and spread by a few units (which a type of few digits rounds away far from zero)."""
    x = randn(shape, "fp32", seed, 2.0).double()
    rows = x.view(-1, shape[-1])
    top = torch.finfo(TYPES[dtype]).max
    bases = [s * b for b in FAR for s in (1, -1)] + [top, -top]
    for i in range(rows.shape[0]):
        base, kind = bases[(i + seed) % len(bases)], (i // len(bases)) % 3
        if kind == 2 and abs(base) < top:
            rows[i] += base
            continue
        rows[i] = base
        if kind == 1 and shape[-1] > 4:
            rows[i, 1] = base - abs(base) / 64
            rows[i, 3] = -top
            rows[i, 4] = -math.inf
    return x.to(TYPES[dtype])


@pytest.mark.gpu
@pytest.mark.parametrize("K", [5, 81, 399, 765, 1001])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_logits_far_from_zero(dtype, K, cuda_lib):
    """A row's weights depend on the differences of its logits, wherever they lie."""
    na = cuda_lib
    shape, kernel, heads = (1, max(K, 80), 3, K), (K,), 3
    x1, x2, dy = far_logits(shape, dtype, 0), far_logits(shape, dtype, 7), randn(shape, dtype, 3)
    lam = randn((heads,), "fp32", 4)
    d1, d2, dd, dl, rng = x1.cuda(), x2.cuda(), dy.cuda(), lam.cuda(), tb.rng_state()
    y, dx, z, g1, g2 = (torch.full_like(d1, 5.0) for _ in range(5))
    gl = torch.full_like(dl, 5.0)
    na.na_softmax_dropout(d1, y, kernel, 0.2, rng)
    na.na_softmax_dropout_bwd(d1, dd, dx, kernel, 0.2, rng)
    na.na_diff_softmax(d1, d2, dl, z, kernel)
    na.na_diff_softmax_bwd(d1, d2, dl, dd, g1, g2, gl, kernel)
    tb.status_ok(na)
    X1, X2, D, L = f64(x1), f64(x2), f64(dy), f64(lam)
    s1, s2 = ob.softmax(X1), ob.softmax(X2)
    e1, e2 = tb.map_error(X1, s1), tb.map_error(X2, s2)
    f, one = ob.dropout_factor(x1.numel(), 0.2, tb.SEED, tb.OFFSET).reshape(shape), np.ones(shape)
    ref = ob.softmax_dropout(X1, f)
    close("y", y, ref, np.abs(ref) * e1 + 2.0 ** -120, TYPES[dtype])
    close("dx", dx, ob.softmax_dropout_bwd(X1, D, f), tb.grad_slack(s1, e1, D, f)[0], TYPES[dtype])
    lr = np.abs(L)[:, None]
    close("diff", z, ob.diff_softmax(X1, X2, L, one), s1 * e1 + lr * s2 * (e2 + 4 * E) + 2.0 ** -120, TYPES[dtype])
    r1, r2, rl = ob.diff_softmax_bwd(X1, X2, L, D, one)
    (k1, _), (k2, row) = tb.grad_slack(s1, e1, D, one), tb.grad_slack(s2, e2, D, one)
    close("dx1", g1, r1, k1, TYPES[dtype])
    close("dx2", g2, r2, lr * (k2 + 4 * E * np.abs(r2)), TYPES[dtype])
    each = np.abs((s2 * D).sum(-1)).reshape(-1, heads).sum(0)
    close("dlam", gl, rl, row.reshape(-1, heads).sum(0) + (shape[1] / 8 + 300) * E * each)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [5, 81, 201, 399, 1001])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_logits_far_from_zero_without_dropout(dtype, K, cuda_lib):
    """The plain window softmax of the same rows."""
    na = cuda_lib
    x = far_logits((1, max(K, 80), 3, K), dtype, 0)
    y = torch.full_like(x, 5.0).cuda()
    na.na_softmax(x.cuda(), y, (K,))
    tb.status_ok(na)
    s = ob.softmax(f64(x))
    close("y", y, s, s * tb.map_error(f64(x), s) + 2.0 ** -120, TYPES[dtype])


@pytest.mark.gpu
@pytest.mark.parametrize("K", [1, 5, 81, 399, 1001])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_a_row_does_not_depend_on_its_neighbours(dtype, K, cuda_lib):
    """Bit for bit, the sign of zeros at masked places included: rows beside one whose gradient is infinite, and rows
    after a launch that leaves NaN in shared memory."""
    na = cuda_lib
    L = max(K, 37)   # 3 L rows: no whole number of a kernel's passes
    shape, kernel = (1, L, 3, K), (K,)
    x1, x2, dy = tb.logits(shape, dtype, 1, True).cuda(), tb.logits(shape, dtype, 2, True).cuda(), randn(shape, dtype, 3).cuda()
    lam = torch.rand(3, device="cuda")
    x1[0, 20, 1], x2[0, 20, 1] = 0.5, 0.25   # a row without masked places
    ill = dy.clone()
    ill[0, 20, 1] = float("inf")
    others = torch.ones(shape[:-1], dtype=torch.bool, device="cuda")
    others[0, 20, 1] = False

    def grads(dy):
        a, b, c, l = torch.empty_like(x1), torch.empty_like(x1), torch.empty_like(x1), torch.empty(shape[:-1], device="cuda")
        na.na_softmax_dropout_bwd(x1, dy, a, kernel, 0.0, None)
        na.na_diff_softmax_bwd(x1, x2, lam[None, None].expand(shape[:-1]).contiguous(), dy, b, c, l, kernel)
        return a, b, c, l

    def litter(value):   # every multiprocessor's shared memory
        t = torch.full((1, max(K, 400000 // K), 3, K), value, dtype=x1.dtype, device="cuda")
        na.na_softmax_dropout_bwd(t, t, torch.empty_like(t), kernel, 0.0, None)

    litter(0.0)
    ref = grads(dy)
    for got in (grads(ill), (litter(float("nan")), grads(dy))[1]):
        for name, g, r in zip(("dx", "dx1", "dx2", "dlam"), got, ref):
            assert torch.equal(bits(g)[others], bits(r)[others]), name
    assert torch.isnan(grads(ill)[0][0, 20, 1]).all()
    tb.status_ok(na)


@pytest.mark.gpu
def test_host_threads_with_rows_of_one_kernel(cuda_lib):
    """Rows of 363 and 383 weights are the same kernel's with different amounts of shared memory, both over what a launch
    has without asking; calls of several host threads do not take it from one another.  The library is called as it
    is, so that the threads meet there and not before."""
    na = cuda_lib
    call, stream = na.load().na_diff_softmax_bwd, torch.cuda.current_stream().cuda_stream
    start, failed, work = threading.Barrier(6), [], []
    for i in range(6):
        K = (363, 383)[i % 2]
        shape = (1, 400, 1, K)
        x1, x2, dy = (randn(shape, "bf16", i // 2 * 3 + j).cuda() for j in range(3))
        lam = torch.rand(shape[:-1], device="cuda")
        want, got = ([torch.empty_like(x1), torch.empty_like(x1), torch.empty_like(lam)] for _ in range(2))
        na.na_diff_softmax_bwd(x1, x2, lam, dy, *want, (K,))
        p = lambda t: t.data_ptr()
        args = (p(x1), p(x2), p(lam), 1, p(dy), *map(p, got), 1, 1, na._ints((400,)), 1, na._ints((K,)), 0.0, None, na.NA_BF16,
                None, 0, stream)
        work.append((args, want, got, (x1, x2, dy, lam)))
    torch.cuda.synchronize()

    def run(args):
        start.wait(60)
        failed.extend(st for st in (call(*args) for _ in range(4000)) if st)

    threads = [threading.Thread(target=run, args=(w[0],)) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    tb.status_ok(na)
    assert not failed, f"{len(failed)} calls refused, status {set(failed)}"
    for _, want, got, _ in work:
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.gpu
@pytest.mark.parametrize("case", tb.WIN, ids=tb.WIN_IDS)
def test_zeros_are_where_the_reference_has_them(case, cuda_lib):
    """Dropped and masked places are zero, and places whose weight is well within the type's range are not."""
    na = cuda_lib
    dtype, B, grid, heads, kernel = case
    shape = (B, *grid, heads, math.prod(kernel))
    x = tb.logits(shape, dtype, 21, True)
    y = torch.full_like(x, 5.0).cuda()
    na.na_softmax_dropout(x.cuda(), y, kernel, 0.2, tb.rng_state())
    tb.status_ok(na)
    ref = ob.softmax_dropout(f64(x), ob.dropout_factor(x.numel(), 0.2, tb.SEED, tb.OFFSET).reshape(shape))
    zero = f64(y) == 0
    assert zero[ref == 0].all()
    # exponentials under 2^-126 count as zero; a weight times the gain is at most 1.25 of its exponential
    assert not zero[ref > max(2.0 ** -120, torch.finfo(TYPES[dtype]).smallest_normal)].any()


# ---------------------------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("dtype,rows,C", [("bf16", 9, 33), ("fp32", 9, 63), ("fp16", 257, 7), ("fp32", 33, 3)])
def test_gradients_of_odd_rows_whose_last_is_not_finite(dtype, rows, C, cuda_lib):
    """An infinite value in the last row reaches its own column of dw and no other sum, and the weights' gradients
    do not depend on whether dx overwrites its inputs."""
    na = cuda_lib
    x, dy, w = randn((rows, C), dtype, 1), randn((rows, C), dtype, 2), 1 + 0.3 * randn((C,), "fp32", 3)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    x[-1, 0], dy[-1, 0] = float("inf"), 1.0
    xd, dyd, wd = x.cuda(), dy.cuda(), w.cuda()
    dx, dw, db = torch.empty_like(xd), torch.empty_like(wd), torch.empty_like(wd)
    na.na_layernorm_bwd(dyd, xd, wd, mean, rstd, dx, dw, db)
    assert torch.isposinf(dw[0])
    ref = (f64(dy) * np.where(np.isinf(f64(x)), 0, f64(x))).sum(0)
    close("dw", dw[1:], ref[1:], DEPTH * E * np.abs(f64(dy)[:, 1:] * f64(x)[:, 1:]).sum(0))
    close("db", db, f64(dy).sum(0), DEPTH * E * np.abs(f64(dy)).sum(0))
    # a row of dx that is not finite, written over the row of x that teams past the end read
    xd[-1, 0] = 0.5
    dyd[-1, -1] = float("inf")
    na.na_layernorm_bwd(dyd, xd, wd, mean, rstd, dx, dw, db)
    assert not torch.isfinite(dx[-1]).any() and torch.isfinite(dw[:-1]).all() and torch.isfinite(dx[:-1]).all()
    for _ in range(20):
        over, dw2, db2 = xd.clone(), torch.empty_like(dw), torch.empty_like(db)
        na.na_layernorm_bwd(dyd, over, wd, mean, rstd, over, dw2, db2)
        assert torch.equal(dw2, dw) and torch.equal(db2, db) and torch.equal(over[:-1], dx[:-1])
    tb.status_ok(na)


def norm_slack(g, h, r):
    """Error bound of dx, as in test_block_ops.py."""
    mean = lambda a: a.mean(-1, keepdims=True)
    c1, c2 = np.abs(mean(g)), np.abs(mean(g * h))
    return r * E * (8 * (np.abs(g) + c1 + np.abs(h) * c2) + (DEPTH + 8) * (mean(np.abs(g)) + np.abs(h) * mean(np.abs(g * h))))


def norm_grads_close(na, dtype, x, dy, w, mean, rstd):
    """dx, dw, db of one call against the reference at the given statistics.  A column's sum here: a thread's run of at
    most a dozen rows, then shuffles, warps and blocks, within DEPTH steps."""
    C = x.shape[-1]
    dx, dw, db = torch.full_like(x, 5.0), torch.full((C,), 9.0, device="cuda"), torch.full((C,), 9.0, device="cuda")
    na.na_layernorm_bwd(dy, x, w, mean, rstd, dx, dw, db)
    tb.status_ok(na)
    X, D, W, m, r = f64(x), f64(dy), f64(w), f64(mean), f64(rstd)
    rdx, rdw, rdb = ob.layernorm_bwd(D, X, W, m, r)
    h = (X - m[:, None]) * r[:, None]
    close("dx", dx, rdx, norm_slack(D * W, h, r[:, None]), TYPES[dtype])
    close("dw", dw, rdw, DEPTH * E * np.abs(D * h).sum(0))
    close("db", db, rdb, DEPTH * E * np.abs(D).sum(0))
    return dx, dw, db


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [1e-22, 1e22])
@pytest.mark.parametrize("dtype,rows,C", [
    ("bf16", 700, 32), ("fp32", 700, 200), ("bf16", 1600, 520), ("fp32", 1600, 520), ("bf16", 9, 2048), ("fp32", 9, 8192),
    ("bf16", 57, 65), ("fp32", 19, 7), ("fp32", 9, 1001)])
def test_gradients_of_very_small_and_large_spreads(dtype, rows, C, spread, cuda_lib):
    """rstd far from 1, its square past the range of fp32 (eps = 0, or statistics from elsewhere): the gradient's own terms
    are all within it."""
    x = (randn((rows, C), "fp32", 1).double() * spread).to(TYPES[dtype]).cuda()
    dy, w = randn((rows, C), dtype, 2).cuda(), (1 + 0.3 * randn((C,), "fp32", 3)).cuda()
    X = x.double()
    mean = X.mean(-1)
    rstd = (X - mean[:, None]).square().mean(-1).rsqrt().clamp(max=4 / spread)   # rows of few channels too
    norm_grads_close(cuda_lib, dtype, x, dy, w, mean.float(), rstd.float())


NORM_TURNS = [
    # dtype, rows, C, whether the gradients take the one launch of few wide rows
    # gradients of block-wide rows on both sides of that launch's limits, of every type and number of chunks to a thread
    ("fp32", 1536, 520, True), ("fp32", 1537, 520, False), ("fp32", 1537, 2048, False), ("fp32", 1537, 8192, False),
    ("fp16", 1536, 2048, True), ("fp16", 1537, 2048, False), ("bf16", 1537, 2048, False), ("bf16", 1537, 8192, False),
    ("fp32", 1024, 8192, True), ("fp32", 1025, 8192, False),
    # several turns of a block's loop: wide rows, odd rows, and rings of five tiles a block and more
    ("fp32", 2600, 2048, False), ("fp32", 1300, 8192, False), ("bf16", 6000, 2048, False), ("bf16", 3000, 1001, False),
    ("fp32", 3000, 1001, False), ("fp16", 1300, 4099, False), ("bf16", 20000, 33, False), ("bf16", 100000, 64, False),
    ("fp16", 100000, 40, False), ("fp32", 20000, 200, False), ("fp32", 60000, 72, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,rows,C,few", NORM_TURNS, ids=[str(c) for c in NORM_TURNS])
def test_layernorm_of_many_turns(dtype, rows, C, few, cuda_lib):
    na = cuda_lib
    assert (na.na_layernorm_bwd_workspace_size(rows, C, TYPES[dtype]) == 0) == few
    x = (randn((rows, C), "fp32", 1) * 1.5 + randn((rows, 1), "fp32", 2)).to(TYPES[dtype]).cuda()
    w, b = (1 + 0.3 * randn((C,), "fp32", 3)).cuda(), randn((C,), "fp32", 4).cuda()
    dy = randn((rows, C), dtype, 5).cuda()
    y, mean, rstd = torch.full_like(x, 5.0), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    na.na_layernorm(x, w, b, y, mean, rstd)
    tb.status_ok(na)
    X, W, Bv = f64(x), f64(w), f64(b)
    ry, rm, rr = ob.layernorm(X, W, Bv, float(np.float32(1e-5)))
    em = DEPTH * E * np.abs(X).mean(-1)
    er = (DEPTH + 8) * E + (em * rr) ** 2
    close("mean", mean, rm, em)
    close("rstd", rstd, rr, rr * er)
    h = np.abs(X - rm[:, None]) * rr[:, None]
    W = np.abs(W)
    close("y", y, ry, W * (rr * em)[:, None] + h * W * (er[:, None] + 8 * E) + 2 * E * np.abs(Bv), TYPES[dtype])
    dx, dw, db = norm_grads_close(na, dtype, x, dy, w, mean, rstd)
    z = x.clone()
    na.na_layernorm(z, w, b, z)
    assert torch.equal(z, y)
    for over in (0, 1):   # dx over x, over dy
        t = [x.clone(), dy.clone()]
        dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
        na.na_layernorm_bwd(t[1], t[0], w, mean, rstd, t[over], dw2, db2)
        assert torch.equal(t[over], dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
    tb.status_ok(na)


# ---------------------------------------------------------------------------------------------
# The binding
# ---------------------------------------------------------------------------------------------

BIG = 2 ** 32 + 7   # 7 to a C int
UNSUPPORTED = 2


@pytest.fixture(scope="module")
def lib():
    nabuild.build()
    return nab.load()


def test_sizes_past_32_bits_are_refused(lib, monkeypatch):
    """Every size that the library takes as a C int; the tensors have no memory, so no call could be launched."""
    monkeypatch.setattr(nab, "_launch_stream", lambda stream, *tensors: None)
    m = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="meta")
    f32 = torch.float32
    f = nab.RopeFreqs.scaled((16,))
    rope = lambda q, k: (q, k, q, k, f)
    bad = [
        (nab.na_rope, rope(m(1, BIG, 1, 16), None)), (nab.na_rope, rope(m(BIG, 1, 1, 16), None)),
        (nab.na_rope, rope(m(1, 1, BIG, 16), None)), (nab.na_rope_bwd, rope(m(1, 1, 1, 16), m(1, 1, BIG, 16))),
        (nab.na_rope, rope(m(1, 1, 1, BIG), None)),
        (nab.na_layernorm, (m(2, BIG), None, None, m(2, BIG))),
        (nab.na_layernorm_bwd, (m(2, BIG), m(2, BIG), None, m(2, dtype=f32), m(2, dtype=f32), m(2, BIG))),
    ]
    for shape, kernel in (((1, BIG, 1, 3), 3), ((BIG, 4, 1, 3), (3,)), ((1, 4, BIG, 3), (3,))):
        x, lam = m(*shape), m(*shape[:-1], dtype=f32)
        bad += [(nab.na_softmax_dropout, (x, x, kernel, 0.0, None)), (nab.na_softmax_dropout_bwd, (x, x, x, kernel, 0.0, None)),
                (nab.na_diff_softmax, (x, x, lam, x, kernel)), (nab.na_diff_softmax_bwd, (x, x, lam, x, x, x, lam, kernel))]
    for call, args in bad:
        with pytest.raises(nab.NAError) as e:
            call(*args)
        assert e.value.status == UNSUPPORTED, (call.__name__, [tuple(a.shape) for a in args if torch.is_tensor(a)])
    assert nab.na_layernorm_bwd_workspace_size(8, BIG) == 0
    assert nab.na_layernorm_bwd_workspace_size(BIG, 8) > 0          # rows are counted in 64 bits
    assert nab.na_diff_softmax_bwd_workspace_size(1, (BIG,), 1, (3,)) == 0
    assert nab.na_diff_softmax_bwd_workspace_size(BIG, (8,), 1, (3,)) == 0
    assert nab.na_diff_softmax_bwd_workspace_size(1, (8,), BIG, (3,)) == 0


def test_origins_past_64_bits_are_refused(lib, monkeypatch):
    monkeypatch.setattr(nab, "_launch_stream", lambda stream, *tensors: None)
    q = torch.empty((1, 4, 4, 1, 16), device="meta")
    for origin in (1 << 63, (0, -(1 << 63) - 1)):
        with pytest.raises(ValueError):
            nab.na_rope(q, None, q, None, nab.RopeFreqs.scaled((8, 8)), origin=origin)


def test_a_workspace_without_memory_of_its_own_is_refused():
    """A workspace's bytes are counted from its elements, so a broadcast view would promise more than there is."""
    for ws in (torch.empty(1, dtype=torch.uint8).expand(1 << 20), torch.empty(4, 4).t()):
        with pytest.raises(ValueError):
            nab._workspace(ws, None, lambda: 1 << 20, "cpu")
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    assert nab._workspace(ws, None, lambda: 1 << 20, "cpu") == (ws, ws.data_ptr(), 1 << 20)


@pytest.mark.gpu
def test_workspaces_elsewhere_are_refused(cuda_lib):
    """On the host, or a broadcast view of a few bytes: every call that takes a workspace raises before it launches."""
    na = cuda_lib
    e = torch.empty_like
    q = randn((1, 8, 8, 2, 32), "bf16", 1).cuda()
    lse = torch.zeros(q.shape[:-1], device="cuda")
    x, lam = randn((1, 8, 8, 2, 9), "bf16", 2).cuda(), torch.rand(2, device="cuda")
    rows, w, st = randn((64, 64), "bf16", 3).cuda(), torch.rand(64, device="cuda"), torch.ones(64, device="cuda")
    for ws in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 20)):
        for call in (lambda: na.na_bwd(q, q, q, q, q, lse, e(q), e(q), e(q), (3, 3), workspace=ws),
                     lambda: na.na_rpb_grad(x, torch.empty(2, 5, 5, device="cuda"), (3, 3), workspace=ws),
                     lambda: na.na_layernorm_bwd(rows, rows, w, st, st, e(rows), e(w), e(w), workspace=ws),
                     lambda: na.na_diff_softmax_bwd(x, x, lam, x, e(x), e(x), e(lam), (3, 3), workspace=ws)):
            with pytest.raises(ValueError):
                call()
    tb.status_ok(na)
