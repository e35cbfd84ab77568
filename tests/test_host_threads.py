"""Calls from host threads of the program's own, as a loader or a server makes them."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def bf16(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()


def attention(na, q, k, v, kernel):
    """The fused forward and gradients, and the unfused chain: [o, lse, dq, dk, dv, weights, sums, and their gradients]."""
    e = torch.empty_like
    o, lse, d = e(q), torch.empty(q.shape[:-1], device="cuda"), [e(q) for _ in range(3)]
    na.na_fwd(q, k, v, o, lse, kernel)
    na.na_bwd(q, k, v, o, v, lse, *d, kernel)
    K = kernel[0] * kernel[1]
    w, dw, av, dv, dq, dk = torch.empty(q.shape[:-1] + (K,), dtype=q.dtype, device="cuda"), None, e(q), e(q), e(q), e(q)
    na.na_qk(q, k, w, kernel)
    na.na_softmax(w, w, kernel)
    na.na_av(w, v, av, kernel)
    dw = e(w)
    na.na_av_bwd(q, w, v, dw, dv, kernel)
    na.na_qk_bwd(dw, q, k, dq, dk, kernel)
    return [o, lse, *d, w, av, dw, dv, dq, dk]


def test_the_first_calls_of_a_thread(cuda_lib):
    """A thread that has made no CUDA call yet gets what the main thread gets, bit for bit."""
    na = cuda_lib
    q, k, v = (bf16((1, 20, 24, 2, 32), i) for i in range(3))
    e = torch.empty_like
    ref = attention(na, q, k, v, (5, 5))
    o, lse = e(q), torch.empty(q.shape[:-1], device="cuda")
    w, av, dq, dk = e(ref[5]), e(q), e(q), e(q)
    torch.cuda.synchronize()
    calls = {   # each the first of a thread of its own; outputs made before
        "na_fwd": lambda: na.na_fwd(q, k, v, o, lse, (5, 5)),
        "na_qk": lambda: na.na_qk(q, k, w, (5, 5)),
        "na_av": lambda: na.na_av(ref[5], v, av, (5, 5)),
        "na_qk_bwd": lambda: na.na_qk_bwd(ref[7], q, k, dq, dk, (5, 5)),
    }
    failed = {}

    def run(name, call):
        try:
            call()
        except Exception as ex:   # noqa: BLE001  (handed to the test's own thread)
            failed[name] = ex

    for item in calls.items():
        t = threading.Thread(target=run, args=item)
        t.start()
        t.join()
    assert not failed, failed
    torch.cuda.synchronize()
    logits = e(w)
    na.na_qk(q, k, logits, (5, 5))
    for name, got, want in (("o", o, ref[0]), ("lse", lse, ref[1]), ("logits", w, logits), ("sums", av, ref[6]), ("dq", dq, ref[9]),
                            ("dk", dk, ref[10])):
        assert torch.equal(got, want), name


@pytest.mark.parametrize("what", ["na_softmax_bwd", "na_fwd"])
def test_sizes_of_one_kernel_at_once(what, cuda_lib):
    """Windows that are the same kernel's with different amounts of shared memory, over what a launch has without asking: calls
    of several host threads do not take it from one another.  The library is called as it is, so that the threads
    meet there and not before."""
    na = cuda_lib
    stream, p = torch.cuda.current_stream().cuda_stream, lambda t: t.data_ptr()
    work, check = [], []
    for i in range(6):
        if what == "na_softmax_bwd":
            K = (225, 255)[i % 2]
            y, dy = (bf16((1, 256, 2, K), i // 2 * 2 + j) for j in range(2))
            want, got = torch.empty_like(y), torch.empty_like(y)
            na.na_softmax_bwd(y, dy, want, (K,))
            keep = (y, dy)
            work.append((p(y), p(dy), p(got), 1, 1, na._ints((256,)), 2, na._ints((K,)), na.NA_BF16, stream))
        else:
            kernel = ((3, 3), (13, 13))[i % 2]
            q, k, v = (bf16((1, 32, 32, 2, 64), i // 2 * 3 + j) for j in range(3))
            want, got, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(q.shape[:-1], device="cuda")
            na.na_fwd(q, k, v, want, lse, kernel)
            keep = (q, k, v, lse)
            work.append((p(q), p(k), p(v), p(got), p(lse), 1, 2, na._ints((32, 32)), 2, 64, na._ints(kernel), na._ints((1, 1)), 0.125,
                         na.NA_BF16, stream))
        check.append((want, got, keep))
    torch.cuda.synchronize()
    call, start, failed = getattr(na.load(), what), threading.Barrier(6), []

    def run(args):
        start.wait(60)
        failed.extend(st for st in (call(*args) for _ in range(4000)) if st)

    threads = [threading.Thread(target=run, args=(args,)) for args in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, f"{len(failed)} calls refused, status {set(failed)}"
    for want, got, _ in check:
        assert torch.equal(want, got)
