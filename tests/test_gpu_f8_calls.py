"""How the 8-bit operators are called: from several host threads, under graph capture, with tensors that require
gradients, and what they report."""
import threading
import weakref

import pytest
import torch

from gpu_util import rg  # noqa: F401
from test_gpu_f8 import moe_inputs, normal

pytestmark = pytest.mark.gpu


def steps(rg, seed):  # noqa: F811
    """A training step and an expert layer on inputs of their own: a call of several launches each."""
    x = normal((300, 256), seed, 1.0, torch.bfloat16).cuda()
    w, dy = normal((200, 256), seed + 1).cuda(), normal((300, 200), seed + 2, 0.1, torch.bfloat16).cuda()
    args = [a.cuda() for a in moe_inputs(5 + seed % 3, 256, 64, 8, torch.bfloat16, seed)]

    def run():
        y, saved = rg.linear_f8(x, w, sync=False)
        return (y, *rg.linear_f8_backward(dy, saved, sync=False), rg.moe_layer_f8(*args, 2, sync=False))

    return run


def test_threads_on_one_stream(rg):  # noqa: F811
    """Each thread's calls give what they give alone, although all share the default stream's workspace."""
    runs = [steps(rg, 100 * i) for i in range(4)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    got = [[] for _ in runs]
    start = threading.Barrier(len(runs))

    def work(i):
        start.wait()
        for _ in range(50):
            got[i].append(runs[i]())

    ts = [threading.Thread(target=work, args=(i,)) for i in range(len(runs))]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert len(g) == 50
        for outs in g:
            assert all(torch.equal(a, b) for a, b in zip(w, outs))


@pytest.mark.parametrize("m", [4, 70, 2100])
def test_product_is_a_threads_first_call(rg, m):  # noqa: F811
    """A host thread whose first use of the GPU is a product, by each of the product's kernels."""
    q, s = rg.quantize_f8(normal((m, 200), 1).cuda())
    qw, sw = rg.quantize_f8(normal((2304, 200), 2).cuda(), "tiles")
    want, out = rg.scaled_gemm_f8(q, s, qw, sw, transb=True), []
    t = threading.Thread(target=lambda: out.append(rg.scaled_gemm_f8(q, s, qw, sw, transb=True)))
    t.start()
    t.join()
    assert len(out) == 1 and torch.equal(out[0], want)


def test_a_call_keeps_its_workspace(rg):  # noqa: F811
    """A workspace that another thread drops from the cache lives until the calls that use it have ended."""
    x, w = normal((70, 200), 1).cuda(), normal((96, 200), 2).cuda()
    q, s = rg.quantize_f8(x)
    qw, sw = rg.quantize_f8(w, "tiles")
    Y, saved = rg.linear_f8(x, w)
    calls = (lambda: rg.linear_f8(x, w)[0], lambda: rg.linear_f8_backward(Y, saved)[0],
             lambda: rg.scaled_gemm_f8(q, s, qw, sw, transb=True))
    want = [f() for f in calls]
    for f, y in zip(calls, want):
        f()  # fills the cache again
        ws = rg.workspace(4096, x.device)
        p, alive, out = ws.data_ptr(), weakref.ref(ws), []
        del ws
        assert rg.library().rg_hold_workspace(p, 1) == rg.RG_OK
        try:
            t = threading.Thread(target=lambda: out.append(f()))
            t.start()
            t.join(0.3)
            assert t.is_alive()  # in the library, waiting for its turn
            rg.release_workspaces()
            assert alive() is not None
        finally:
            assert rg.library().rg_hold_workspace(p, 0) == rg.RG_OK
        t.join()
        assert alive() is None and torch.equal(out[0], y)
