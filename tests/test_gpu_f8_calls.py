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


def captured(rg, run, stream):  # noqa: F811
    """(graph, outputs) of run(), captured on a stream that has run it before."""
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = run()
    return graph, outs


def exact_and_f8(rg, seed):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(seed)
    A, B = (torch.randint(-(2**20), 2**20, s, generator=g, device="cuda") for s in ((130, 70), (70, 200)))
    rest = steps(rg, seed)
    return lambda: (rg.res_gemm_i64(A, B, sync=False), *rest())


@pytest.mark.parametrize("drop", [True, False])
def test_graph_keeps_its_scratch(rg, drop):  # noqa: F811
    """A graph replays in scratch of its own after the capture stream's workspace was replaced or dropped and its
    memory went to other tensors, which stay as they are."""
    run, stream = exact_and_f8(rg, 5), torch.cuda.Stream()
    want = [t.clone() for t in run()]
    graph, outs = captured(rg, run, stream)
    with torch.cuda.stream(stream):
        old = rg.workspace(4096, outs[0].device).numel()
        if drop:
            rg.release_workspaces()
        else:
            rg.workspace(4 * old, outs[0].device)
        fill = [torch.full((old,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
        for t in outs:
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert all(bool((f == 7).all()) for f in fill)


def test_graphs_replay_at_the_same_time(rg):  # noqa: F811
    """Graphs captured on one stream share no scratch: replayed on two streams at once they give what they give alone."""
    stream, others = torch.cuda.Stream(), [torch.cuda.Stream(), torch.cuda.Stream()]
    runs = [exact_and_f8(rg, 11), exact_and_f8(rg, 31)]
    want = [[t.clone() for t in run()] for run in runs]
    graphs = [captured(rg, run, stream) for run in runs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (graph, outs), s in zip(graphs, others):
            with torch.cuda.stream(s):
                for t in outs:
                    t.zero_()
                graph.replay()
    torch.cuda.synchronize()
    for (_, outs), w in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, w))


def test_status_of_a_captured_call(rg):  # noqa: F811
    """The caller's workspace serves a captured step, eager calls of the same tensors, and the status afterwards."""
    x, w, dy = normal((70, 200), 1).cuda(), normal((96, 200), 2).cuda(), normal((70, 96), 3).cuda()
    ws = torch.empty(rg.library().linear_f8_ws_bytes(70, 96, 200), dtype=torch.uint8, device="cuda")

    def step(**kw):
        y, saved = rg.linear_f8(x, w, sync=False, **kw)
        return (y, *rg.linear_f8_backward(dy, saved, sync=False, **kw))

    want = step()
    graph, outs = captured(rg, lambda: step(ws=ws), torch.cuda.Stream())
    graph.replay()
    assert rg.status(ws) == rg.RG_OK
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("dtype,wtype", [(torch.bfloat16, torch.float32), (torch.float16, torch.bfloat16),
                                         (torch.float32, torch.float16)])
def test_linear_has_a_gradient(rg, dtype, wtype):  # noqa: F811
    """autograd through linear_f8 gives what linear_f8_backward gives, for either input alone too."""
    x, w = normal((70, 200), 1, 1.0, dtype).cuda(), normal((96, 200), 2, 0.1, wtype).cuda()
    dy = normal((70, 96), 3, 1.0, dtype).cuda()
    want, saved = rg.linear_f8(x, w)
    dx, dw = rg.linear_f8_backward(dy, saved, dw_dtype=wtype)
    for needs in ((True, True), (True, False), (False, True)):
        a, b = (t.clone().requires_grad_(n) for t, n in zip((x, w), needs))
        y, kept = rg.linear_f8(a, b, sync=False)
        assert y.requires_grad and torch.equal(y, want)
        assert all(torch.equal(p, q) for p, q in zip(rg.linear_f8_backward(dy, kept, dw_dtype=wtype), (dx, dw)))
        y.backward(dy)
        for t, n, g in ((a, needs[0], dx), (b, needs[1], dw)):
            assert (t.grad is not None) == n and (not n or (t.grad.dtype == t.dtype and torch.equal(t.grad, g)))
        with torch.no_grad():
            y, _ = rg.linear_f8(a, b)
        assert not y.requires_grad and torch.equal(y, want)
    a = x.clone().requires_grad_()
    (grad,) = torch.autograd.grad(rg.linear_f8(a, w)[0].sum(), a)  # an expanded gradient
    assert torch.equal(grad, rg.linear_f8_backward(torch.ones_like(want), saved)[0])


def test_calls_without_a_gradient_do_not_cut_it_silently(rg):  # noqa: F811
    x, w = normal((5, 256), 1).cuda(), normal((96, 256), 2).cuda()
    q, s = rg.quantize_f8(x)
    qw, sw = rg.quantize_f8(w, "tiles")
    args = [a.cuda() for a in moe_inputs(5, 256, 64, 8, torch.bfloat16, 3)]
    gemm = lambda sa, **kw: rg.scaled_gemm_f8(q, sa, qw, sw, transb=True, **kw)  # noqa: E731
    experts = lambda t, **kw: rg.moe_layer_f8(t, *args[1:], 2, **kw)  # noqa: E731
    for call, t in ((gemm, s), (experts, args[0])):
        want, needs = call(t), t.clone().requires_grad_()
        y = call(needs, sync=False)
        assert torch.equal(y, want) and y.requires_grad
        with pytest.raises(NotImplementedError):
            y.sum().backward()
        with pytest.raises(ValueError):
            call(needs, out=torch.empty_like(want))
        with torch.no_grad():
            out = torch.empty_like(want)
            assert call(needs, out=out) is out and torch.equal(out, want)
            assert not call(needs).requires_grad


def test_few_row_product_clears_an_earlier_time_out(rg):  # noqa: F811
    """Both words of an earlier call's time-out, the status and where it happened, are gone after the next call."""
    lib = rg.library()
    q, s = rg.quantize_f8(normal((300, 256), 1).cuda())
    qw, sw = rg.quantize_f8(normal((256, 256), 2).cuda(), "tiles")
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    words = lambda: (int(ws[:4].view(torch.int32)), int(ws[136:140].view(torch.int32)))  # noqa: E731
    old = lib.rg_set_wait_limit_ns(50_000_000)
    try:
        lib.rg_inject_fault(1)
        with pytest.raises(rg.ResGemmError):
            rg.scaled_gemm_f8(q, s, qw, sw, transb=True, ws=ws)
        assert words()[0] == rg.RG_ERR_TIMEOUT and words()[1] != 0
    finally:
        lib.rg_inject_fault(0)
        lib.rg_set_wait_limit_ns(old)
    rg.scaled_gemm_f8(q[:3], s[:3], qw, sw, transb=True, ws=ws)
    assert words() == (0, 0)
