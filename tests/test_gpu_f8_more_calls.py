"""How the 8-bit products by group and with an epilogue are called: from several host threads, on other streams, under
graph capture, with gradients, one after another."""
import threading
import weakref

import pytest
import torch

from gpu_util import rg  # noqa: F401
from test_gpu_f8 import normal
from test_gpu_f8_calls import captured
from test_gpu_f8_grouped import offsets_of

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


def steps(rg, seed, counts=(30, 0, 140, 5), k=256, n=200):  # noqa: F811
    """A training step of each layer and a product of each kind, on inputs of their own."""
    t = sum(counts)
    x, r = normal((t, k), seed, 1.0, bf).cuda(), normal((t, n), seed + 5, 1.0, bf).cuda()
    w, dy = normal((n, k), seed + 1, 0.1).cuda(), normal((t, n), seed + 2, 0.1, bf).cuda()
    we, b = normal((len(counts), n, k), seed + 3, 0.1).cuda(), normal((n,), seed + 4).cuda()
    off = offsets_of(counts)
    qx, sx = rg.quantize_f8(x)
    qw, sw = rg.quantize_f8(w, "tiles")
    qe, se = rg.quantize_f8(we, "tiles")

    def run():
        y, saved = rg.linear_act_f8(x, w, bias=b, act="gelu", residual=r, sync=False)
        z, kept = rg.expert_linear_f8(x, we, off, sync=False)
        return (y, *rg.linear_act_f8_backward(dy, saved, sync=False), z,
                *rg.expert_linear_f8_backward(dy, kept, sync=False),
                rg.scaled_gemm_act_f8(qx[:3], sx[:3], qw, sw, bias=b, act="silu", sync=False),
                rg.grouped_gemm_f8(qx, sx, qe, se, off, transb=True, sync=False))

    return run


def test_threads_on_one_stream(rg):  # noqa: F811
    """Each thread's calls give what they give alone, although all share the default stream's workspace."""
    runs = [steps(rg, 100 * i, (30 + 40 * i, 0, 140, 5)) for i in range(4)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    got = [[] for _ in runs]
    start = threading.Barrier(len(runs))

    def work(i):
        start.wait()
        for _ in range(30):
            got[i].append(runs[i]())

    ts = [threading.Thread(target=work, args=(i,)) for i in range(len(runs))]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert len(g) == 30
        for outs in g:
            assert all(torch.equal(a, b) for a, b in zip(w, outs))


def test_streams_at_once(rg):  # noqa: F811
    """The same calls on four streams at once, each with a workspace of its own."""
    run, streams = steps(rg, 7), [torch.cuda.Stream() for _ in range(4)]
    want = run()
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(run())
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(want, o))


@pytest.mark.parametrize("per", [3, 600])
def test_product_is_a_threads_first_call(rg, per):  # noqa: F811
    """A host thread whose first use of the GPU is a product, by each of the kernels."""
    off = offsets_of([per, per])
    x = normal((2 * per, 200), 1).cuda()
    q, s, qt, st = rg.quantize_f8(x, "both", offsets=off)
    qw, sw = rg.quantize_f8(normal((2, 300, 200), 2).cuda(), "tiles")
    for call in (lambda: rg.grouped_gemm_f8(q, s, qw, sw, off, transb=True),
                 lambda: rg.grouped_wgrad_f8(qt, st, qt, st, off),
                 lambda: rg.scaled_gemm_act_f8(q, s, qw[0], sw[0], act="silu")):
        want, out = call(), []
        t = threading.Thread(target=lambda: out.append(call()))
        t.start()
        t.join()
        assert len(out) == 1 and torch.equal(out[0], want)


def test_a_call_keeps_its_workspace(rg):  # noqa: F811
    """A workspace that another thread drops from the cache lives until the calls that use it have ended."""
    off = offsets_of([30, 40])
    x, w, we = normal((70, 200), 1).cuda(), normal((96, 200), 2).cuda(), normal((2, 96, 200), 3).cuda()
    q, s, qt, st = rg.quantize_f8(x, "both", offsets=off)
    qw, sw = rg.quantize_f8(w, "tiles")
    qe, se = rg.quantize_f8(we, "tiles")
    Y, saved = rg.linear_act_f8(x, w, act="silu")
    Z, kept = rg.expert_linear_f8(x, we, off)
    calls = (lambda: rg.scaled_gemm_act_f8(q, s, qw, sw, act="silu"), lambda: rg.linear_act_f8(x, w, act="silu")[0],
             lambda: rg.linear_act_f8_backward(Y, saved)[0], lambda: rg.grouped_gemm_f8(q, s, qe, se, off, transb=True),
             lambda: rg.grouped_wgrad_f8(qt, st, qt, st, off), lambda: rg.expert_linear_f8(x, we, off)[0],
             lambda: rg.expert_linear_f8_backward(Z, kept)[1])
    rg.release_workspaces()  # one that a failed call of an earlier test still holds in its traceback
    for f in calls:
        want = f()  # fills the cache again
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
        assert alive() is None and torch.equal(out[0], want)


def test_graphs_replay_at_the_same_time(rg):  # noqa: F811
    """Graphs captured on one stream share no scratch: replayed on two streams at once they give what they give alone,
    also after the capture stream's workspace has gone to other tensors."""
    stream, others = torch.cuda.Stream(), [torch.cuda.Stream(), torch.cuda.Stream()]
    runs = [steps(rg, 11), steps(rg, 31, (200, 3, 0, 9))]
    want = [[t.clone() for t in run()] for run in runs]
    graphs = [captured(rg, run, stream) for run in runs]
    rg.release_workspaces()
    fill = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
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
    assert all(bool((f == 7).all()) for f in fill)


@pytest.mark.parametrize("per", [4, 500])
def test_graph_follows_its_offsets(rg, per):  # noqa: F811
    """A captured step serves other group sizes: the offsets are read when the graph runs."""
    counts = [per, 0, 2 * per, per // 2]
    t = sum(counts)
    x, w, dy = normal((t, 130), 1, 1.0, bf).cuda(), normal((4, 96, 130), 2, 0.1).cuda(), normal((t, 96), 3, 1.0, bf).cuda()
    off = offsets_of(counts)

    def step():
        y, saved = rg.expert_linear_f8(x, w, off, sync=False)
        return (y, *rg.expert_linear_f8_backward(dy, saved, sync=False))

    graph, outs = captured(rg, step, torch.cuda.Stream())
    for counts in ([0, t, 0, 0], [1, 1, 1, 1], [per, per, per, per // 2], [0, 0, 0, 0]):
        off.copy_(offsets_of(counts))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_captured_status(rg):  # noqa: F811
    """The caller's workspace serves a captured step and its status, bad offsets among it."""
    x, w, dy = normal((70, 200), 1).cuda(), normal((2, 96, 200), 2).cuda(), normal((70, 96), 3).cuda()
    off = offsets_of([30, 40])
    ws = torch.empty(rg.library().expert_linear_f8_ws_bytes(70, 96, 200, 2), dtype=torch.uint8, device="cuda")

    def step(**kw):
        y, saved = rg.expert_linear_f8(x, w, off, sync=False, **kw)
        return (y, *rg.expert_linear_f8_backward(dy, saved, sync=False, **kw))

    want = step()
    graph, outs = captured(rg, lambda: step(ws=ws), torch.cuda.Stream())
    graph.replay()
    assert rg.status(ws) == rg.RG_OK and all(torch.equal(a, b) for a, b in zip(outs, want))
    off[1] = 80
    graph.replay()
    assert rg.status(ws) == rg.RG_ERR_ARG
    off[1] = 30
    for t in outs:
        t.zero_()
    graph.replay()
    assert rg.status(ws) == rg.RG_OK and all(torch.equal(a, b) for a, b in zip(outs, want))


def layer(rg, seed):  # noqa: F811
    """A feed-forward layer with a residual, and experts behind it, as leaves and a function of them."""
    g = [normal(s, seed + i, 0.1, d).cuda().requires_grad_() for i, (s, d) in enumerate(
        [((300, 128), torch.float32), ((300,), bf), ((128, 300), torch.float32), ((3, 128, 128), torch.float32)])]
    x, off = normal((100, 128), seed + 9, 1.0, bf).cuda(), offsets_of([20, 0, 80])

    def loss(w1, b1, w2, we):
        h, _ = rg.linear_act_f8(x, w1, bias=b1, act="gelu_tanh", sync=False)
        y, _ = rg.linear_act_f8(h, w2, residual=x, sync=False)
        z, _ = rg.expert_linear_f8(y, we, off, sync=False)
        return z.float().square().mean()

    return g, loss


def test_layers_train_together(rg):  # noqa: F811
    """A run of the layers as they are used: its gradients are those of the calls one after another."""
    (w1, b1, w2, we), loss = layer(rg, 1)
    loss(w1, b1, w2, we).backward()
    x, off = normal((100, 128), 10, 1.0, bf).cuda(), offsets_of([20, 0, 80])
    with torch.no_grad():
        h, s1 = rg.linear_act_f8(x, w1, bias=b1, act="gelu_tanh")
        y, s2 = rg.linear_act_f8(h, w2, residual=x)
        z, s3 = rg.expert_linear_f8(y, we, off)
        dz = (z.float() * (2 / z.numel())).to(bf)
        dy, dwe = rg.expert_linear_f8_backward(dz, s3)
        dh, dw2, none = rg.linear_act_f8_backward(dy, s2)
        _, dw1, db1 = rg.linear_act_f8_backward(dh, s1)
    assert none is None
    for t, g in ((w1, dw1), (b1, db1), (w2, dw2), (we, dwe)):
        assert t.grad.dtype == t.dtype and torch.equal(t.grad, g)


def test_captured_backward_pass(rg):  # noqa: F811
    """A whole training step in a graph.  While a graph of the same leaves from another stream lives, the capture is
    refused before anything is enqueued; freed, it goes through."""
    leaves, loss = layer(rg, 20)
    want = torch.autograd.grad(loss(*leaves), leaves)
    stream = torch.cuda.Stream()
    alive = loss(*leaves)

    def capture():
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            for t in leaves:
                t.grad = None
            loss(*leaves).backward()
        return graph

    with pytest.raises(RuntimeError, match="free that graph"):
        capture()
    torch.cuda.synchronize()
    assert torch.isfinite(alive)
    del alive
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        loss(*leaves).backward()  # the stream's workspace and the grads
    torch.cuda.synchronize()
    graph = capture()
    for t in leaves:
        t.grad.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(t.grad, g) for t, g in zip(leaves, want))


def test_repeats_are_equal(rg):  # noqa: F811
    """No result depends on the order in which anything arrives."""
    run = steps(rg, 3, (700, 0, 257, 1000), 640, 520)
    want = run()
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(run(), want))


def test_offsets_on_another_type_or_layout(rg):  # noqa: F811
    x, w = normal((70, 200), 1).cuda(), normal((2, 96, 200), 2).cuda()
    off = offsets_of([30, 40])
    want = rg.expert_linear_f8(x, w, off)[0]
    for o in (off.long(), torch.stack((off, off), 1)[:, 0], torch.stack((off.long(), off.long()), 1)[:, 1]):
        assert torch.equal(rg.expert_linear_f8(x, w, o)[0], want)
        y, saved = rg.expert_linear_f8(x, w, o)
        assert all(torch.isfinite(t).all() for t in rg.expert_linear_f8_backward(y, saved))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("k", [512, 508, 510, 505, 260, 9])
def test_quantise_on_every_boundary(rg, k, dtype):  # noqa: F811
    """Rows 0, 1, 2, 4 entries off 16-byte boundaries: what the same rows on them give."""
    m = 300
    x = normal((m, k), 5, 1.0, dtype).cuda()
    even = torch.zeros((m, 520), dtype=dtype, device="cuda")[:, :k]
    even.copy_(x)
    offsets = torch.tensor([0, 100, 100, 290], device="cuda")
    calls = [(form, off) for form in ("rows", "columns", "both") for off in (None, offsets)
             if not (form == "rows" and off is not None)] + [("tiles", None)]
    for form, off in calls:
        want = rg.quantize_f8(even, form, offsets=off)
        for shift in (0, 1, 2, 4):
            for width in (k, k + 16 - k % 8):
                buf = torch.full((m * width + 8,), float("nan"), dtype=dtype, device="cuda")
                odd = buf[shift : shift + m * width].view(m, width)[:, :k]
                odd.copy_(x)
                for a, b in zip(rg.quantize_f8(odd, form, offsets=off), want):
                    assert torch.equal(a.float(), b.float())
