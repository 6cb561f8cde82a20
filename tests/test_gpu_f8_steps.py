"""Training steps of the 8-bit layers at the ends of their ranges: infinite values before an activation, sums over rows
on both sides of a cluster, gradients that are not wanted, offsets that change between the passes, captures."""
import math

import pytest
import torch

from gpu_util import rg  # noqa: F401
from test_gpu_f8 import normal
from test_gpu_f8_act import ACTS, layer_inputs
from test_gpu_f8_act import test_layer_gradients as check_layer_gradients

pytestmark = pytest.mark.gpu
bf, f16, f32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype,big", [(f16, 7e4), (f16, math.inf), (bf, math.inf), (f32, math.inf)])
def test_slopes_of_infinite_values(rg, dtype, big, act):  # noqa: F811
    """Values before the activation that are kept as infinities (fp16: finite ones beyond 65504) have the slopes of
    large ones, 0 or 1, and leave every gradient finite."""
    m, n, k = 150, 200, 72
    x, w, b, dy = layer_inputs(m, n, k, dtype)
    b = b.float()
    b[::5], b[2::7] = -big, big
    near = b.clamp(-6e4, 6e4)
    _, saved = rg.linear_act_f8(x, w, bias=b, act=act)
    got = rg.linear_act_f8_backward(dy, saved)
    _, saved = rg.linear_act_f8(x, w, bias=near, act=act)
    for g, want in zip(got, rg.linear_act_f8_backward(dy, saved)):
        assert torch.isfinite(g).all() and torch.equal(g, want)
    ref = dy.double().sum(0)
    tol = (m / 8 + 24) * 2.0**-24 * dy.double().abs().sum(0)
    assert ((got[2] - ref).abs() <= tol)[2::7].all()
    if act is not None:
        gone = torch.ones(n, dtype=torch.bool)[::5]
        gone[[i for i in range(len(gone)) if (5 * i) % 7 == 2]] = False  # overwritten by +big
        assert (got[2][::5][gone] == 0).all()


def test_status_of_two_products_at_once(rg):  # noqa: F811
    """The weight gradient's kernel may run beside the input gradient's, whose first block clears the status for both:
    what either reports stays."""
    x, w, dy = normal((40, 128), 1, 1.0, bf).cuda(), normal((2, 96, 128), 2, 0.1).cuda(), normal((40, 96), 3, 1.0, bf).cuda()
    off = torch.tensor([0, 10, 40], dtype=torch.int32, device="cuda")
    ws = torch.empty(rg.library().expert_linear_f8_ws_bytes(40, 96, 128, 2), dtype=torch.uint8, device="cuda")
    _, (kept, _, *rest) = rg.expert_linear_f8(x, w, off, ws=ws)
    bad = torch.tensor([0, 50, 40], dtype=torch.int32, device="cuda")
    for i in range(100):
        at, code = (bad, rg.RG_ERR_ARG) if i % 3 else (off, rg.RG_OK)
        rg.expert_linear_f8_backward(dy, (kept, at, *rest), sync=False, ws=ws)
        assert rg.status(ws) == code


def layers(rg, seed):  # noqa: F811
    """Leaves, and a loss of them through each of the layers."""
    w1, b1, w2, w3, we = (normal(s, seed + i, 0.1, d).cuda().requires_grad_() for i, (s, d) in enumerate(
        [((200, 128), f32), ((200,), bf), ((128, 200), f32), ((96, 128), bf), ((3, 64, 96), f32)]))
    x, off = normal((70, 128), seed + 9, 1.0, bf).cuda(), torch.tensor([0, 20, 20, 70], device="cuda")

    def out():
        h, _ = rg.linear_act_f8(x, w1, bias=b1, act="silu", sync=False)
        y, _ = rg.linear_act_f8(h, w2, residual=x, sync=False)
        z, _ = rg.linear_f8(y, w3, sync=False)
        return rg.expert_linear_f8(z, we, off, sync=False)[0]

    return (w1, b1, w2, w3, we), out


def test_capture_beside_a_living_graph_of_a_side_stream(rg):  # noqa: F811
    """Warm-up on a side stream, whose last output and loss stay variables, then the capture on a stream of its own."""
    leaves, out = layers(rg, 1)
    want = torch.autograd.grad(out().float().square().mean(), leaves)
    side, own = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            for t in leaves:
                t.grad = None
            y = out()
            loss = y.float().square().mean()
            loss.backward()
    torch.cuda.synchronize()
    for t in leaves:
        t.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=own):
        out().float().square().mean().backward()
    for t in leaves:
        t.grad.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.isfinite(loss.detach()) and all(torch.equal(t.grad, g) for t, g in zip(leaves, want))


def test_captured_forward_pass_with_gradients_enabled(rg):  # noqa: F811
    """Nothing is accumulated: a living graph of the default stream is no reason to refuse it."""
    _, out = layers(rg, 20)
    alive = out()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        y = out()
    graph.replay()
    torch.cuda.synchronize()
    assert y.requires_grad and torch.equal(y, alive)


@pytest.mark.parametrize("on_default", [False, True])
def test_capture_with_a_node_that_is_held_for_good(rg, on_default):  # noqa: F811
    """As data-parallel wrappers hold them: the stream on which the layers first met the leaf decides."""
    leaves, out = layers(rg, 40)
    want = torch.autograd.grad(out().float().square().mean(), leaves)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(torch.cuda.default_stream() if on_default else side):
        held = [torch.autograd.graph.get_gradient_edge(t).node for t in leaves]
        out().float().square().mean().backward()
    torch.cuda.synchronize()
    for t in leaves:
        t.grad = None

    def capture():
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out().float().square().mean().backward()
        return graph

    if on_default:
        for _ in range(2):
            with pytest.raises(RuntimeError, match="default stream"):
                capture()
        torch.cuda.synchronize()
        del held
    graph = capture()
    for t in leaves:
        t.grad.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(t.grad, g) for t, g in zip(leaves, want))


def test_differentiable_calls_read_the_nodes_off_their_results(rg, monkeypatch):  # noqa: F811
    """A leaf's accumulation node by way of the leaf is a view of it, 12 us; no call does that."""
    leaves, out = layers(rg, 60)
    for name in ("get_gradient_edge", "_get_grad_fn_or_grad_acc"):
        monkeypatch.setattr(torch.autograd.graph, name, None, raising=False)
    views = []
    monkeypatch.setattr(torch.Tensor, "view_as", lambda t, other: views.append(t), raising=True)
    y = out()
    monkeypatch.undo()
    assert not views
    assert all(t.grad is None for t in leaves)
    y.float().square().mean().backward()
    assert all(torch.isfinite(t.grad).all() for t in leaves)


@pytest.mark.parametrize("m", [70, 1100])
@pytest.mark.parametrize("act", [None, "relu", "gelu"])
def test_gradients_that_are_not_wanted(rg, act, m):  # noqa: F811
    """Each subset of the gradients is that part of all of them, by the native and by the general call path."""
    x, w, b, dy = layer_inputs(m, 136, 264, bf)
    _, saved = rg.linear_act_f8(x, w, bias=b, act=act)
    grads = rg.linear_act_f8_backward(dy, saved)
    ws = torch.empty(rg.library().linear_act_f8_ws_bytes(m, 136, 264), dtype=torch.uint8, device="cuda")
    for n in range(8):
        need = (bool(n & 1), bool(n & 2), bool(n & 4))
        for kw in ({}, {"ws": ws}):
            got = rg.linear_act_f8_backward(dy, saved, dx=need[0], dw=need[1], db=need[2], **kw)
            for g, want, wanted in zip(got, grads, need):
                assert torch.equal(g, want) if wanted else g is None
    _, saved = rg.linear_act_f8(x, w, act=act)  # without a bias
    dx, dw, _ = rg.linear_act_f8_backward(dy, saved)
    assert torch.equal(rg.linear_act_f8_backward(dy, saved, dw=False)[0], dx)
    assert torch.equal(rg.linear_act_f8_backward(dy, saved, dx=False)[1], dw)
    if act is None:
        _, saved = rg.linear_f8(x, w)
        ws = torch.empty(rg.library().linear_f8_ws_bytes(m, 136, 264), dtype=torch.uint8, device="cuda")
        for kw in ({}, {"ws": ws}):
            assert torch.equal(rg.linear_f8_backward(dy, saved, dw=False, **kw)[0], dx)
            assert torch.equal(rg.linear_f8_backward(dy, saved, dx=False, **kw)[1], dw)
            assert rg.linear_f8_backward(dy, saved, dx=False, dw=False, **kw) == (None, None)


@pytest.mark.parametrize("counts", [(3, 0, 70, 50), (300, 0, 0, 257), (0, 0, 0, 0)])
def test_expert_gradients_that_are_not_wanted(rg, counts):  # noqa: F811
    t = sum(counts) + 5
    x, w, dy = normal((t, 200), 1, 1.0, bf).cuda(), normal((4, 96, 200), 2, 0.1).cuda(), normal((t, 96), 3, 1.0, bf).cuda()
    off = torch.tensor([0, *torch.tensor(counts).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    _, saved = rg.expert_linear_f8(x, w, off)
    dx, dw = rg.expert_linear_f8_backward(dy, saved)
    ws = torch.empty(rg.library().expert_linear_f8_ws_bytes(t, 96, 200, 4), dtype=torch.uint8, device="cuda")
    for kw in ({}, {"ws": ws}):
        got = rg.expert_linear_f8_backward(dy, saved, dw=False, **kw)
        assert torch.equal(got[0], dx) and got[1] is None
        got = rg.expert_linear_f8_backward(dy, saved, dx=False, **kw)
        assert got[0] is None and torch.equal(got[1], dw)
        assert rg.expert_linear_f8_backward(dy, saved, dx=False, dw=False, **kw) == (None, None)
    kept, _, *rest = saved
    bad = torch.tensor([0, 5, 4, 4, 4], dtype=torch.int32, device="cuda")
    for kw in ({"dx": False}, {"dw": False}):  # each product reports
        with pytest.raises(rg.ResGemmError) as err:
            rg.expert_linear_f8_backward(dy, (kept, bad, *rest), **kw)
        assert err.value.code == rg.RG_ERR_ARG


def test_frozen_weights_take_no_memory(rg):  # noqa: F811
    """No gradient of frozen weights is made and dropped."""
    x, dy = normal((64, 1024), 1, 1.0, bf).cuda().requires_grad_(), normal((64, 1024), 2, 1.0, bf).cuda()
    we, w = torch.randn((8, 1024, 1024), device="cuda"), torch.randn((1024, 1024), device="cuda")
    r = normal((64, 1024), 3, 1.0, bf).cuda().requires_grad_()
    off = torch.arange(0, 65, 8, device="cuda")
    for call, most in ((lambda: rg.expert_linear_f8(x, we, off)[0], we.numel()), (lambda: rg.linear_f8(x, w)[0], w.numel()),
                       (lambda: rg.linear_act_f8(x, w, act="silu")[0], w.numel()),
                       (lambda: rg.linear_act_f8(x.detach(), w, residual=r)[0], x.numel())):
        for _ in range(2):  # the workspace first
            y = call()
            torch.cuda.synchronize()
            before = torch.cuda.memory_allocated()
            torch.cuda.reset_peak_memory_stats()
            y.backward(dy)
            assert torch.cuda.max_memory_allocated() - before < max(most, 1 << 20)
            x.grad = r.grad = None


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
@pytest.mark.parametrize("general", [False, True])
def test_offsets_are_rewritten_between_the_passes(rg, general, kind):  # noqa: F811
    """One buffer of offsets for several micro-batches: each backward call uses those of its forward call."""
    first, second = (torch.tensor(o, dtype=kind, device="cuda") for o in ([0, 20, 20, 70], [0, 0, 65, 70]))
    w = normal((3, 96, 200), 9, 0.1).cuda()
    ws = torch.empty(rg.library().expert_linear_f8_ws_bytes(70, 96, 200, 3), dtype=torch.uint8, device="cuda")
    kw = {"ws": ws} if general else {}
    batches = [(normal((70, 200), i, 1.0, bf).cuda(), normal((70, 96), i + 1, 1.0, bf).cuda()) for i in (1, 3)]
    want = []
    for (x, dy), off in zip(batches, (first, second)):
        y, saved = rg.expert_linear_f8(x, w, off, **kw)
        want.append((y, *rg.expert_linear_f8_backward(dy, saved, **kw)))
    buf = first.clone()
    kept = []
    for (x, _), off, outs in zip(batches, (first, second), want):
        buf.copy_(off)
        y, saved = rg.expert_linear_f8(x, w, buf, sync=False, **kw)
        assert torch.equal(y, outs[0])
        kept.append(saved)
    for (_, dy), saved, outs in reversed(list(zip(batches, kept, want))):
        assert all(torch.equal(a, b) for a, b in zip(rg.expert_linear_f8_backward(dy, saved, **kw), outs[1:]))


def test_offsets_are_kept_without_rows_or_columns(rg):  # noqa: F811
    """512 groups, and calls that multiply nothing: the copy of the offsets is there all the same."""
    for t, n, e in ((0, 30, 2), (5, 0, 3), (700, 16, 512)):
        off = (torch.arange(e + 1, device="cuda") * t // e).int()
        x, w = normal((t, 40), 1, 1.0, bf).cuda(), torch.ones((e, n, 40), device="cuda")
        y, saved = rg.expert_linear_f8(x, w, off)
        want = rg.expert_linear_f8_backward(y, saved)
        off.fill_(7)
        assert all(torch.equal(a, b) for a, b in zip(rg.expert_linear_f8_backward(y, saved), want))


@pytest.mark.parametrize("act", [None, "relu", "silu", "gelu"])
@pytest.mark.parametrize("m,dtype", [(897, f16), (1000, bf), (1024, bf), (1024, f32), (1025, bf), (1025, f16)])
def test_sums_on_both_sides_of_a_cluster(rg, m, dtype, act):  # noqa: F811
    """Up to 1024 rows, eight blocks of 128, the bias's gradient is summed within a cluster, beyond by a kernel of its
    own, beside which the input gradient's product runs."""
    check_layer_gradients(rg, m, 264, 136, dtype, act)


def test_capture_while_another_operators_graph_lives(rg):  # noqa: F811
    """Whoever's graph was the first to hold the leaf: made on the default stream it is refused before anything would be
    accumulated there, on a side stream it takes part, whatever ran on the default stream since."""
    w = normal((96, 128), 1, 0.1).cuda().requires_grad_()
    x, dy = normal((70, 128), 2, 1.0, bf).cuda(), normal((70, 96), 3, 1.0, bf).cuda()
    step = lambda: rg.linear_f8(x, w, sync=False)[0].backward(dy)  # noqa: E731
    own, side = torch.cuda.Stream(), torch.cuda.Stream()

    def capture():
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=own):
            w.grad = None
            step()
        return graph

    step()
    want = w.grad.clone()
    alive = (2 * w).sum()
    with pytest.raises(RuntimeError, match="default stream"):
        capture()
    torch.cuda.synchronize()
    assert torch.isfinite(alive)
    del alive
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        alive = (2 * w).sum()
    torch.cuda.current_stream().wait_stream(side)
    w.grad = None
    step()
    torch.cuda.synchronize()
    graph = capture()
    w.grad.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.isfinite(alive) and torch.equal(w.grad, want)


def test_weight_gradients_alone_report_offsets_past_the_rows(rg):  # noqa: F811
    """Within the last block of 128 rows too, which the blocks alone do not show."""
    x, w, dy = normal((7, 50), 1, 1.0, bf).cuda(), normal((2, 40, 50), 2, 0.1).cuda(), normal((7, 40), 3, 1.0, bf).cuda()
    off = torch.tensor([0, 3, 7], device="cuda")
    _, (kept, _, *rest) = rg.expert_linear_f8(x, w, off)
    want = rg.expert_linear_f8_backward(dy, (kept, off, *rest), dx=False)[1]
    for end in (8, 100, 127, 128, 1000):
        for bad in (torch.tensor([0, 3, end], device="cuda"), torch.tensor([0, end, end], device="cuda").int()):
            with pytest.raises(rg.ResGemmError) as err:
                rg.expert_linear_f8_backward(dy, (kept, bad, *rest), dx=False)
            assert err.value.code == rg.RG_ERR_ARG
    assert torch.equal(rg.expert_linear_f8_backward(dy, (kept, off, *rest), dx=False)[1], want)


def test_graphed_callable(rg):  # noqa: F811
    """torch.cuda.make_graphed_callables: forward and backward pass captured one after the other."""
    class Layer(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.w1, self.w2 = (torch.nn.Parameter(normal((128, 128), i, 0.1).cuda()) for i in (1, 2))
            self.b = torch.nn.Parameter(normal((128,), 3, 0.1).cuda())

        def forward(self, x):
            h, _ = rg.linear_act_f8(x, self.w1, bias=self.b, act="gelu", sync=False)
            return rg.linear_f8(h, self.w2, sync=False)[0]

    layer = Layer()
    xs = [normal((70, 128), 10 + i, 1.0, bf).cuda().requires_grad_() for i in range(3)]
    dy = normal((70, 128), 20, 1.0, bf).cuda()
    want = []
    for x in xs:
        y = layer(x)
        want.append((y.detach(), *torch.autograd.grad(y, (x, *layer.parameters()), dy)))
        del y
    torch.cuda.synchronize()
    graphed = torch.cuda.make_graphed_callables(layer, (xs[0].detach().clone().requires_grad_(),))
    for x, outs in zip(xs, want):
        y = graphed(x)
        got = (y.detach(), *torch.autograd.grad(y, (x, *layer.parameters()), dy))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, outs))


def test_captured_subsets_of_the_gradients(rg):  # noqa: F811
    """Calls that end in a memset, or leave a kernel out between two others, one behind the other in one graph."""
    x, w, b, dy = layer_inputs(300, 136, 264, bf)
    we, off = normal((3, 136, 264), 9, 0.1).cuda(), torch.tensor([0, 20, 20, 290], device="cuda")

    def step():
        outs = []
        y, saved = rg.linear_act_f8(x, w, bias=b, act="gelu", sync=False)
        z, kept = rg.expert_linear_f8(x, we, off, sync=False)
        for n in (4, 1, 0, 2, 6, 5, 3, 7):
            need = bool(n & 1), bool(n & 2)
            outs += rg.linear_act_f8_backward(dy, saved, False, f32, None, *need, bool(n & 4))
            outs += rg.expert_linear_f8_backward(dy, kept, False, f32, None, *need)
        return [t for t in (y, z, *outs) if t is not None]

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        got = step()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert len(got) == len(want) and all(torch.equal(a, c) for a, c in zip(got, want))
