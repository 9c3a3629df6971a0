"""Calls of the operators around the layer on a stream that is not the current one: what they allocate is
not memory that kernels pending on the current stream still use."""
import pytest
import torch

import mixture_experts_fp8_b200 as moe
from _block_ref import random_weights

pytestmark = pytest.mark.gpu

T, H, N, E, K = 2048, 1024, 1024, 256, 8


def problems():
    g = torch.Generator().manual_seed(0)
    x = torch.randn((T, H), generator=g).bfloat16().cuda()
    l = torch.randn((T, E), generator=g).cuda()
    idx = torch.topk(l, K)[1].int()
    dw, pes = torch.randn((T, K), generator=g).cuda(), torch.rand(E, generator=g).cuda()
    codes, scales, _ = (t.cuda() for t in random_weights(g, H, N, 1))
    cfg, lin = moe.Config(T, H, 128, E, K, recipe=1), moe.LinearConfig(T, H, N, 1)
    w = moe.transform_linear_weights(lin, codes, scales)
    nw = torch.ones(H, device="cuda")
    return {
        "add_rms_norm": lambda s: [t for o in moe.add_rms_norm(cfg, x, nw, 1e-6, residual=x, stream=s)
                                   for t in (o if isinstance(o, tuple) else (o,))],
        "linear": lambda s: [moe.linear(lin, w, x=x, stream=s)],
        "balance_loss": lambda s: list(moe.balance_loss(cfg, l, idx, 0.1, stream=s)),
        "route_backward": lambda s: list(moe.route_backward(cfg, l, idx, dw, pes, stream=s)),
        "transform_linear_weights": lambda s: list(moe.transform_linear_weights(lin, codes, scales, stream=s)),
    }


def rows(t):
    """The values that a call writes (scale words behind the rows are left as they were)."""
    return t[:, :T] if t.dtype is torch.int32 and t.shape[-1] > T else t


@pytest.mark.parametrize("name", ["add_rms_norm", "linear", "balance_loss", "route_backward", "transform_linear_weights"])
def test_blocks_that_the_current_stream_still_writes(name):
    call = problems()[name]
    want = [t.clone() for t in call(None)]
    # one spare block of every size that the call asks for, and a few for its own temporaries
    sizes = [t.numel() * t.element_size() for t in want] + [T * H + 16384, T * H * 2, T * E * 4, 1 << 16, 1024, 512]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
        spans = [(b.data_ptr(), b.data_ptr() + b.numel()) for b in blocks]
        torch.cuda._sleep(20_000_000)                     # about 10 ms; side does not wait for what follows
        for b in blocks:
            b.fill_(0xFF)
        del blocks, b
        got = call(side)
        for t in got:
            p = t.data_ptr()
            assert not any(lo <= p < hi for lo, hi in spans)
        torch.cuda.synchronize()
        assert all(torch.equal(rows(a), rows(b)) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["add_rms_norm", "linear", "route_backward", "transform_linear_weights"])
def test_results_that_the_current_stream_still_reads(name):
    """A result is dropped while the current stream has yet to copy it; the next call must not take its block."""
    call = problems()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    copies, held = [], []
    for _ in range(4):
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(5_000_000)
        copies.append([t.clone() for t in got])
        del got
        with torch.cuda.stream(side):                     # would take a freed block of side's at once
            held.append([torch.full_like(t, 77) for t in want])
    torch.cuda.synchronize()
    assert all(torch.equal(rows(a), rows(b)) for c in copies for a, b in zip(c, want))


def test_the_layer_and_its_gate():
    """The same of the layer's own calls: what they return, and the workspace of a call that is given none."""
    import synth
    prob = synth.make_problem("tiny")
    d = prob.to("cuda:0")
    cfg = moe.Config(**prob.shape.cfg())
    weights = moe.transform_weights(cfg, d.w13, d.w13_scale, d.w2, d.w2_scale)
    nw, rw, eps = synth.make_gate(prob.shape)
    nw, rw = nw.cuda(), rw.cuda()
    gw = moe.transform_gate_weights(cfg, nw, rw)
    calls = [lambda s: [moe.forward(cfg, d.x, weights, router_logits=d.logits, stream=s)],
             lambda s: list(moe.route(cfg, d.logits, stream=s)), lambda s: list(moe.gate(cfg, d.x, gw, eps, stream=s)),
             lambda s: list(moe.transform_weights(cfg, d.w13, d.w13_scale, d.w2, d.w2_scale, stream=s)),
             lambda s: [moe.transform_gate_weights(cfg, nw, rw, stream=s)]]
    for call in calls:
        want = [t.clone() for t in call(None)]
        sizes = [t.numel() * t.element_size() for t in want] + [moe.workspace_size(cfg)]
        side = torch.cuda.Stream()
        for _ in range(3):
            torch.cuda.synchronize()
            blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
            spans = [(b.data_ptr(), b.data_ptr() + b.numel()) for b in blocks]
            side.wait_stream(torch.cuda.current_stream())
            torch.cuda._sleep(20_000_000)
            for b in blocks:
                b.fill_(0xFF)
            del blocks, b
            got = call(side)
            assert not any(lo <= t.data_ptr() < hi for t in got for lo, hi in spans)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            del got


@pytest.mark.parametrize("name", ["add_rms_norm", "linear", "balance_loss", "route_backward"])
def test_captured_on_a_side_stream(name):
    """A graph that forks to another stream for the call and joins it again."""
    call = problems()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cur = torch.cuda.current_stream()
        side.wait_stream(cur)
        first = call(side)
        second = call(side)
        cur.wait_stream(side)
        copies = [t.clone() for t in first]
    for _ in range(2):
        for t in (*first, *second, *copies):
            t.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        for got in (first, second, copies):
            assert all(torch.equal(rows(a), rows(b)) for a, b in zip(got, want))


@pytest.mark.parametrize("T,K,N,recipe", [(16, 1024, 512, 0), (64, 1024, 512, 1), (300, 768, 514, 0), (2048, 256, 2304, 0),
                                          (2048, 1152, 4096, 0), (2048, 1152, 4095, 1), (1500, 256, 2048, 2), (2048, 1152, 4096, 1)])
def test_a_chain_in_place(T, K, N, recipe):
    """Products that add to one buffer one after the other, with nothing between them: each reads what the last one
    wrote, though its blocks start while that one's are still running."""
    g = torch.Generator().manual_seed(6)
    codes, scales, _ = (t.cuda() for t in random_weights(g, K, N, recipe))
    lin = moe.LinearConfig(T, K, N, recipe)
    w = moe.transform_linear_weights(lin, codes, scales)
    q = moe.add_rms_norm(moe.Config(T, K, 128, 8, 1, recipe=recipe), torch.randn((T, K), generator=g).bfloat16().cuda(),
                         torch.ones(K, device="cuda"), 1e-6)[2]
    ws = moe.new_linear_workspace(lin)
    start = torch.randn((T, N), generator=g).bfloat16().cuda()

    def chain(wait):
        y = start.clone()
        torch.cuda.synchronize()
        for _ in range(12):
            moe.linear(lin, w, quantized=q, residual=y, y=y, workspace=ws)
            if wait:
                torch.cuda.synchronize()
        return y
    want = chain(True)
    for _ in range(5):
        assert torch.equal(chain(False), want)
