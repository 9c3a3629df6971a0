"""The dense FP8 product against 64 bits: every recipe, activation and epilogue input, one token to
several tiles, output counts that are no multiple of anything, quantized and bf16 inputs."""
import pytest
import torch

import mixture_experts_fp8_b200 as moe
from _block_ref import F64, HALF, dequantize, linear, quantize, random_weights

pytestmark = pytest.mark.gpu


def problem(T, K, N, recipe, seed=0):
    g = torch.Generator().manual_seed(seed)
    codes, scales, wd = random_weights(g, K, N, recipe)
    x = torch.randn((T, K), generator=g).bfloat16()
    bias = torch.randn(N, generator=g).bfloat16()
    res = torch.randn((T, N), generator=g).bfloat16()
    return codes, scales, wd, x, bias, res


def check(y, want, off):
    y = y.cpu().to(F64)
    assert torch.all(torch.isfinite(y))
    bad = (y - want).abs() > want.abs() * HALF[torch.bfloat16] + off
    assert not bad.any(), f"{int(bad.sum())} values off, first at {torch.nonzero(bad)[0].tolist()}"


# N: a multiple of 128 and of 256, of 8 only, even, odd, one; T around the tiles
SHAPES = [(1, 128, 16), (1, 7168, 2048), (2, 256, 1), (31, 384, 250), (33, 512, 96), (64, 2816, 2816), (65, 128, 333),
          (127, 640, 1000), (129, 256, 130), (300, 768, 514), (700, 256, 264), (1237, 768, 1152), (1500, 384, 2050),
          (1111, 128, 3333), (3000, 256, 1000), (2600, 640, 2112), (520, 1152, 5000),
          (1301, 256, 4965), (2049, 384, 2227)]


@pytest.mark.parametrize("recipe", [0, 1, 2])
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_against_64_bits(T, K, N, recipe):
    N += N % 2 if recipe == 2 else 0
    codes, scales, wd, x, bias, res = problem(T, K, N, recipe, T * 31 + N)
    a = (T + N) % 5
    cfg = moe.LinearConfig(T, K, N, recipe, a)
    w = moe.transform_linear_weights(cfg, codes.cuda(), scales.cuda())
    q = quantize(x, recipe)
    y = moe.linear(cfg, w, quantized=tuple(t.cuda() for t in q), bias=bias.cuda(), residual=res.cuda())
    y2 = moe.linear(cfg, w, x=x.cuda(), bias=bias.cuda(), residual=res.cuda())      # quantized by the call
    torch.cuda.synchronize()
    assert torch.equal(y, y2)
    check(y, *linear(dequantize(q[0], q[1], recipe), wd, bias, a, res))


# tiles of 512 tokens (from seven K groups on, an even and an odd number of them; the last one's second half empty or
# ragged; N in eights, even and odd) and of 256
@pytest.mark.parametrize("T,K,N", [(1024, 256, 4736), (1500, 640, 4738), (900, 384, 4729), (1100, 128, 4800), (2048, 1152, 2304),
                                   (900, 1152, 4729), (1024, 1024, 4730), (1500, 1408, 4736), (1700, 1280, 4673)])
def test_long_batches_of_fp32_scales(T, K, N):
    codes, scales, wd, x, bias, res = problem(T, K, N, 0, T + N)
    cfg = moe.LinearConfig(T, K, N, 0, N % 5)
    w = moe.transform_linear_weights(cfg, codes.cuda(), scales.cuda())
    q = quantize(x, 0)
    ws = moe.new_linear_workspace(cfg)
    buf = res.cuda()
    y = moe.linear(cfg, w, quantized=tuple(t.cuda() for t in q), bias=bias.cuda(), residual=buf, y=buf, workspace=ws)
    assert moe.read_status(ws) == 0
    check(y, *linear(dequantize(q[0], q[1], 0), wd, bias, N % 5, res))
    # the same bits in a batch of few enough rows for the smaller tile
    part = moe.LinearConfig(256, K, N, 0, N % 5)
    r = T - 256
    few = moe.linear(part, w, x=x[r:].cuda(), bias=bias.cuda(), residual=res[r:].contiguous().cuda())
    assert torch.equal(few, y[r:])


# tiles of 256 columns: one and several a pair, the last one narrow, N in eights, even and odd
@pytest.mark.parametrize("recipe", [1, 2])
@pytest.mark.parametrize("T,K,N", [(512, 1024, 9472), (1500, 896, 4738), (2500, 768, 3594), (2048, 1152, 4096), (1030, 640, 7937), (1500, 1024, 4737)])
def test_long_batches_of_block_scales(T, K, N, recipe):
    N += N % 2 if recipe == 2 else 0
    codes, scales, wd, x, bias, res = problem(T, K, N, recipe, T + N)
    cfg = moe.LinearConfig(T, K, N, recipe, N % 5)
    w = moe.transform_linear_weights(cfg, codes.cuda(), scales.cuda())
    q = quantize(x, recipe)
    ws = moe.new_linear_workspace(cfg)
    buf = res.cuda()
    y = moe.linear(cfg, w, quantized=tuple(t.cuda() for t in q), bias=bias.cuda(), residual=buf, y=buf, workspace=ws)
    assert moe.read_status(ws) == 0
    check(y, *linear(dequantize(q[0], q[1], recipe), wd, bias, N % 5, res))


@pytest.mark.parametrize("a", range(5))
@pytest.mark.parametrize("recipe,T,N", [(0, 5, 256), (1, 200, 264), (2, 70, 130)])
@pytest.mark.parametrize("with_bias,with_res", [(False, False), (True, False), (False, True)])
def test_epilogues(recipe, T, N, a, with_bias, with_res):
    codes, scales, wd, x, bias, res = problem(T, 256, N, recipe, a)
    cfg = moe.LinearConfig(T, 256, N, recipe, a)
    w = moe.transform_linear_weights(cfg, codes.cuda(), scales.cuda())
    q = quantize(x, recipe)
    bias, res = bias if with_bias else None, res if with_res else None
    ws = moe.new_linear_workspace(cfg)
    y = moe.linear(cfg, w, x=x.cuda(), bias=None if bias is None else bias.cuda(),
                   residual=None if res is None else res.cuda(), workspace=ws)
    assert moe.read_status(ws) == 0
    check(y, *linear(dequantize(q[0], q[1], recipe), wd, bias, a, res))


@pytest.mark.parametrize("recipe", [0, 1, 2])
@pytest.mark.parametrize("T,N", [(3, 384), (150, 384), (150, 386)])
def test_rows_stay_apart_and_in_place_residual(recipe, T, N):
    """A row of NaN or infinities leaves the others' bits alone; the residual's buffer may be y."""
    codes, scales, wd, x, bias, res = problem(T, 512, N, recipe, 9)
    cfg = moe.LinearConfig(T, 512, N, recipe, moe.ACT_SILU)
    w = moe.transform_linear_weights(cfg, codes.cuda(), scales.cuda())
    y = moe.linear(cfg, w, x=x.cuda(), bias=bias.cuda(), residual=res.cuda())
    bad = x.clone()
    bad[1, 3] = float("nan")
    buf = res.cuda()
    y2 = moe.linear(cfg, w, x=bad.cuda(), bias=bias.cuda(), residual=buf, y=buf)
    torch.cuda.synchronize()
    keep = [t for t in range(T) if t != 1]
    assert torch.equal(y2[keep], y[keep]) and torch.isnan(y2[1].float()).any()


def test_captured_and_two_workspaces():
    T, K, N = 70, 384, 520
    for recipe in (0, 1):
        codes, scales, _, x, bias, res = problem(T, K, N, recipe, 11)
        cfg = moe.LinearConfig(T, K, N, recipe, moe.ACT_GELU)
        w = moe.transform_linear_weights(cfg, codes.cuda(), scales.cuda())
        x, bias, res = x.cuda(), bias.cuda(), res.cuda()
        want = moe.linear(cfg, w, x=x, bias=bias, residual=res)
        wss = [moe.new_linear_workspace(cfg) for _ in range(2)]
        ys = [torch.zeros_like(want) for _ in range(2)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.linear(cfg, w, x=x, bias=bias, residual=res, y=ys[0], workspace=wss[0])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        x.copy_(x.flip(0))
        res.copy_(res.flip(0))
        s.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(s):                        # at the same time, with a workspace of its own
            moe.linear(cfg, w, x=x, bias=bias, residual=res, y=ys[1], workspace=wss[1])
        torch.cuda.synchronize()
        assert torch.equal(ys[0], want.flip(0)) and torch.equal(ys[1], want.flip(0))


def test_a_block_of_them():
    """norm -> product -> residual product -> norm -> layer gate's input, as a transformer block runs them."""
    T, H, N = 48, 512, 896
    g = torch.Generator().manual_seed(3)
    for recipe in (0, 1, 2):
        c1, s1, w1 = random_weights(g, H, N, recipe)
        c2, s2, w2 = random_weights(g, N, H, recipe)
        l1, l2 = moe.LinearConfig(T, H, N, recipe, moe.ACT_GELU_TANH), moe.LinearConfig(T, N, H, recipe)
        t1, t2 = (moe.transform_linear_weights(l, c.cuda(), s.cuda()) for l, c, s in ((l1, c1, s1), (l2, c2, s2)))
        x = torch.randn((T, H), generator=g).bfloat16()
        r = torch.randn((T, H), generator=g).bfloat16()
        nw = (1 + 0.1 * torch.randn(H, generator=g))
        cfg = moe.Config(T, H, 128, 8, 1, recipe=recipe)
        h, _, q = moe.add_rms_norm(cfg, x.cuda(), nw.cuda(), 1e-6, residual=r.cuda(), want_y=False)
        mid = moe.linear(l1, t1, quantized=q)
        out = moe.linear(l2, t2, x=mid, residual=h)
        h2, y, _ = moe.add_rms_norm(cfg, out, nw.cuda(), 1e-6)
        torch.cuda.synchronize()
        # each step against 64 bits from the step before
        want, off = linear(dequantize(q[0], q[1], recipe), w1, None, 4, None)
        check(mid, want, off)
        qm = quantize(mid.cpu(), recipe)
        want, off = linear(dequantize(qm[0], qm[1], recipe), w2, None, 0, h.cpu())
        check(out, want, off)
        o = out.cpu().to(F64)
        ref = o / torch.sqrt((o * o).mean(1, keepdim=True) + 1e-6) * nw.to(F64)
        assert torch.all((y.cpu().to(F64) - ref).abs() <= ref.abs() * (HALF[torch.bfloat16] + 40 * 2.0 ** -24))
