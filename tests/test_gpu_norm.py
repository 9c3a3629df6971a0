"""The residual RMS norm with its 8-bit output against 64 bits: every residual type and recipe, rows
from one warp to the longest, odd batches, buffers used in place, rows of zeros, infinities and NaN."""
import pytest
import torch

import mixture_experts_fp8_b200 as moe
from _block_ref import F64, HALF, U, dequantize, words_to_scales

pytestmark = pytest.mark.gpu
EPS = 1e-6
# y in fp32: the sum of squares takes at most 8 * 4 terms a thread, 5 steps a warp and 32 warps in
# sequence (70 roundings, halved by the root), then five more operations
REL = 40 * U


def cfg(T, H, recipe=0):
    return moe.Config(T, H, 128, 8, 1, recipe=recipe)


def inputs(T, H, res, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((T, H), generator=g) * scale).bfloat16()
    r = None if res is None else (torch.randn((T, H), generator=g) * 2 * scale).to(res)
    return x, r, 1 + 0.1 * torch.randn(H, generator=g)


def reference(x, r, w, eps=EPS):
    h = x.to(F64) if r is None else x.to(F64) + r.to(F64)
    return h, h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * w.to(F64)


def check_quantized(q, y, recipe):
    codes, words = q
    T, H = y.shape
    s = words_to_scales(words, recipe, T)
    amax = y.reshape(T, s.shape[1], -1).abs().amax(-1)
    if recipe == 0:
        want = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
        assert torch.all((s - want).abs() <= want * (REL + 2 * U))
    else:   # the smallest power of two that keeps the group within 448
        assert torch.all(amax <= s * 448 * (1 + REL))
        assert torch.all((amax > s * 224 * (1 - REL)) | (amax == 0) | (s == 2.0 ** -127))
        assert torch.all(s[amax == 0] == 1)
    # E4M3: half a step is 2^-4 of the value, 2^-10 of the scale below the normal codes
    got = dequantize(codes, words, recipe)
    tol = y.abs() * (2.0 ** -4 + 2 * REL) + (s * 2.0 ** -10).repeat_interleave(H // s.shape[1], 1)
    assert torch.all((got - y).abs() <= tol)


@pytest.mark.parametrize("recipe", [0, 1])
@pytest.mark.parametrize("res", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 128), (3, 256), (77, 384), (64, 2816), (5, 7168), (2, 32768), (1000, 640)])
def test_against_64_bits(T, H, res, recipe):
    x, r, w = inputs(T, H, res, seed=T + H)
    h, y = reference(x, r, w)
    ro, yo, q = moe.add_rms_norm(cfg(T, H, recipe), x.cuda(), w.cuda(), EPS, residual=None if r is None else r.cuda())
    torch.cuda.synchronize()
    if r is not None:
        assert torch.equal(ro.cpu(), (x.float() + r.float()).to(res))      # one fp32 sum, rounded once
    assert torch.all((yo.cpu().to(F64) - y).abs() <= y.abs() * (HALF[torch.bfloat16] + REL) + 1e-38)
    check_quantized(q, y, recipe)


def test_outputs_one_at_a_time_agree():
    T, H = 33, 1152
    x, r, w = (t.cuda() for t in inputs(T, H, torch.float32, 3))
    c = cfg(T, H, 1)
    ro, y, q = moe.add_rms_norm(c, x, w, EPS, residual=r)
    _, y1, q1 = moe.add_rms_norm(c, x, w, EPS, residual=r, want_quantized=False)
    _, y2, q2 = moe.add_rms_norm(c, x, w, EPS, residual=r, want_y=False)
    assert q1 is None and y2 is None
    assert torch.equal(y, y1) and torch.equal(q[0], q2[0]) and torch.equal(q[1][:, :T], q2[1][:, :T])


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_in_place_and_batch_independent(res):
    T, H = 130, 2816
    x, r, w = (t.cuda() for t in inputs(T, H, res, 4))
    ro, y, q = moe.add_rms_norm(cfg(T, H), x, w, EPS, residual=r)
    x1, r1 = x.clone(), r.clone()
    moe.add_rms_norm(cfg(T, H), x1, w, EPS, residual=r1, residual_out=r1, y=x1)
    assert torch.equal(r1, ro) and torch.equal(x1, y)
    rows = torch.tensor([129, 0, 64], device="cuda")
    _, ys, qs = moe.add_rms_norm(cfg(3, H), x[rows], w, EPS, residual=r[rows])
    assert torch.equal(ys, y[rows]) and torch.equal(qs[0], q[0][rows]) and torch.equal(qs[1][:, :3], q[1][:, rows])


@pytest.mark.parametrize("recipe", [0, 1])
def test_zeros_extremes_and_non_finite_rows(recipe):
    T, H = 8, 512
    x, _, w = inputs(T, H, None, 5)
    x[1] = 0
    x[2] *= 1e-30
    x[3] *= 1e15
    x[4, 7] = float("inf")
    x[5, 9] = float("nan")
    x[6, :256] = 0
    _, y, q = moe.add_rms_norm(cfg(T, H, recipe), x.cuda(), w.cuda(), EPS)
    torch.cuda.synchronize()
    fine = [0, 1, 2, 3, 6, 7]
    _, want = reference(x[fine], None, w)
    got = y.cpu().to(F64)
    assert torch.all((got[fine] - want).abs() <= want.abs() * (HALF[torch.bfloat16] + REL) + 1e-38)
    assert torch.all(got[1] == 0)
    deq = dequantize(q[0], q[1], recipe)
    assert torch.all(deq[1] == 0) and torch.all(torch.isfinite(deq[fine]))
    check_quantized((q[0][fine].cpu(), q[1][:, fine]), want, recipe)
    for v in (got, deq):
        assert not torch.isfinite(v[4]).all() and torch.isnan(v[5]).any()


def test_scale_words_behind_the_rows_stay():
    T, H = 5, 256
    x, _, w = (t if t is None else t.cuda() for t in inputs(T, H, None, 6))
    codes, words = moe.new_quantized(T, H)
    words.fill_(0x1234567)
    moe.add_rms_norm(cfg(T, H), x, w, EPS, quantized=(codes, words))
    assert torch.all(words[:, T:] == 0x1234567)


def test_captured_and_on_another_stream():
    T, H = 40, 768
    x, r, w = (t.cuda() for t in inputs(T, H, torch.bfloat16, 7))
    c = cfg(T, H, 1)
    ro, y, q = moe.add_rms_norm(c, x, w, EPS, residual=r)
    outs = (torch.zeros_like(ro), torch.zeros_like(y), tuple(torch.zeros_like(t) for t in q))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        moe.add_rms_norm(c, x, w, EPS, residual=r, residual_out=outs[0], y=outs[1], quantized=outs[2])
    s.synchronize()
    assert torch.equal(outs[0], ro) and torch.equal(outs[1], y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.add_rms_norm(c, x, w, EPS, residual=r, residual_out=outs[0], y=outs[1], quantized=outs[2])
    x.copy_(x.flip(0))
    r.copy_(r.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[1], y.flip(0)) and torch.equal(outs[2][0], q[0].flip(0))


@pytest.mark.parametrize("recipe", [0, 1])
def test_values_below_the_smallest_scale(recipe):
    # amax / 448 is under half the smallest fp32 number: no scale can hold it
    T, H = 2, 256
    x, w = torch.ones((T, H), dtype=torch.bfloat16), torch.zeros(H)
    w[0] = 1e-44
    codes, words = moe.add_rms_norm(cfg(T, H, recipe), x.cuda(), w.cuda(), EPS)[2]
    assert float(dequantize(codes.cpu(), words, recipe).abs().max()) <= 1e-43      # NaN fails
