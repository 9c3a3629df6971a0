"""Values at the ends of the operators around the layer: infinities through the quantizers, activations far in
their tails, gradients that are not a row's."""
import math

import pytest
import torch

import mixture_experts_fp8_b200 as moe
from _block_ref import F64, HALF, U, dequantize, random_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("recipe", [0, 1, 2])
@pytest.mark.parametrize("T", [3, 300])
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_an_infinite_input_of_the_product(recipe, T, value):
    """No column of its row is finite; the other rows keep their bits."""
    K, N = 512, 256
    codes, scales, _ = random_weights(torch.Generator().manual_seed(1), K, N, recipe)
    lin = moe.LinearConfig(T, K, N, recipe)
    w = moe.transform_linear_weights(lin, codes.cuda(), scales.cuda())
    x = torch.randn((T, K), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    y = moe.linear(lin, w, x=x)
    x[1, 77] = value
    bad = moe.linear(lin, w, x=x)
    assert not torch.isfinite(bad[1]).any()
    keep = [t for t in range(T) if t != 1]
    assert torch.equal(bad[keep], y[keep])


@pytest.mark.parametrize("recipe", [0, 1])
def test_a_norm_that_overflows(recipe):
    """y passes the largest fp32 number where the weight does: its codes do not stand for a finite value there."""
    T, H = 4, 512
    x = torch.randn((T, H), generator=torch.Generator().manual_seed(3)).bfloat16()
    w = torch.ones(H)
    x[2, 200], w[200] = 100.0, 3e38
    _, y, q = moe.add_rms_norm(moe.Config(T, H, 128, 8, 1, recipe=recipe), x.cuda(), w.cuda(), 1e-6)
    v = dequantize(q[0], q[1], recipe)
    assert torch.isinf(y[2, 200]) and not torch.isfinite(v[2, 200])
    assert torch.isfinite(v[2, :128]).all() and torch.isfinite(v[2, 256:]).all()


@pytest.mark.parametrize("T", [3, 300])
@pytest.mark.parametrize("a", range(5))
def test_activations_in_their_tails(T, a):
    """The sums are zero, so that the activation's argument is the bias; relative to each value."""
    K, N = 128, 1280
    v = torch.linspace(-9.5, 9.5, N).bfloat16()
    lin = moe.LinearConfig(T, K, N, 0, a)
    w = moe.transform_linear_weights(lin, torch.zeros((K, N), dtype=torch.uint8, device="cuda"), torch.ones((1, N), device="cuda"))
    y = moe.linear(lin, w, x=torch.zeros((T, K), dtype=torch.bfloat16, device="cuda"), bias=v.cuda()).cpu().to(F64)
    d = v.to(F64)
    u2 = 2 * math.sqrt(2 / math.pi) * (d + 0.044715 * d ** 3)
    want = (d, d.clamp(min=0), d / (1 + torch.exp(-d)), 0.5 * d * torch.special.erfc(-d / math.sqrt(2)), d / (1 + torch.exp(-u2)))[a]
    # fp32 roundings before the last one: an argument's relative error of up to 8 is worth that times the argument in an
    # exponential, and times 2 x^2 + 1, x = v / sqrt 2, in erfc; 32 for the functions' own and the products
    arg = (d * 0, d * 0, d.abs(), d ** 2 + 1, u2.abs())[a]
    assert torch.all((y - want).abs() <= want.abs() * (HALF[torch.bfloat16] + (8 * arg + 32) * U))


@pytest.mark.parametrize("T", [3, 300])
@pytest.mark.parametrize("a", range(5))
def test_activations_of_nan_and_infinity(T, a):
    K, N = 128, 128
    v = torch.zeros(N)
    v[5], v[70], v[71], v[72] = float("nan"), float("inf"), 1e30, -1e30
    lin = moe.LinearConfig(T, K, N, 1, a)
    w = moe.transform_linear_weights(lin, torch.zeros((K, N), dtype=torch.uint8, device="cuda"),
                                     torch.full((K // 32, N), 127, dtype=torch.uint8, device="cuda"))
    v = v.bfloat16()
    y = moe.linear(lin, w, x=torch.zeros((T, K), dtype=torch.bfloat16, device="cuda"), bias=v.cuda())
    assert torch.isnan(y[:, 5]).all() and torch.all(y[:, 70] == float("inf")) and torch.all(y[:, 71] == v[71].item())
    assert torch.all(y[:, 72] == (v[72].item() if a == 0 else 0)) and torch.all(y[:, 73:] == 0)


MODES = [(0, 0), (0, 1), (1, 0)]                          # routing, renormalize


@pytest.mark.parametrize("T,E,k", [(75, 16, 4), (60000, 16, 4), (15000, 130, 20)])   # a token a lane group, and several
@pytest.mark.parametrize("routing,renorm", MODES)
def test_tokens_outside_the_loss_take_no_part_of_its_gradient(T, E, k, routing, renorm):
    """A loss whose gradient overflowed: masked tokens, and those of no sequence, keep the gradient of their weights."""
    g = torch.Generator().manual_seed(4)
    l = torch.randn((T, E), generator=g).cuda()
    idx = torch.topk(l, k)[1].int()
    dw = torch.randn((T, k), generator=g).cuda()
    mask = torch.rand(T, generator=g).cuda() < 0.5
    off = torch.tensor([3, T // 2, T - 5], dtype=torch.int32, device="cuda")
    cfg = moe.Config(T, 128, 128, E, k, routing=routing, renormalize=renorm)
    _, counts, tokens, _ = moe.balance_loss(cfg, l, idx, 0.1, seq_offsets=off, token_mask=mask)
    alone, _ = moe.route_backward(cfg, l, idx, d_topk_weights=dw)
    outside = ~mask
    outside[:3] = outside[T - 5:] = True
    for d in (float("inf"), float("nan"), 1e38):
        both, _ = moe.route_backward(cfg, l, idx, d_topk_weights=dw, d_loss=torch.full((1,), d, device="cuda"), coef=1e3,
                                     expert_counts=counts, seq_tokens=tokens, seq_offsets=off, token_mask=mask)
        assert torch.equal(both[outside], alone[outside])
        assert not torch.isfinite(both[~outside]).all(1).any() or d == 1e38


@pytest.mark.parametrize("E,k", [(16, 4), (130, 20)])
@pytest.mark.parametrize("routing,renorm", MODES)
def test_slots_without_an_expert(E, k, routing, renorm):
    """A padded row (ids of -1 or past E; logits and weights' gradients of anything) has a gradient of zero, and such a
    slot among others adds nothing to its row or to the scales."""
    T = 60
    g = torch.Generator().manual_seed(5)
    l = torch.randn((T, E), generator=g).cuda()
    idx = torch.topk(l, k)[1].int()
    dw, pes = torch.randn((T, k), generator=g).cuda(), torch.rand(E, generator=g).cuda()
    pad, part = list(range(0, T, 7)), list(range(3, T, 7))
    zeroed = dw.clone()
    zeroed[pad] = 0
    zeroed[part, k - 1] = 0
    l[pad] = float("nan")
    l[pad[0]] = float("inf")
    idx[pad] = -1
    idx[pad[1:3]] = E
    idx[part, k - 1] = 1 << 30
    dw[part, k - 1] = float("nan")
    cfg = moe.Config(T, 128, 128, E, k, routing=routing, renormalize=renorm)
    dl, dp = moe.route_backward(cfg, l, idx, d_topk_weights=dw, per_expert_scale=pes)
    dl0, dp0 = moe.route_backward(cfg, l, idx, d_topk_weights=zeroed, per_expert_scale=pes)
    assert torch.all(dl[pad] == 0) and torch.isfinite(dl).all() and torch.isfinite(dp).all()
    assert torch.equal(dl, dl0) and torch.equal(dp, dp0)
