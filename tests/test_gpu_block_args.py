"""Tensors that the operators around the layer refuse: wrong shapes, types, orders and devices."""
import pytest
import torch

import mixture_experts_fp8_b200 as moe

pytestmark = pytest.mark.gpu


def refused(call, word):
    with pytest.raises(moe.MoeError) as e:
        call()
    assert e.value.code == moe.MOE_ERR_INVALID_ARG and word in str(e.value)


def test_norm_and_linear():
    T, H, N = 8, 256, 64
    cfg, lin = moe.Config(T, H, 128, 8, 1), moe.LinearConfig(T, H, N)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(H, device="cuda")
    refused(lambda: moe.add_rms_norm(cfg, x.float(), w, 1e-6), "x must be")
    refused(lambda: moe.add_rms_norm(cfg, x[:7], w, 1e-6), "x must be")
    refused(lambda: moe.add_rms_norm(cfg, torch.zeros((H, T), dtype=torch.bfloat16, device="cuda").t(), w, 1e-6), "not contiguous")
    refused(lambda: moe.add_rms_norm(cfg, x, w.cpu(), 1e-6), "norm_weight")
    refused(lambda: moe.add_rms_norm(cfg, x, w, 1e-6, residual=x.half()), "residual")
    refused(lambda: moe.add_rms_norm(cfg, x, w, 1e-6, residual=x, residual_out=x.float()), "residual_out")
    refused(lambda: moe.add_rms_norm(cfg, x, w, 1e-6, quantized=moe.new_quantized(T + 4, H)), "codes")
    refused(lambda: moe.add_rms_norm(cfg, x.cpu(), w, 1e-6), "current device")
    codes = torch.zeros((H, N), dtype=torch.uint8, device="cuda")
    scales = torch.ones((H // 128, N), device="cuda")
    refused(lambda: moe.transform_linear_weights(lin, codes.t(), scales), "w must be")
    refused(lambda: moe.transform_linear_weights(lin, codes, scales.to(torch.uint8)), "w_scale")
    weights = moe.transform_linear_weights(lin, codes, scales)
    refused(lambda: moe.linear(lin, weights), "exactly one")
    refused(lambda: moe.linear(lin, weights, x=x[:, :128]), "x must be")
    refused(lambda: moe.linear(lin, weights[::-1], x=x), "w_t")
    refused(lambda: moe.linear(lin, weights, x=x, bias=torch.zeros(N, device="cuda")), "bias")
    refused(lambda: moe.linear(lin, weights, x=x, residual=torch.zeros((T, N), device="cuda")), "residual")
    refused(lambda: moe.linear(lin, weights, x=x, workspace=torch.empty(512, dtype=torch.uint8, device="cuda")), "workspace")
    odd = torch.empty(T * N + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, N)
    refused(lambda: moe.linear(lin, weights, x=x, y=odd), "misaligned")


def test_router():
    T, E, k = 8, 16, 2
    cfg = moe.Config(T, 128, 128, E, k)
    l = torch.zeros((T, E), device="cuda")
    idx = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    refused(lambda: moe.balance_loss(cfg, l.double(), idx, 0.1), "router_logits")
    refused(lambda: moe.balance_loss(cfg, l, idx.long(), 0.1), "topk_idx")
    refused(lambda: moe.balance_loss(cfg, l, idx, 0.1, token_mask=torch.ones(T, device="cuda")), "token_mask")
    refused(lambda: moe.balance_loss(cfg, l, idx, 0.1, seq_offsets=torch.zeros(1, dtype=torch.int32, device="cuda")), "two offsets")
    refused(lambda: moe.balance_loss(cfg, l, idx, 0.1, seq_offsets=torch.zeros(3, device="cuda")), "seq_offsets")
    refused(lambda: moe.route_backward(cfg, l, idx), "one of")
    refused(lambda: moe.route_backward(cfg, l, idx, d_loss=torch.ones(1, device="cuda")), "expert_counts")
    refused(lambda: moe.route_backward(cfg, l, idx, d_topk_weights=torch.ones((T, k + 1), device="cuda")), "d_topk_weights")
