"""The dense product where an output's offset passes 32 bits, against 64 bits."""
import pytest
import torch

import mixture_experts_fp8_b200 as moe
from _block_ref import F64, HALF, dequantize, linear, quantize, random_weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("recipe", [0, 1, 2])
def test_last_rows_against_64_bits(recipe):
    T, K, N, n = 1100000, 256, 2050, 300                  # 2.26e9 outputs, by words
    codes, scales, wd = random_weights(torch.Generator().manual_seed(1), K, N, recipe)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    rows = torch.cat([torch.arange(n), torch.arange(T - n, T)])
    xr = torch.randn((2 * n, K), generator=torch.Generator().manual_seed(2)).bfloat16()
    x[rows.cuda()] = xr.cuda()
    bias = torch.randn(N, generator=torch.Generator().manual_seed(3)).bfloat16()
    lin = moe.LinearConfig(T, K, N, recipe, moe.ACT_GELU)
    ws = moe.new_linear_workspace(lin)
    y = moe.linear(lin, moe.transform_linear_weights(lin, codes.cuda(), scales.cuda()), x=x, bias=bias.cuda(), workspace=ws)
    assert moe.read_status(ws) == 0
    want, off = linear(dequantize(*quantize(xr, recipe), recipe), wd, bias, 3, None)
    got = y[rows.cuda()].cpu().to(F64)
    assert torch.all((got - want).abs() <= want.abs() * HALF[torch.bfloat16] + off)
    zero, _ = linear(torch.zeros((1, K), dtype=F64), wd, bias, 3, None)
    assert torch.all((y[T // 2].cpu().to(F64) - zero).abs() <= zero.abs() * HALF[torch.bfloat16] * 1.001)
