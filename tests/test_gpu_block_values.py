"""Values at the ends of the operators around the layer: infinities through the quantizers, activations far in
their tails, gradients that are not a row's."""
import pytest
import torch

import mixture_experts_fp8_b200 as moe
from _block_ref import dequantize, random_weights

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
