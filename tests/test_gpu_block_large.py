"""The operators around the layer where an offset passes 32 bits: the rows behind it equal, bit for bit,
the same rows in a small call (a row does not depend on the batch)."""
import pytest
import torch

import mixture_experts_fp8_b200 as moe
from _block_ref import quantize, random_weights

pytestmark = pytest.mark.gpu


def test_norm():
    T, H = 66000, 32768                                   # 2.16e9 elements
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    rows = [0, T // 2, T - 2, T - 1]
    x[rows] = torch.randn((4, H), generator=g, device="cuda").bfloat16()
    w = 1 + 0.1 * torch.randn(H, generator=g, device="cuda")
    _, y, q = moe.add_rms_norm(moe.Config(T, H, 128, 8, 1), x, w, 1e-6)
    _, ys, qs = moe.add_rms_norm(moe.Config(4, H, 128, 8, 1), x[rows], w, 1e-6)
    assert torch.equal(y[rows], ys) and torch.equal(q[0][rows], qs[0]) and torch.equal(q[1][:, rows], qs[1][:, :4])
    assert not y[1].any() and not y[T - 3].any()


@pytest.mark.parametrize("recipe", [0, 1])
def test_linear(recipe):
    T, K, N = 1100000, 128, 2048                          # 2.25e9 outputs
    gen = torch.Generator().manual_seed(1)
    codes, scales, _ = random_weights(gen, K, N, recipe)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    lin = moe.LinearConfig(T, K, N, recipe)
    w = moe.transform_linear_weights(lin, codes.cuda(), scales.cuda())
    y = moe.linear(lin, w, x=x)
    # the last 70000 rows alone run the same kernel
    n = 70000
    tail = moe.linear(moe.LinearConfig(n, K, N, recipe), w, x=x[T - n:])
    assert torch.equal(y[T - n:], tail) and torch.isfinite(y[::1000]).all()
    assert quantize(x[-2:].cpu(), recipe)[0].shape == (2, K)


def test_router():
    T, E, k = 8500000, 256, 2                             # 2.18e9 logits
    g = torch.Generator(device="cuda").manual_seed(3)
    l = torch.randn((T, E), generator=g, device="cuda")
    idx = torch.stack((torch.randint(0, 128, (T,), generator=g, device="cuda"),
                       torch.randint(128, E, (T,), generator=g, device="cuda")), 1).int()
    cfg = moe.Config(T, 128, 128, E, k, renormalize=1)
    loss, counts, tokens, mean = moe.balance_loss(cfg, l, idx, 0.01)
    want = torch.bincount(idx.reshape(-1).long(), minlength=E).int()
    assert torch.equal(counts[0], want) and tokens.tolist() == [T, 1]
    # every mean is 1/E up to sampling: sqrt(var p / T) is far below a thousandth of it
    assert torch.all((mean * E - 1).abs() < 1e-2) and abs(float(loss) / 0.01 - 1) < 1e-2
    dw = torch.randn((T, k), generator=g, device="cuda")
    dl, _ = moe.route_backward(cfg, l, idx, d_topk_weights=dw)
    rows = torch.tensor([0, T // 2, T - 2, T - 1], device="cuda")
    ds, _ = moe.route_backward(moe.Config(4, 128, 128, E, k, renormalize=1), l[rows], idx[rows], d_topk_weights=dw[rows])
    assert torch.equal(dl[rows], ds)


def test_temporaries_on_another_stream():
    """The call's own workspace and outputs are kept until its stream has used them."""
    T, K, N = 4096, 1024, 1024
    codes, scales, _ = random_weights(torch.Generator().manual_seed(4), K, N, 1)
    lin = moe.LinearConfig(T, K, N, 1)
    w = moe.transform_linear_weights(lin, codes.cuda(), scales.cuda())
    x = torch.randn((T, K), device="cuda").bfloat16()
    want = moe.linear(lin, w, x=x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(8):
        y = moe.linear(lin, w, x=x, stream=s)
        junk = [torch.full((T * K + 300000,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]   # would reuse it
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        del junk
