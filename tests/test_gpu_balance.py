"""The balance loss and the router's gradients against 64 bits and against differences: both scores,
ragged, empty and masked sequences, rows behind the last one, every size of expert set."""
import pytest
import torch

import mixture_experts_fp8_b200 as moe
from _block_ref import F64, U, balance, probs, route_weights, token_seq

pytestmark = pytest.mark.gpu
COEF = 0.02
# positive terms: exp, reciprocal and product of p, its sum over the experts, and at most 250
# additions on any token's way through a warp, the warps, the chunks and the division
REL = 300 * U


def problem(T, E, k, S, masked, seed=0):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn((T, E), generator=g) + 0.5 * torch.randn(E, generator=g)
    idx = torch.topk(l, k, dim=1)[1].int()
    if S == 1:
        off = [0, T]
    else:
        end = T - T // 8
        cuts = torch.sort(torch.randint(0, end + 1, (S - 1,), generator=g))[0].tolist()
        off = [min(1, end)] + [max(c, min(1, end)) for c in cuts] + [end]
        if S > 2:
            off[2] = off[1]
    mask = (torch.rand(T, generator=g) < 0.8) if masked else None
    return l, idx, off, mask


def cuda(t):
    return None if t is None else t.cuda()


def run_balance(cfg, l, idx, off, mask, ws=None):
    o = None if off == [0, cfg.num_tokens] else torch.tensor(off, dtype=torch.int32).cuda()
    return moe.balance_loss(cfg, l.cuda(), idx.cuda(), COEF, seq_offsets=o, token_mask=cuda(mask), workspace=ws), o


SHAPES = [(1, 8, 1, 1), (1, 8, 8, 3), (5, 9, 3, 2), (64, 32, 2, 1), (100, 33, 4, 7), (1000, 64, 8, 60), (777, 128, 8, 5),
          (4096, 256, 8, 9), (9000, 100, 6, 1), (500, 256, 40, 3),
          (20000, 12, 3, 300), (6000, 40, 2, 2000), (300000, 8, 2, 40), (5000, 256, 8, 1)]


@pytest.mark.parametrize("routing", [0, 1])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,E,k,S", SHAPES)
def test_balance_against_64_bits(T, E, k, S, masked, routing):
    l, idx, off, mask = problem(T, E, k, S, masked, T + S)
    cfg = moe.Config(T, 128, 128, E, k, routing=routing)
    ws = moe.new_balance_workspace(cfg, S)
    (loss, counts, tokens, mean), _ = run_balance(cfg, l, idx, off, mask, ws)
    assert moe.read_status(ws) == 0
    want, wc, wt, wm = balance(l.to(F64), idx, token_seq(T, off, mask), S, k, routing, COEF)
    assert torch.equal(counts.cpu(), wc) and torch.equal(tokens.cpu(), wt)
    assert torch.all((mean.cpu().to(F64) - wm).abs() <= wm * REL)
    assert abs(float(loss) - float(want)) <= REL * float(want)


@pytest.mark.parametrize("routing,renorm", [(0, 0), (0, 1), (1, 0)])
@pytest.mark.parametrize("parts", ["both", "weights", "loss"])
@pytest.mark.parametrize("T,E,k,S", SHAPES)
def test_gradients_against_64_bits(T, E, k, S, parts, routing, renorm):
    l, idx, off, mask = problem(T, E, k, S, T % 2 == 1, T + S)
    g = torch.Generator().manual_seed(1)
    dw = torch.randn((T, k), generator=g) if parts != "loss" else None
    pes = 0.5 + torch.rand(E, generator=g) if T % 3 else None
    dloss = torch.tensor([1.7]) if parts != "weights" else None
    rsf = 2.5
    cfg = moe.Config(T, 128, 128, E, k, routing=routing, renormalize=renorm, routed_scaling_factor=rsf)
    (_, counts, tokens, _), o = run_balance(cfg, l, idx, off, mask)
    dl, dpes = moe.route_backward(cfg, l.cuda(), idx.cuda(), d_topk_weights=cuda(dw), per_expert_scale=cuda(pes),
                                  d_loss=cuda(dloss), coef=COEF, expert_counts=counts, seq_tokens=tokens, seq_offsets=o,
                                  token_mask=cuda(mask))
    torch.cuda.synchronize()
    # the definition, differentiated in 64 bits
    ld = l.to(F64).requires_grad_(True)
    pd = None if pes is None else pes.to(F64).requires_grad_(True)
    seq = token_seq(T, off, mask)
    total = ld.sum() * 0
    if dloss is not None:
        total = total + 1.7 * balance(ld, idx, seq, S, k, routing, COEF)[0]
    if dw is not None:
        total = total + (route_weights(ld, idx, routing, renorm, pd, rsf) * dw.to(F64)).sum()
    total.backward()
    # what the terms of a gradient weigh before they cancel; 64 roundings each
    p = probs(l.to(F64), routing)
    mag, ref_off = torch.zeros_like(p), torch.zeros((), dtype=F64)
    if dloss is not None:
        n = tokens.cpu()[:S].to(F64).clamp(min=1)[:, None]
        dp = 1.7 * COEF * counts.cpu().to(F64) * E / (k * n * n) / max(1, int(tokens[S]))
        dp = torch.where(seq[:, None] >= 0, dp[seq.clamp(min=0)], torch.zeros((), dtype=F64))
        mag += p * (dp + (p * dp).sum(1, keepdim=True))
    if dw is not None:
        u = route_weights(l.to(F64), idx, routing, renorm, None if pes is None else pes.to(F64), rsf)
        t = u * dw.to(F64).abs()
        mag = mag.scatter_add(1, idx.long(), t + u * t.sum(1, keepdim=True) / u.sum(1, keepdim=True))
        if routing == 0 and not renorm:
            mag += p * t.sum(1, keepdim=True)
        # the 64-bit reference's own rounding: differentiating u = p_j / sum p gives an expert that was not
        # selected p_e * sum_j p_j g_j, which is 0 but is summed with at most 2 k + 8 <= 88 < 2^7 roundings
        # of 2^-53 of terms that weigh t together
        ref_off = 2.0 ** -46 * t.sum(1, keepdim=True)
    got = dl.cpu().to(F64)
    assert torch.all((got - ld.grad).abs() <= 64 * U * mag + ref_off + 1e-38)
    if pes is not None and dw is not None:
        w = (route_weights(l.to(F64), idx, routing, renorm, None, rsf) * dw.to(F64).abs())
        weigh = torch.zeros(E, dtype=F64).index_add_(0, idx.long().reshape(-1), w.reshape(-1))
        assert torch.all((dpes.cpu().to(F64) - pd.grad).abs() <= REL * weigh + 1e-38)


def test_gradient_against_differences():
    """Along a random direction, central differences of the 64-bit loss."""
    T, E, k, S = 60, 16, 3, 4
    l, idx, off, mask = problem(T, E, k, S, True, 5)
    g = torch.Generator().manual_seed(2)
    dw, pes = torch.randn((T, k), generator=g), 0.5 + torch.rand(E, generator=g)
    for routing, renorm in ((0, 0), (0, 1), (1, 0)):
        cfg = moe.Config(T, 128, 128, E, k, routing=routing, renormalize=renorm)
        (_, counts, tokens, _), o = run_balance(cfg, l, idx, off, mask)
        dl, dpes = moe.route_backward(cfg, l.cuda(), idx.cuda(), d_topk_weights=dw.cuda(), per_expert_scale=pes.cuda(),
                                      d_loss=torch.ones(1).cuda(), coef=COEF, expert_counts=counts, seq_tokens=tokens,
                                      seq_offsets=o, token_mask=mask.cuda())
        seq = token_seq(T, off, mask)

        def f(a, b):
            return float(balance(a, idx, seq, S, k, routing, COEF)[0] +
                         (route_weights(a, idx, routing, renorm, b, 1.0) * dw.to(F64)).sum())
        for _ in range(4):
            va, vb = torch.randn((T, E), generator=g).to(F64), torch.randn(E, generator=g).to(F64)
            h = 1e-5
            diff = (f(l.to(F64) + h * va, pes.to(F64) + h * vb) - f(l.to(F64) - h * va, pes.to(F64) - h * vb)) / (2 * h)
            got = float((dl.cpu().to(F64) * va).sum() + (dpes.cpu().to(F64) * vb).sum())
            # h^2 of the differences, and the gradient's fp32 roundings over T * E values
            assert abs(got - diff) <= 1e-5 * float((dl.cpu().to(F64) * va).abs().sum() + 1)


def test_masked_rows_may_hold_anything():
    """Rows of NaN and infinities that are masked, or behind the last sequence, and experts at -inf."""
    T, E, k, S = 40, 24, 4, 2
    for routing in (0, 1):
        l, idx, _, _ = problem(T, E, k, 1, False, 6)
        off = [0, 13, 30]
        mask = torch.ones(T, dtype=torch.bool)
        mask[[0, 12, 20]] = False
        l[5, 3] = l[20, 1] = float("-inf")
        idx[5] = torch.tensor([0, 1, 2, 4], dtype=torch.int32)
        bad, bad_idx = l.clone(), idx.clone()
        bad[[0, 31]] = float("nan")
        bad[[12, 39]] = float("inf")
        bad_idx[0] = 1 << 30
        cfg = moe.Config(T, 128, 128, E, k, routing=routing)
        ws = moe.new_balance_workspace(cfg, S)
        (loss, counts, tokens, mean), o = run_balance(cfg, bad, bad_idx, off, mask, ws)
        assert moe.read_status(ws) == 0
        want, wc, wt, wm = balance(l.to(F64), idx, token_seq(T, off, mask), S, k, routing, COEF)
        assert torch.equal(counts.cpu(), wc) and torch.equal(tokens.cpu(), wt)
        assert torch.all((mean.cpu().to(F64) - wm).abs() <= wm * REL) and abs(float(loss) - float(want)) <= REL * float(want)
        dw = torch.randn((T, k), generator=torch.Generator().manual_seed(1))
        dw[[0, 12, 31, 39]] = 0
        dl, _ = moe.route_backward(cfg, bad.cuda(), bad_idx.cuda(), d_topk_weights=dw.cuda(), d_loss=torch.ones(1).cuda(),
                                   coef=COEF, expert_counts=counts, seq_tokens=tokens, seq_offsets=o, token_mask=mask.cuda())
        torch.cuda.synchronize()
        assert torch.all(dl[[0, 12, 31, 39]] == 0) and torch.isfinite(dl).all()


def test_nothing_counted():
    T, E, k = 10, 16, 2
    l, idx, _, _ = problem(T, E, k, 1, False, 7)
    cfg = moe.Config(T, 128, 128, E, k)
    for off, mask in (([0, T], torch.zeros(T, dtype=torch.bool)), ([4, 4, 4], None)):
        (loss, counts, tokens, mean), o = run_balance(cfg, l, idx, off, mask)
        assert float(loss) == 0 and not counts.any() and not tokens.any() and not mean.any()
        dl, _ = moe.route_backward(cfg, l.cuda(), idx.cuda(), d_loss=torch.ones(1).cuda(), coef=COEF, expert_counts=counts,
                                   seq_tokens=tokens, seq_offsets=o, token_mask=cuda(mask))
        assert not dl.any()


def test_bad_ids_and_offsets_are_reported():
    T, E, k = 50, 16, 2
    l, idx, _, _ = problem(T, E, k, 1, False, 8)
    cfg = moe.Config(T, 128, 128, E, k)
    ws = moe.new_balance_workspace(cfg, 2)
    bad = idx.clone()
    bad[7, 1], bad[8, 0] = E, -1
    (_, counts, _, _), _ = run_balance(cfg, l, bad, [0, T], None, ws)
    assert moe.read_status(ws) == moe.MOE_ERR_BOUNDS and int(counts.sum()) == T * k - 2
    dl, _ = moe.route_backward(cfg, l.cuda(), bad.cuda(), d_topk_weights=torch.ones((T, k)).cuda())
    assert torch.isfinite(dl).all()
    for off in ([0, 30, 20], [0, 20, T + 1], [-1, 20, T]):
        run_balance(cfg, l, idx, off, None, ws)
        assert moe.read_status(ws) == moe.MOE_ERR_BOUNDS
    run_balance(cfg, l, idx, [0, 20, T], None, ws)
    assert moe.read_status(ws) == 0


def test_same_bits_every_time_and_captured():
    T, E, k, S = 5000, 128, 8, 11
    l, idx, off, mask = problem(T, E, k, S, True, 9)
    pes = (0.5 + torch.rand(E)).cuda()
    cfg = moe.Config(T, 128, 128, E, k, renormalize=1)
    l, idx, mask = l.cuda(), idx.cuda(), mask.cuda()
    o = torch.tensor(off, dtype=torch.int32).cuda()
    dw = torch.randn((T, k), generator=torch.Generator().manual_seed(4)).cuda()
    ws = moe.new_balance_workspace(cfg, S)

    def step():
        loss, counts, tokens, mean = moe.balance_loss(cfg, l, idx, COEF, seq_offsets=o, token_mask=mask, workspace=ws)
        dl, dp = moe.route_backward(cfg, l, idx, d_topk_weights=dw, per_expert_scale=pes, d_loss=torch.ones_like(loss),
                                    coef=COEF, expert_counts=counts, seq_tokens=tokens, seq_offsets=o, token_mask=mask,
                                    workspace=ws)
        return loss, counts, tokens, mean, dl, dp
    first = step()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, step()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for t in outs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))


def test_training_step_of_the_router():
    """gate -> layer, and the loss and gradients from the gate's own ids and logits."""
    T, E, k, H = 96, 16, 4, 256
    g = torch.Generator().manual_seed(12)
    x = torch.randn((T, H), generator=g).bfloat16().cuda()
    cfg = moe.Config(T, H, 128, E, k, routing=1, group_count=4, k_group=2, group_select_mode=1, routed_scaling_factor=2.5)
    gw = moe.transform_gate_weights(cfg, torch.ones(H).cuda(), (torch.randn((E, H), generator=g) / 16).cuda())
    logits, idx, w = moe.gate(cfg, x, gw, 1e-6)
    loss, counts, tokens, mean = moe.balance_loss(cfg, logits, idx, COEF)
    dw = torch.randn((T, k), generator=g).cuda()
    dl, _ = moe.route_backward(cfg, logits, idx, d_topk_weights=dw, d_loss=torch.ones(1).cuda(), coef=COEF,
                               expert_counts=counts, seq_tokens=tokens)
    torch.cuda.synchronize()
    ld = logits.cpu().to(F64).requires_grad_(True)
    seq = token_seq(T, [0, T], None)
    want = balance(ld, idx.cpu(), seq, 1, k, 1, COEF)[0]
    rw = route_weights(ld, idx.cpu(), 1, 0, None, 2.5)
    assert torch.all((w.cpu().to(F64) - rw).abs() <= 2e-6 * rw.clamp(min=1))
    assert abs(float(loss) - float(want)) <= REL * float(want) and int(counts.sum()) == T * k
    (want + (rw * dw.cpu().to(F64)).sum()).backward()
    assert torch.all((dl.cpu().to(F64) - ld.grad).abs() <= 64 * U * 2.5 * dw.cpu().abs().sum(1, keepdim=True))


def test_one_slot_has_no_gradient_through_its_normalized_weight():
    """k = 1: the normalized weight is 1 whatever the logit, so only the balance loss moves the logits."""
    T, E = 300, 24
    for routing, renorm in ((1, 0), (0, 1)):
        l, idx, off, mask = problem(T, E, 1, 1, False, 10)
        cfg = moe.Config(T, 128, 128, E, 1, routing=routing, renormalize=renorm)
        (_, counts, tokens, _), _ = run_balance(cfg, l, idx, off, mask)
        args = dict(d_loss=torch.ones(1).cuda(), coef=COEF, expert_counts=counts, seq_tokens=tokens)
        dw = torch.randn((T, 1), generator=torch.Generator().manual_seed(3)).cuda()
        a, _ = moe.route_backward(cfg, l.cuda(), idx.cuda(), **args)
        b, _ = moe.route_backward(cfg, l.cuda(), idx.cuda(), d_topk_weights=dw, **args)
        c, _ = moe.route_backward(cfg, l.cuda(), idx.cuda(), d_topk_weights=dw)
        assert torch.equal(a, b) and not c.any()
