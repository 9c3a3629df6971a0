"""The marshalling of the operators around the layer: arguments that are refused before any launch, and references."""
import sys

import pytest
import torch

import mixture_experts_fp8_b200 as moe

T, H, E, K = 4, 256, 8, 2
X = torch.zeros(T, H, dtype=torch.bfloat16)
LOGITS, IDX = torch.zeros(T, E), torch.zeros(T, K, dtype=torch.int32)


def cfg(**kw):
    return moe.Config(**{**dict(num_tokens=T, hidden=H, inter=128, num_experts=E, top_k=K), **kw})


def calls(x, config=cfg(), lin=moe.LinearConfig(T, H, 64)):
    q = (x, torch.zeros(2, 8, dtype=torch.int32))
    return {"add_rms_norm": lambda: moe.add_rms_norm(config, x, torch.ones(H), 1e-6),
            "linear of rows": lambda: moe.linear(lin, q, x=x),
            "linear of codes": lambda: moe.linear(lin, q, quantized=q),
            "balance_loss": lambda: moe.balance_loss(config, x, IDX, 0.1),
            "route_backward": lambda: moe.route_backward(config, x, IDX)}


def refused(f, *words):
    with pytest.raises(moe.MoeError) as e:
        f()
    assert e.value.code == moe.MOE_ERR_INVALID_ARG
    assert all(w in str(e.value) for w in words), str(e.value)


@pytest.mark.parametrize("name", calls(X))
def test_host_tensors_and_other_objects_are_refused(name):
    refused(calls(X)[name], "is on cpu")
    for other in (X.float().numpy(), 7, "x"):
        refused(calls(other)[name], "must be a tensor")


@pytest.mark.parametrize("name", calls(X))
def test_config_numbers(name):
    big = calls(X, cfg(num_tokens=2 ** 32 + T), moe.LinearConfig(2 ** 32 + T, H, 64))
    refused(big[name], "num_tokens", "32 bits")
    with pytest.raises((TypeError, ValueError)):
        calls(X, cfg(num_tokens=None), moe.LinearConfig(None, H, 64))[name]()
    with pytest.raises(AttributeError):
        calls(X, object(), object())[name]()


def test_one_kind_of_rows_and_a_pair():
    lin, w = moe.LinearConfig(T, H, 64), (X, X)
    refused(lambda: moe.linear(lin, w), "exactly one")
    refused(lambda: moe.linear(lin, w, x=X, quantized=(X, X)), "exactly one")
    for bad in ((), [], X, 3):
        refused(lambda: moe.linear(lin, w, quantized=bad), "pair")


def test_refusals_keep_no_references():
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    fs = list(calls(x).values())
    n = sys.getrefcount(x)
    for _ in range(50):
        for f in fs:
            with pytest.raises(moe.MoeError):
                f()
    assert sys.getrefcount(x) == n


@pytest.mark.gpu
def test_results_are_freed_and_inputs_not_kept():
    dev = "cuda"
    config, lin = cfg(), moe.LinearConfig(T, H, 64)
    x, l, idx = X.to(dev), LOGITS.to(dev), IDX.to(dev)
    idx[:, 1] = 1
    w = torch.ones(H, device=dev)
    weights = moe.transform_linear_weights(lin, torch.zeros((H, 64), dtype=torch.uint8, device=dev), torch.ones((H // 128, 64), device=dev))
    q = moe.add_rms_norm(config, x, w, 1e-6)[2]
    side = torch.cuda.Stream()
    dw, dl, pes = torch.ones((T, K), device=dev), torch.ones(1, device=dev), torch.ones(E, device=dev)

    def once(stream=None):
        moe.add_rms_norm(config, x, w, 1e-6, stream=stream)
        moe.add_rms_norm(config, x, w, 1e-6, residual=x, quantized=q, stream=stream)
        moe.linear(lin, weights, x=x, stream=stream)
        moe.linear(lin, list(weights), quantized=list(q), residual=None, stream=stream)
        loss, counts, tokens, mean = moe.balance_loss(config, l, idx, 0.1, stream=stream)
        moe.route_backward(config, l, idx, dw, pes, dl, 0.1, counts, tokens, stream=stream)

    def settle():
        torch.cuda.synchronize()
        torch.empty(1, device=dev)          # the allocator frees what other streams were done with
        return torch.cuda.memory_allocated()

    once()
    refs = [sys.getrefcount(t) for t in (x, l, idx, w, q, dw, dl, pes, *q, *weights)]
    before = settle()
    for _ in range(20):
        once()
        once(side)
    assert settle() == before
    assert refs == [sys.getrefcount(t) for t in (x, l, idx, w, q, dw, dl, pes, *q, *weights)]


@pytest.mark.gpu
def test_config_numbers_of_other_types():
    x, w = torch.randn(T, H, device="cuda").bfloat16(), torch.ones(H, device="cuda")
    a = moe.add_rms_norm(cfg(), x, w, 1e-6)[1]
    n = torch.tensor(T)
    b = moe.add_rms_norm(cfg(num_tokens=n, hidden=n.numpy().dtype.type(H), routed_scaling_factor=1), x, w, n.new_tensor(1e-6, dtype=torch.float64))[1]
    assert torch.equal(a, b)


@pytest.mark.gpu
def test_calls_from_two_threads():
    """Each thread with a stream and a workspace of its own; a refusal in one leaves the other's calls alone."""
    import threading
    lin = moe.LinearConfig(T, H, 64)
    w = moe.transform_linear_weights(lin, torch.full((H, 64), 56, dtype=torch.uint8, device="cuda"), torch.ones((H // 128, 64), device="cuda"))
    nw = torch.ones(H, device="cuda")
    xs = [torch.randn(T, H, device="cuda").bfloat16() for _ in range(2)]
    want = [moe.linear(lin, w, x=moe.add_rms_norm(cfg(), x, nw, 1e-6)[1]) for x in xs]
    torch.cuda.synchronize()
    wrong = [0, 0]

    def run(i):
        s, ws = torch.cuda.Stream(), moe.new_linear_workspace(lin)
        with torch.cuda.stream(s):
            for _ in range(200):
                y = moe.linear(lin, w, x=moe.add_rms_norm(cfg(), xs[i], nw, 1e-6)[1], workspace=ws)
                try:
                    moe.linear(lin, w, x=xs[i], workspace=ws[:512])
                    wrong[i] += 1
                except moe.MoeError as e:
                    wrong[i] += "512 bytes" not in str(e)
            s.synchronize()
            wrong[i] += not torch.equal(y, want[i])

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0, 0]
