"""The operators around the layer on a machine without a GPU: sizes, and every refusal before any CUDA
call, with a message."""
import ctypes

import pytest
import torch

import mixture_experts_fp8_b200 as moe

BAD, UNS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
_buf = ctypes.create_string_buffer(8192)
AL = (ctypes.addressof(_buf) + 255) & ~255


def cfg(**kw):
    return moe.Config(**(dict(num_tokens=16, hidden=256, inter=128, num_experts=8, top_k=2) | kw))


def refused(fn, code, word):
    rc = fn()
    assert rc == code and word in moe.lib().moe_last_error(), (rc, moe.lib().moe_last_error())


def test_sizes():
    codes, scales, rows = moe.quantized_size(5, 384)
    assert codes == 5 * 384 and rows == 140 and scales == 3 * 140 * 4
    q, s = moe.new_quantized(5, 384, device="cpu")
    assert q.shape == (5, 384) and s.shape == (3, 140)
    for recipe, pk in ((0, 1), (1, 1), (2, 2)):
        c = moe.LinearConfig(3, 256, 130, recipe)
        w, ws = moe.transformed_linear_size(c)
        assert w * pk == 256 * 130 and ws == 2 * 256 * 4          # columns padded to 256 in the scales
        assert moe.linear_workspace_size(c) == moe.MOE_LINEAR_STATUS_BYTES + 1024 + 2 * 136 * 4
    assert moe.balance_workspace_size(cfg(), 1) < moe.balance_workspace_size(cfg(), 1000)


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=0), BAD), (dict(in_features=0), BAD), (dict(out_features=-4), BAD), (dict(recipe=3), BAD),
    (dict(activation=5), BAD), (dict(activation=-1), BAD), (dict(in_features=200), UNS),
    (dict(recipe=2, out_features=7), UNS), (dict(num_tokens=1 << 25), UNS), (dict(out_features=1 << 21), UNS),
])
def test_linear_config(kw, code):
    c = moe.LinearConfig(**(dict(num_tokens=4, in_features=256, out_features=64) | kw))
    for f in (moe.transformed_linear_size, moe.linear_workspace_size):
        with pytest.raises(moe.MoeError) as e:
            f(c)
        assert e.value.code == code and len(str(e.value)) > 10


def test_norm_refusals():
    lib, c, f = moe.lib(), ctypes.byref(cfg().c()), ctypes.c_float

    def call(x=AL, res=None, w=AL, eps=1e-6, ro=None, y=AL, q=None, s=None, c=c):
        return lambda: lib.moe_add_rms_norm(c, x, res, 0, w, f(eps), ro, y, q, s, None)
    refused(call(x=None), BAD, b"NULL")
    refused(call(w=None), BAD, b"NULL")
    refused(call(q=AL), BAD, b"both codes and scales")
    refused(call(y=None), BAD, b"no output")
    refused(call(ro=AL), BAD, b"needs a residual")
    for name in ("x", "res", "w", "y"):
        refused(call(**{name: AL | 8}), BAD, b"16-byte")
    refused(call(q=AL | 4, s=AL), BAD, b"16-byte")
    refused(lambda: lib.moe_add_rms_norm(c, AL, AL | 16, 1, AL, f(1e-6), None, AL, None, None, None), BAD, b"32-byte")
    for eps in (-1.0, float("nan")):
        refused(call(eps=eps), BAD, b"rms_eps")
    refused(call(c=ctypes.byref(cfg(hidden=32768 + 128).c())), UNS, b"32768")
    refused(call(c=ctypes.byref(cfg(num_tokens=0).c())), BAD, b"num_tokens")
    refused(lambda: lib.moe_quantized_size(0, 128, None, None, None), BAD, b"rows")
    refused(lambda: lib.moe_quantized_size(4, 100, None, None, None), UNS, b"128")


def test_linear_refusals():
    lib = moe.lib()
    c = ctypes.byref(moe.LinearConfig(4, 256, 64).c())
    need = moe.linear_workspace_size(moe.LinearConfig(4, 256, 64))

    def call(x=AL, q=None, s=None, w=AL, ws=AL, b=None, r=None, y=AL, wk=AL, n=need):
        return lambda: lib.moe_linear(c, x, q, s, w, ws, b, r, y, wk, n, None)
    for name in ("w", "ws", "y", "wk"):
        refused(call(**{name: None}), BAD, b"NULL")
    refused(call(q=AL, s=AL), BAD, b"exactly one")
    refused(call(x=None), BAD, b"exactly one")
    refused(call(x=None, q=AL), BAD, b"exactly one")
    refused(call(s=AL), BAD, b"exactly one")
    for name, off in (("x", 8), ("w", 16), ("ws", 8), ("b", 2), ("r", 8), ("y", 4), ("wk", 128)):
        refused(call(**{name: AL + off}), BAD, b"misaligned")
    refused(call(n=need - 1), BAD, b"workspace has")
    refused(call(x=None, q=AL, s=AL, n=moe.MOE_LINEAR_STATUS_BYTES - 1), BAD, b"workspace has")
    refused(lambda: lib.moe_transform_linear_weights(c, AL, AL, None, AL, None), BAD, b"NULL")
    refused(lambda: lib.moe_transform_linear_weights(c, AL, AL, AL + 16, AL, None), BAD, b"misaligned")


def test_router_refusals():
    lib, c, f = moe.lib(), ctypes.byref(cfg().c()), ctypes.c_float
    need = moe.balance_workspace_size(cfg(), 2)

    def loss(l=AL, i=AL, off=AL, S=2, counts=AL, out=AL, wk=AL, n=need):
        return lambda: lib.moe_balance_loss(c, l, i, None, off, S, f(0.1), counts, AL, AL, out, wk, n, None)
    for name in ("l", "i", "counts", "out", "wk"):
        refused(loss(**{name: None}), BAD, b"NULL")
    refused(loss(S=0), BAD, b"num_seqs")
    refused(loss(off=None), BAD, b"need seq_offsets")
    refused(loss(l=AL + 2), BAD, b"misaligned")
    refused(loss(wk=AL + 64), BAD, b"misaligned")
    refused(loss(n=need - 1), BAD, b"workspace has")

    def back(l=AL, i=AL, dw=AL, dl=AL, counts=AL, off=AL, S=2, out=AL, pes=None, dp=None, wk=None, n=0):
        return lambda: lib.moe_route_backward(c, l, pes, i, dw, dl, f(0.1), counts, AL, None, off, S, out, dp, wk, n, None)
    for name in ("l", "i", "out"):
        refused(back(**{name: None}), BAD, b"NULL")
    refused(back(dw=None, dl=None), BAD, b"one of")
    refused(back(counts=None), BAD, b"expert_counts")
    refused(back(off=None), BAD, b"need seq_offsets")
    refused(back(dp=AL, wk=AL, n=need), BAD, b"per_expert_scale")
    refused(back(pes=AL, dp=AL), BAD, b"workspace")
    refused(back(pes=AL, dp=AL, wk=AL, n=need - 1), BAD, b"workspace has")
    refused(back(out=AL + 1), BAD, b"misaligned")


def test_python_refuses_tensors_elsewhere():
    x = torch.zeros((16, 256), dtype=torch.bfloat16)
    for call in (lambda: moe.add_rms_norm(cfg(), x, torch.ones(256), 1e-6),
                 lambda: moe.linear(moe.LinearConfig(16, 256, 64), (x, x), x=x),
                 lambda: moe.balance_loss(cfg(), torch.zeros((16, 8)), torch.zeros((16, 2), dtype=torch.int32), 0.1)):
        with pytest.raises((moe.MoeError, RuntimeError, AssertionError)):
            call()
    with pytest.raises(moe.MoeError):
        moe.linear(moe.LinearConfig(16, 256, 64), (x, x))
