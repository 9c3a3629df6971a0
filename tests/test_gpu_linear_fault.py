"""Failure detection inside the dense product, without a GPU fault: in the debug library an armed fault makes
CTA 0 drop its first K stage (every cluster's first CTA, in the kernel for few tokens).  A bounded wait runs
out, every role leaves, the status word reads MOE_ERR_TIMEOUT, what was not computed is NaN (in place of a
residual too), the rest is as ever, and the next call works.  In a child process, which loads that library."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# (kernel, T, K, N, recipe): few tokens with K split and whole; tiles of 256 and 512 tokens, of 192 and 256 columns;
# few and many K groups for the ring; outputs that leave by TMA and by words; one and several units a pair
CASES = [("narrow", 16, 1024, 256, 0), ("narrow", 64, 1024, 250, 1), ("narrow", 5, 128, 9600, 0), ("narrow", 5, 128, 96, 2),
         ("pair", 300, 768, 514, 0), ("pair", 300, 768, 512, 0), ("pair", 1024, 1024, 4736, 0), ("pair", 1024, 1024, 4730, 0),
         ("pair", 700, 256, 264, 1), ("pair", 1300, 384, 4965, 1), ("pair", 2048, 1152, 4096, 1), ("pair", 1500, 1024, 4738, 2)]

CHILD = r"""
import json, sys, torch
sys.path.insert(0, ROOT); sys.path.insert(0, ROOT + "/tests")
import mixture_experts_fp8_b200 as moe
from mixture_experts_fp8_b200 import build as b
moe.LIB_PATH = b.build(debug=True)
from _block_ref import random_weights
out = []
for kind, T, K, N, recipe in CASES:
    g = torch.Generator().manual_seed(T + N)
    codes, scales, _ = random_weights(g, K, N, recipe)
    x = torch.randn((T, K), generator=g).bfloat16().cuda()
    res = torch.randn((T, N), generator=g).bfloat16().cuda()
    cfg = moe.LinearConfig(T, K, N, recipe)
    w = moe.transform_linear_weights(cfg, codes.cuda(), scales.cuda())
    ws = moe.new_linear_workspace(cfg)
    def call():
        y = res.clone()
        moe.linear(cfg, w, x=x, residual=y, y=y, workspace=ws)
        return y, moe.read_status(ws)
    want, s0 = call()
    moe.debug_inject_fault(moe.MOE_FAULT_SKIP_STAGE)
    y, s1 = call()
    again, s2 = call()
    nan = torch.isnan(y)
    out.append([s0, s1, s2, bool(torch.equal(again, want)), bool(torch.equal(y[~nan], want[~nan])),
                bool(nan[:128, :128].all()), bool(nan.all()), bool(torch.isfinite(want).all())])
print(json.dumps(out))
"""


def test_injected_stage_loss_leaves_nan_and_recovers():
    import mixture_experts_fp8_b200 as moe
    code = f"ROOT = {ROOT!r}\nCASES = {CASES!r}\n" + CHILD
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-3000:]
    for case, (s0, s1, s2, same, rest, first, every, finite) in zip(CASES, json.loads(r.stdout.strip().splitlines()[-1])):
        assert finite and s0 == 0, case              # no fault armed
        assert s1 == moe.MOE_ERR_TIMEOUT, case
        assert first and rest, case                  # the first tile is NaN, all that is not NaN is right
        # few tokens: all of it; one unit a pair: the others' units are there
        assert every == (case[0] == "narrow"), case
        assert s2 == 0 and same, case
