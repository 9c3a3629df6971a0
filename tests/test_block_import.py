"""The package on a machine without PyTorch: its host calls, and the build of the C library."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    r = subprocess.run([sys.executable, "-c", "import sys; sys.modules['torch'] = None\n" + code], capture_output=True,
                       text=True, cwd=ROOT, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout


def test_host_calls():
    out = run("""
import mixture_experts_fp8_b200 as moe
from mixture_experts_fp8_b200 import ep
cfg = moe.Config(16, 256, 128, 8, 2)
moe.check_config(cfg)
print(moe.workspace_size(cfg) > 0, moe.workspace_layout(cfg)["status"], moe.quantized_size(5, 384)[2],
      moe.linear_workspace_size(moe.LinearConfig(3, 256, 130)), moe.balance_workspace_size(cfg, 3) > 0)
""")
    assert out.split() == ["True", "0", "140", str(1024 + 1024 + 2 * 136 * 4), "True"]


def test_build_of_the_library():
    out = run("import runpy; sys.argv = ['build']; runpy.run_module('mixture_experts_fp8_b200.build', run_name='__main__')")
    assert "libmoefp8.so" in out and "_binding" not in out


def test_a_module_built_for_another_pytorch_is_built_again(monkeypatch, tmp_path):
    import mixture_experts_fp8_b200 as moe
    from mixture_experts_fp8_b200 import build
    build.build_binding()
    moe._bind()
    assert build.binding_matches()
    other = tmp_path / "binding.for"
    monkeypatch.setattr(build, "BINDING_FOR", str(other))
    assert not build.binding_matches()
    other.write_text("torch 1.0.0, cpython-38\n")
    assert not build.binding_matches()
    called = []
    monkeypatch.setattr(build, "build_binding", lambda force=False: called.append(force))
    monkeypatch.setattr(moe, "_bound", None)
    moe._bind()
    assert called == [True]
