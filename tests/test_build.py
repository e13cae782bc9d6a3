"""When the build takes the extension module of the attention calls to be stale
(no GPU needed; nothing is compiled)."""
import importlib.util
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def build_script():
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(ROOT, "bit_dequant_expert_b200", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_binding_is_fresh_for_what_it_was_built_for():
    b = build_script()
    assert os.path.exists(b.BINDING) and not b.binding_stale()


def test_binding_is_stale_for_another_torch_python_or_compiler(monkeypatch, tmp_path):
    b = build_script()
    with monkeypatch.context() as mp:
        mp.setattr(b.importlib.metadata, "version", lambda name: "1.2.3")
        assert b.binding_stale()
    with monkeypatch.context() as mp:
        mp.setattr(b, "_torch_dir", lambda: str(tmp_path))
        assert b.binding_stale()
    with monkeypatch.context() as mp:
        mp.setattr(b.sys, "version", "another")
        assert b.binding_stale()
    with monkeypatch.context() as mp:
        cxx = tmp_path / "cxx"
        cxx.write_text("#!/bin/sh\necho another compiler\n")
        cxx.chmod(0o755)
        mp.setenv("CXX", str(cxx))
        assert b.binding_stale()
    with monkeypatch.context() as mp:
        mp.setattr(b, "BINDING_FOR", str(tmp_path / "none"))
        assert b.binding_stale()
    assert not b.binding_stale()


def test_without_the_attention_binding_the_other_calls_run():
    """A module that does not load (here: one that is hidden) costs the
    attention calls, which say so, and nothing else."""
    code = """
import sys
sys.modules["bit_dequant_expert_b200._attn_binding"] = None       # importing it raises ImportError
import bit_dequant_expert_b200 as m
assert m.moe_workspace_size(m.config(), 4) > 0
assert m.moe_combine(m.config(), 0, 0, None, None, None, None, None, stream=0, raise_on_error=False) == m.MOE_ERR_INVALID_ARG
for call in (lambda: m.attn_decode_workspace_size(m.attn_config(), 1, 1, 1), lambda: m.AttentionLayer(16, 2, 128, 4)):
    try:
        call()
    except ImportError as e:
        assert "attn_decode_workspace_size" in str(e) and "build.py" in str(e)
    else:
        raise SystemExit("no error")
"""
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True, timeout=300)
