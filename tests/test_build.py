"""When the build takes the extension module of the attention calls to be stale
(no GPU needed; nothing is compiled)."""
import importlib.util
import os

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
