"""The build's two parts: the C library needs neither torch nor a host C++ compiler, and is in place even where the
binding's part fails.  The compilers are stubs that write what they are asked for."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import sys
sys.modules["torch"] = None                       # importing it raises
sys.path.insert(0, {root!r})
import dispatch_fp8_grouped_topk_amd.build as b
b.BUILD, b.LIB, b.BINDING, b.HIPCC = {tmp!r} + "/o", {tmp!r} + "/lib.so", {tmp!r} + "/binding.so", {tmp!r} + "/hipcc"
{call}
"""


def _run(tmp_path, call):
    stub = tmp_path / "hipcc"
    stub.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\necho made > "$2"\n')
    stub.chmod(0o755)
    env = dict(os.environ, CXX="/nonexistent/c++")
    return subprocess.run([sys.executable, "-c", SCRIPT.format(root=ROOT, tmp=str(tmp_path), call=call)], env=env,
                          capture_output=True, text=True, timeout=120)


def test_the_library_builds_without_torch(tmp_path):
    r = _run(tmp_path, "b.build(binding=False)")
    assert r.returncode == 0, r.stderr
    assert (tmp_path / "lib.so").exists() and not (tmp_path / "binding.so").exists()


def test_the_library_is_in_place_where_the_binding_fails(tmp_path):
    r = _run(tmp_path, "b.build()")
    assert r.returncode != 0 and (tmp_path / "lib.so").exists() and not (tmp_path / "binding.so").exists()


def test_unknown_options_are_refused():
    r = subprocess.run([sys.executable, "-m", "dispatch_fp8_grouped_topk_amd.build", "--what"], cwd=ROOT,
                       capture_output=True, text=True, timeout=120)
    assert r.returncode != 0 and "--library-only" in r.stderr


def test_a_missing_binding_says_how_to_build_it(monkeypatch):
    import dispatch_fp8_grouped_topk_amd as mm
    monkeypatch.setattr(mm, "_binding_module", None)
    monkeypatch.setattr(mm, "_load", lambda: None)
    monkeypatch.setattr(mm, "HERE", "/nonexistent")
    with pytest.raises(ImportError, match="amd.build"):
        mm._compiled()
