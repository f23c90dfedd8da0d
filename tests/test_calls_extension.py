"""The package does without the extension of csrc/calls.cpp: where it does not load, and where it
cannot be built, for whatever reason."""

import os
import stat
import subprocess
import sys
import textwrap

import pytest

from conftest import ROOT, load_builder


def test_an_extension_that_does_not_load(tmp_path):
    """A file that is no library in the extension's place: a warning, and the calls in Python."""
    broken = tmp_path / "_rf_calls.so"
    broken.write_bytes(b"not a library")
    code = textwrap.dedent(f"""
        import importlib, sys, warnings
        sys.path.insert(0, {ROOT!r})
        import importlib.util
        spec = importlib.util.spec_from_file_location("cascaded_reductions_gb300._build",
                                                      {os.path.join(ROOT, "cascaded_reductions_gb300", "_build.py")!r})
        build = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(build)
        build.calls_path = lambda: ({str(broken)!r}, None)
        sys.modules["cascaded_reductions_gb300._build"] = build
        with warnings.catch_warnings(record=True) as seen:
            warnings.simplefilter("always")
            import cascaded_reductions_gb300 as rf
        assert rf._calls is None
        assert any("does not load" in str(w.message) for w in seen), seen
        import torch
        try:
            rf.attn_decode_window(torch.zeros(2, 8, 128), torch.zeros(2, 2, 9, 128), torch.zeros(2, 2, 9, 128))
        except ValueError:
            print("works")
    """)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=str(tmp_path))
    assert r.returncode == 0 and "works" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("compiler", ["#!/bin/sh\nexit 9\n", "#!/bin/sh\nkill -9 $$\n", None])
def test_a_compiler_that_fails_without_a_word(tmp_path, monkeypatch, capfd, compiler):
    b = load_builder()
    path = tmp_path / "_rf_calls.so"
    path.write_bytes(b"of an older header")
    os.utime(path, (1, 1))
    cxx = tmp_path / "cxx"
    if compiler is not None:
        cxx.write_text(compiler)
        cxx.chmod(cxx.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("CXX", str(cxx))
    _, torch = b.calls_path()
    monkeypatch.setattr(b, "calls_path", lambda: (str(path), torch))
    assert b.build_calls() is None
    assert "calls.cpp not built" in capfd.readouterr().out
    assert not path.exists() and sorted(p.name for p in tmp_path.iterdir()) == (["cxx"] if compiler else [])
