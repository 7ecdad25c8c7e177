"""The library is built and used without torch and without the extension over it; the
extension is rebuilt for another torch."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "static_sparse_attention_b200")


@pytest.fixture
def builder():
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("_builder_under_test", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_the_library_builds_without_torch(builder, monkeypatch):
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else real(name, *a))
    assert builder.build_binding(force=True) is None
    assert builder.build() == builder.LIB
    # stale: the library is compiled all the same, the extension is not
    ran = []
    monkeypatch.setattr(builder, "_stale", lambda lib: True)
    monkeypatch.setattr(builder.subprocess, "check_call", lambda cmd: ran.append(cmd[0]))
    monkeypatch.setattr(builder.os, "replace", lambda a, b: None)
    assert builder.build(debug=True) == builder.LIB_DEBUG
    assert ran == [builder.nvcc()]


def test_the_extension_follows_torch(builder, monkeypatch, tmp_path):
    ran = []
    monkeypatch.setattr(builder, "BINDING_TORCH", str(tmp_path / "made_for" / "torch"))
    monkeypatch.setattr(builder.subprocess, "check_call", lambda cmd: ran.append(cmd[0]))
    monkeypatch.setattr(builder.os, "replace", lambda a, b: None)
    assert builder.build_binding() == builder.BINDING and len(ran) == 1   # nothing says which torch it was for
    assert builder.build_binding() == builder.BINDING and len(ran) == 1
    monkeypatch.setattr(builder, "_torch_version", lambda torch: "another")
    assert builder.build_binding() == builder.BINDING and len(ran) == 2
    assert builder.build_binding() == builder.BINDING and len(ran) == 2


def test_the_entry_points_need_no_extension(builder, tmp_path):
    """The package without _torch_binding.so: it imports, its C entry points answer, and an
    operator that needs the extension says so; without torch too."""
    pkg = tmp_path / "static_sparse_attention_b200"
    pkg.mkdir()
    for name in ("__init__.py", "libradattn.so"):
        shutil.copy(os.path.join(PKG, name), pkg / name)
    code = """
import sys
if {hide}:
    sys.modules["torch"] = None
import static_sparse_attention_b200 as ra
assert ra.ra_status_string(ra.RA_OK) == b"ok"
assert ra.ra_cache8_attention_check(None, None, None, None, None, None, 1, 1, 64, 1, 1, 1, 1, None, 1.0, None, None,
                                    0) == ra.RA_ERR_INVALID_ARG
try:
    ra.qk_norm_rope(None)
except ImportError as e:
    assert {hide} or "build.py" in str(e), e
else:
    raise SystemExit("no error")
print("fine")
"""
    for hide in (False, True):
        r = subprocess.run([sys.executable, "-c", code.format(hide=hide)], cwd=tmp_path, capture_output=True, text=True,
                           env=dict(os.environ, PYTHONPATH=str(tmp_path)), timeout=300)
        assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]
