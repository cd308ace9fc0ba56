"""The C++ way of the MXFP4 binding (_native.so) is an accelerator: the package
works without it, and its status is the call's."""
import os
import shutil
import subprocess
import sys

import pytest

ba = pytest.importorskip("conv_bias_activation_amd")
torch = pytest.importorskip("torch")
B = ba._binding
PKG = os.path.dirname(os.path.abspath(ba.__file__))


# ---- a module that does not load ---------------------------------------------------------

def test_no_module(monkeypatch, tmp_path):
    monkeypatch.setattr(B, "_HERE", str(tmp_path))
    assert B._load_native() is None


@pytest.mark.parametrize("what", ["not a library", "another library"])
def test_a_module_that_does_not_load(monkeypatch, tmp_path, what):
    if what == "not a library":
        (tmp_path / "_native.so").write_bytes(b"not a library")
    else:                                                # no module in it, as with symbols of another torch missing
        src = tmp_path / "empty.c"
        src.write_text("int nothing_here;\n")
        subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(tmp_path / "_native.so")], check=True)
    monkeypatch.setattr(B, "_HERE", str(tmp_path))
    with pytest.warns(RuntimeWarning, match="ctypes"):
        assert B._load_native() is None


def test_the_package_imports_beside_such_a_module(tmp_path):
    pkg = tmp_path / "conv_bias_activation_amd"
    pkg.mkdir()
    for f in ("__init__.py", "_binding.py"):
        shutil.copy(os.path.join(PKG, f), pkg)
    os.symlink(os.path.join(PKG, "libbiasact.so"), pkg / "libbiasact.so")
    (pkg / "_native.so").write_bytes(b"not a library")
    r = subprocess.run([sys.executable, "-W", "ignore", "-c",
                        "import conv_bias_activation_amd as ba; print(ba.mxfp4_shapes(3, 130), ba._binding._native)"],
                       cwd=tmp_path, capture_output=True, text=True, env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == "((3, 128), (3, 8)) None".split()
