"""The C++ way of the MXFP4 binding (_native.so) is an accelerator: the package
works without it, and its status is the call's."""
import importlib.util
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


# ---- a call that the library refuses -------------------------------------------------------

class Refuses:
    """Takes the place of the C++ way: every call is made and fails."""
    calls = 0

    def quantize(self, *a):
        self.calls += 1
        return self.status

    dequantize = gemm = quantize


@pytest.mark.parametrize("status,error", [(B.BA_ERR_HIP, ba.BiasActError), (B.BA_ERR_INVALID, ValueError),
                                          (B.BA_ERR_UNSUPPORTED, ValueError)])
@pytest.mark.parametrize("name,nargs", [("mxfp4_quantize", 3), ("mxfp4_dequantize", 3), ("gemm_mxfp4_bias_act", 6),
                                        ("gemm_mxfp4_bias_add_act", 7)])
def test_a_failed_call_is_not_made_again(monkeypatch, name, nargs, status, error):
    n = Refuses()
    n.status = status
    monkeypatch.setattr(B, "_native", n)
    with pytest.raises(error, match=name + ": ") as e:
        getattr(ba, name)(*[object()] * nargs)           # the Python checks, which come before a second call, would trip
    assert n.calls == 1
    if error is ba.BiasActError:
        assert e.value.status == status


# ---- the build where the module cannot be had ----------------------------------------------

@pytest.fixture
def build(monkeypatch, tmp_path):
    """build.py with an output folder of its own, a stale _native.so in it, and compiler calls that only write
    their output."""
    spec = importlib.util.spec_from_file_location("biasact_build_under_test", os.path.join(PKG, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    for name, at in (("BUILD", "objects"), ("LIB", "lib.so"), ("NATIVE", "_native.so")):
        monkeypatch.setattr(b, name, str(tmp_path / at))
    (tmp_path / "_native.so").write_text("stale")

    def run(cmd):
        if any(c.endswith("native_call.cpp") for c in cmd) and b.native_fails:
            raise RuntimeError("build step failed: Python.h: No such file or directory")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return 0.0, ""

    b.native_fails = False
    monkeypatch.setattr(b, "_run", run)
    return b


def test_build_with_the_module(build):
    with open(build.build()) as lib, open(build.NATIVE) as native:
        assert lib.read() == native.read() == "built"


@pytest.mark.parametrize("why", ["its compiler call fails", "torch is not for HIP", "no torch"])
def test_build_without_the_module(build, monkeypatch, capsys, why):
    if why == "its compiler call fails":
        build.native_fails = True
    elif why == "no torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    else:
        monkeypatch.setattr(torch.version, "hip", None)
    with open(build.build()) as lib:
        assert lib.read() == "built"
    assert not os.path.exists(build.NATIVE)              # the stale one is gone
    assert "_native.so is not built" in capsys.readouterr().out


def test_build_still_fails_for_the_library(build, monkeypatch):
    def run(cmd):
        if any(c.endswith("plan_mx.cpp") for c in cmd):
            raise RuntimeError("build step failed")
        return 0.0, ""
    monkeypatch.setattr(build, "_run", run)
    with pytest.raises(RuntimeError):
        build.build()
