"""The build script with compilers that are not /opt/rocm/bin/hipcc. No GPU is needed."""
import importlib.util
import os
import shutil
import stat

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
needs_hipcc = pytest.mark.skipif(shutil.which(HIPCC) is None, reason="no hipcc")


def script():
    spec = importlib.util.spec_from_file_location(
        "_build_script", os.path.join(ROOT, "bwd_tbe_pooled_amd", "build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@needs_hipcc
@pytest.mark.parametrize("how", ["as given", "name on PATH", "wrapper elsewhere"])
def test_calls_build_with_any_hipcc(how, tmp_path, monkeypatch):
    m = script()
    real = shutil.which(HIPCC)
    if how == "name on PATH":
        monkeypatch.setenv("PATH", os.path.dirname(real) + os.pathsep + os.environ["PATH"])
        m.HIPCC = os.path.basename(real)
    elif how == "wrapper elsewhere":
        wrapper = tmp_path / "bin" / "hipcc"
        wrapper.parent.mkdir()
        wrapper.write_text(f'#!/bin/sh\nexec "{real}" "$@"\n')
        wrapper.chmod(wrapper.stat().st_mode | stat.S_IXUSR)
        m.HIPCC = str(wrapper)
    assert os.path.exists(os.path.join(m._hip_include(), "hip", "hip_runtime_api.h"))
    if how == "name on PATH":
        m.CALLS = str(tmp_path / "_lmcall.so")
        m._build_calls()
        assert os.path.getsize(m.CALLS) > 0


def test_missing_headers_are_named(tmp_path):
    m = script()
    fake = tmp_path / "hipcc"
    fake.write_text("#!/bin/sh\necho no headers here >&2\nexit 1\n")
    fake.chmod(0o755)
    m.HIPCC = str(fake)
    with pytest.raises(RuntimeError, match="HIP's headers not found(.|\n)*no headers here"):
        m._hip_include()
