"""The package where the language-model operators cannot be loaded: the table calls
need libtbe.so alone. No GPU is needed; each case imports a copy in its own process."""
import os
import shutil
import subprocess
import sys

import pytest

pytest.importorskip("bwd_tbe_pooled_amd", reason="libtbe.so not built")
PACKAGE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bwd_tbe_pooled_amd")

TABLE = """
import bwd_tbe_pooled_amd as tbe
d = tbe.Desc(T=2, D=8, B=4, rows=[10, 20], dtype="f32")
assert tbe.tbe_workspace_bytes(d, 16, False, tbe.TBE_OP_BACKWARD) > 0
"""
REFUSED = TABLE + """
assert "tbe_token_forward" in dir(tbe)
for use in (lambda: tbe.tbe_token_forward, lambda: tbe.TokenDesc, lambda: tbe.distill_workspace):
    try:
        use()
    except ImportError as e:
        assert WHY in str(e), e
    else:
        raise AssertionError("not refused")
"""


def run(tmp_path, code, change=None, **env):
    copy = tmp_path / "bwd_tbe_pooled_amd"
    copy.mkdir()
    for f in ("__init__.py", "lm.py", "libtbe.so", "_lmcall.so"):
        os.symlink(os.path.join(PACKAGE, f), copy / f)
    if change:
        change(copy)
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path), **env})
    assert r.returncode == 0, r.stderr


def test_without_the_compiled_calls(tmp_path):
    run(tmp_path, "WHY = 'build.py'\n" + REFUSED, lambda copy: (copy / "_lmcall.so").unlink())


def test_with_compiled_calls_that_do_not_load(tmp_path):
    def broken(copy):
        (copy / "_lmcall.so").unlink()
        (copy / "_lmcall.so").write_bytes(b"built for something else")
    run(tmp_path, "WHY = 'another Python or torch'\n" + REFUSED, broken)


def test_with_a_library_of_the_tables_alone(tmp_path):
    """TBE_LIBRARY names a library without the language-model entry points."""
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    import bwd_tbe_pooled_amd as tbe
    names = [n for n in tbe.exported_symbols()
             if not n.startswith(("tbe_token_", "tbe_expert_", "tbe_distill_"))]
    source, library = tmp_path / "stub.c", tmp_path / "libstub.so"
    source.write_text("".join(f"long {n}(void) {{ return 1; }}\n" for n in names))
    subprocess.run(["g++", "-x", "c", "-shared", "-fPIC", str(source), "-o", str(library)], check=True)
    run(tmp_path, "WHY = 'no language-model operators'\n" + REFUSED, TBE_LIBRARY=str(library))


def test_names_load_at_first_use(tmp_path):
    run(tmp_path, TABLE + """
import sys
assert "bwd_tbe_pooled_amd.lm" not in sys.modules
from bwd_tbe_pooled_amd import TokenDesc
assert tbe.TokenDesc is TokenDesc and "TokenDesc" in vars(tbe) and "tbe_distill_step" in vars(tbe)
assert not hasattr(tbe, "no_such_name")
""")
