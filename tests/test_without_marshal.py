"""The dense operators' compiled marshalling is theirs alone: without it the
rest of the package is built, imported and used."""
import os
import subprocess
import sys

from helpers import ROOT, build_lib


def test_the_rest_imports_and_the_dense_operators_say_so():
    build_lib()
    code = """
import sys
sys.modules["grouped_gemm_top_gb300._marshal"] = None        # its import fails
import torch
from grouped_gemm_top_gb300 import block, layer, ops, optim
assert ops.moe_row_capacity(256, 8, 2) == 1536
x = torch.zeros((4, 64), dtype=torch.bfloat16)
for call in (lambda: ops.linear_fwd(x, x.t().contiguous(), y=x), lambda: ops.rmsnorm_residual_fwd(x, x[0]),
             lambda: ops.gated_ffn_fwd(x, x.t().contiguous(), h=x)):
    try:
        call()
    except ImportError as e:
        assert "_marshal.so" in str(e)
    else:
        raise AssertionError("no error")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_build_without_python_headers_or_a_compiler(tmp_path, monkeypatch, capsys):
    from grouped_gemm_top_gb300 import build
    so = tmp_path / "_marshal.so"

    def left(age, force):
        so.write_bytes(b"built elsewhere")
        if age:
            os.utime(so, (1, 1))
        build._build_marshal(force)
        return os.path.exists(so), capsys.readouterr().err

    monkeypatch.setattr(build, "MARSHAL", str(so))
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda *a: {"include": str(tmp_path)})
    there, said = left(age=True, force=False)                 # older than its source: not left to be loaded
    assert not there and "Python.h" in said
    monkeypatch.setattr(build.shutil, "which", lambda name: None)
    there, said = left(age=True, force=True)
    assert not there and "C compiler" in said
    assert left(age=False, force=False) == (True, "")         # up to date: nothing to do
    there, said = left(age=False, force=True)
    assert there and "C compiler" in said
