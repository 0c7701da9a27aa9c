"""The binding without its compiled part (CPU only)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "spmspv_graph_traversal_amd")

CODE = """
import torch
import spmspv_graph_traversal_amd as dbs
assert dbs.dbs_build and dbs.dbs_spmspv and dbs.dbs_bfs and dbs.binding._lib.dbs_q4_product
freq, scale = dbs.dbs_rope_frequencies(8)
x = torch.zeros(1, 1, 8)
for call in (lambda: dbs.dbs_rope(x, x, freq, x), lambda: dbs.dbs_logits_adjust(x, x)):
    try:
        call()
    except ImportError as e:
        assert "_calls.so" in str(e)
    else:
        raise AssertionError
"""


@pytest.mark.parametrize("broken", [False, True])
def test_sparse_products_need_no_compiled_binding(tmp_path, broken):
    """Where only the HIP library was built, or the compiled part for another interpreter, the package loads, and the decode-step
    calls say what is missing."""
    package = tmp_path / "spmspv_graph_traversal_amd"
    package.mkdir()
    for name in ("__init__.py", "binding.py", "build_lib.py", "libdbs.so"):
        os.symlink(os.path.join(PACKAGE, name), package / name)
    if broken:
        (package / "_calls.so").write_bytes(b"not a library")
    r = subprocess.run([sys.executable, "-c", CODE], cwd=tmp_path, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "PYTHONPATH": str(tmp_path), "PYTHONDONTWRITEBYTECODE": "1"})
    assert r.returncode == 0, r.stderr


def test_the_compiler_may_be_named_without_its_folder(tmp_path, monkeypatch):
    from spmspv_graph_traversal_amd import build_lib

    (tmp_path / "bin").mkdir()
    (tmp_path / "include" / "hip").mkdir(parents=True)
    (tmp_path / "include" / "hip" / "hip_runtime.h").write_text("")
    (tmp_path / "bin" / "hipcc").write_text("#!/bin/sh\n")
    (tmp_path / "bin" / "hipcc").chmod(0o755)
    monkeypatch.setattr(build_lib, "HIPCC", str(tmp_path / "bin" / "hipcc"))
    assert build_lib.rocm_include() == str(tmp_path / "include")
    monkeypatch.setattr(build_lib, "HIPCC", "hipcc")
    monkeypatch.setenv("PATH", str(tmp_path / "bin"))
    assert build_lib.rocm_include() == str(tmp_path / "include")
    monkeypatch.setenv("PATH", "")  # a wrapper elsewhere
    monkeypatch.setenv("ROCM_PATH", str(tmp_path))
    assert build_lib.rocm_include() == str(tmp_path / "include")
