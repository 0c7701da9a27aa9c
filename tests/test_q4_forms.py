"""The calls of q4_forms.py reach every kernel that any call of the 4-bit products does (CPU only: the library's own choice,
compiled for the host)."""
import os
import shutil
import subprocess

import pytest

from q4_forms import CALLS, SCALES

HERE = os.path.dirname(os.path.abspath(__file__))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.mark.skipif(not os.path.exists(HIPCC) and shutil.which("hipcc") is None, reason="hipcc not found")
def test_every_kernel_and_every_kind_of_round_is_reached(tmp_path):
    exe = str(tmp_path / "q4_forms")
    hipcc = HIPCC if os.path.exists(HIPCC) else shutil.which("hipcc")
    r = subprocess.run([hipcc, "--offload-host-only", "-x", "hip", "-std=c++17", "-O2", os.path.join(HERE, "host_checks", "q4_forms.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lines = [f"{x} {int(gated)} 0 {1 if scales == 'bf16' else 2} {128 // group} {m} {n} {tokens}"
             for x, gated, m, tokens, columns in CALLS for n in columns for scales, group in SCALES]
    ours = subprocess.run([exe], input="\n".join(lines), capture_output=True, text=True, timeout=60).stdout.split("\n")
    every = subprocess.run([exe, "all"], capture_output=True, text=True, timeout=60).stdout.split("\n")
    assert len(every) > 200 and not any("none" in f for f in every)
    assert set(every) - {""} == set(ours) - {""}
