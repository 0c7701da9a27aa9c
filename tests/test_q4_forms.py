"""The calls of q4_forms.py reach every kernel that any call of the 4-bit products does (CPU only: the library's own choice,
compiled for the host)."""
import os
import shutil
import subprocess

import pytest

from q4_forms import CALLS, SCALES

HERE = os.path.dirname(os.path.abspath(__file__))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.fixture(scope="module")
def forms(tmp_path_factory):
    """What tests/host_checks/q4_forms.cpp answers."""
    if not os.path.exists(HIPCC) and shutil.which("hipcc") is None:
        pytest.skip("hipcc not found")
    exe = str(tmp_path_factory.mktemp("q4") / "q4_forms")
    hipcc = HIPCC if os.path.exists(HIPCC) else shutil.which("hipcc")
    r = subprocess.run([hipcc, "--offload-host-only", "-x", "hip", "-std=c++17", "-O2", os.path.join(HERE, "host_checks", "q4_forms.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return lambda *args, lines=(): subprocess.run([exe, *args], input="\n".join(lines), capture_output=True, text=True,
                                                  timeout=60).stdout.split("\n")[:-1]


def test_every_kernel_and_every_kind_of_round_is_reached(forms):
    lines = [f"{x} {int(gated)} 0 {1 if scales == 'bf16' else 2} {128 // group} {m} {n} {tokens}"
             for x, gated, m, tokens, columns in CALLS for n in columns for scales, group in SCALES]
    every = forms("all")
    assert len(every) > 200 and not any("none" in f for f in every)
    assert set(every) == set(forms(lines=lines))


def test_rows_that_a_mask_reads_together(forms):
    """As dbs.h says: 16 for up to four tokens, 16 to 128 for more."""
    def rows(tokens, m):
        found = forms(lines=[f"{x} 0 1 1 1 {m} {n} {tokens}" for x in ("bf16", "f32") for n in (300, 4096)])
        return {16 * int(f.split(" r=")[1].split()[0]) * int(f.split(" rw=")[1].split()[0]) for f in found}

    for m in (1, 1000, 5000, 8300, 20000, 65536, 1 << 24):
        assert all(rows(t, m) == {16} for t in (1, 4))
        assert all(rows(t, m) <= {16, 32, 64, 128} for t in (5, 8, 16, 64))
    assert rows(5, 4000) == {16} and rows(64, 65536) == {64, 128}
