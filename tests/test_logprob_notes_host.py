"""The notes of the token log probabilities' forward on the CPU: their room is
never left and no alternative is lost, on rows of infinities among others."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_notes(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "notes")
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wno-unknown-pragmas", "-I",
                    os.path.join(ROOT, "selective_state_space_81_amd", "csrc"),
                    os.path.join(ROOT, "tests", "logprob_notes_host.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
