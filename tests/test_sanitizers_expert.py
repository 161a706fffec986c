"""CPU: the experts' host-side rules under address and undefined-behaviour
sanitizers, over half a million random problems and layers (no GPU)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_expert_checks_under_sanitizers(tmp_path):
    exe = str(tmp_path / "expert_checks_fuzz")
    csrc = os.path.join(ROOT, "combine_topk_ids_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-fno-omit-frame-pointer", "-g", "-O1", "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(csrc, "host_checks.cpp"),
                    os.path.join(ROOT, "tests", "sanitize", "expert_checks_fuzz.cpp"), "-o", exe], check=True)
    res = subprocess.run([exe, "500000"], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "runtime error" not in res.stderr and "AddressSanitizer" not in res.stderr
    assert "no failures" in res.stdout
