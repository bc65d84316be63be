"""Host helpers of the library, compiled by themselves."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_failed_query_is_asked_again(tmp_path):
    """What a kernel's launch asks of it once (its registers): a failure is not kept."""
    if shutil.which("g++") is None:
        pytest.skip("g++ is missing")
    exe = str(tmp_path / "ask_once")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror",
                        "-I", os.path.join(ROOT, "hadamard_rotated_bit_gb300", "csrc"),
                        os.path.join(ROOT, "tests", "c", "ask_once.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert subprocess.run([exe]).returncode == 0
