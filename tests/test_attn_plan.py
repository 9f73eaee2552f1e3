"""Attention's launch plan, checked on the host over random batches."""
import os
import shutil
import subprocess

import pytest

from block_quantized_int8_q8_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(not shutil.which("g++"), reason="needs g++")
def test_the_plan_holds_whatever_the_device_finds(tmp_path):
    exe = str(tmp_path / "check")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", build.CSRC,
                    "-I", os.path.join(build.ROOT, "include"), os.path.join(HERE, "attn_plan_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout + r.stderr
