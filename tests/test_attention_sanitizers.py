"""The attention-block entry points' validation under the address and
undefined-behaviour sanitizers (host code only; launchers and the device
check are stand-ins)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "int4_w4a4_quantized_amd", "csrc")


def test_attention_validation_under_sanitizers(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    exe = tmp_path / "attention_driver"
    subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I",
                    os.path.join(ROOT, "include"), "-I", CSRC, "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-g", "-O1", os.path.join(CSRC, "attention_api.cpp"),
                    os.path.join(ROOT, "tests", "sanitize", "attention_driver.cpp"), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, UBSAN_OPTIONS="print_stacktrace=1"))
    assert r.returncode == 0, r.stdout + r.stderr
    assert "0 failures" in r.stdout and "runtime error" not in r.stderr


def test_line_of_steps_under_sanitizers(tmp_path):
    """The arithmetic that sizes the workspace against the one that cuts tiles, for starts in order and not."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    exe = tmp_path / "attention_line_driver"
    subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I",
                    os.path.join(ROOT, "include"), "-I", CSRC, "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-g", "-O1",
                    os.path.join(ROOT, "tests", "sanitize", "attention_line_driver.cpp"), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, UBSAN_OPTIONS="print_stacktrace=1"))
    assert r.returncode == 0, r.stdout + r.stderr
    assert " 0 failures" in r.stdout and "runtime error" not in r.stderr
