"""The 8-bit operators' host code (argument checks, workspace layouts, the choice of kernel and
its grid: csrc/api_fp8.hip, csrc/schedule.hip) built for the CPU with AddressSanitizer and
UndefinedBehaviorSanitizer against stub launchers that touch every byte of every extent they
are handed (tests/abi_fp8_sanitize_driver.cpp). A planted overflow must be reported."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "token_routing_grouped_amd", "csrc")


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("abi_fp8") / "abi_fp8_sanitize")
    subprocess.run([gxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-fno-omit-frame-pointer", "-Wall", "-Wno-unused-function", "-I",
                    os.path.join(ROOT, "tests", "abi_stub"), "-I", os.path.join(ROOT, "include"), "-x", "c++",
                    os.path.join(CSRC, "api_fp8.hip"), os.path.join(CSRC, "schedule.hip"), "-x", "none",
                    os.path.join(ROOT, "tests", "abi_fp8_sanitize_driver.cpp"), "-o", exe], check=True)
    return exe


def run(driver, *args):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    return subprocess.run([driver, *args], capture_output=True, text=True, timeout=120, env=env)


def test_host_code_under_sanitizers(driver):
    r = run(driver)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "abi ok" in r.stdout and "runtime error" not in r.stderr


def test_planted_overflow_is_caught(driver):
    r = run(driver, "plant")
    assert r.returncode != 0
    assert "AddressSanitizer: heap-buffer-overflow" in r.stderr
