"""Index arithmetic of the experts' row operators (dg_index.h), run on the host
at the ends of the sizes that the entry points take, under AddressSanitizer and
UndefinedBehaviorSanitizer."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
pytestmark = pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "include", "hip")),
                                reason="needs g++ and the HIP headers")


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("index") / "index_san")
    build = subprocess.run(["g++", "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                            "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
                            os.path.join(ROOT, "tests", "sanitize", "index_driver.cpp"), "-o", exe],
                           capture_output=True, text=True, timeout=600)
    assert build.returncode == 0, build.stderr
    return exe


def run(driver, what):
    r = subprocess.run([driver, what], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1"))
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "ok" in out and "runtime error" not in out, out


def test_shares_of_the_most_rows(driver):
    """A workgroup's share of a layout's rows, where the step past its last row reaches 2^31."""
    run(driver, "for_share")


def test_shares_of_the_most_choices(driver):
    """A workgroup's share of a token's choices, up to as many as a call may have."""
    run(driver, "share_of")


def test_runs_of_the_widest_rows(driver):
    """512-column runs of a row, up to the widest that combine takes."""
    run(driver, "runs_of")
