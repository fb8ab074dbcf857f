"""AddressSanitizer + UndefinedBehaviorSanitizer build of the argument
validation of the layer norm and the experts' row operators (moe_api.cpp, CPU
only): every integer argument over its extremes, against launcher stand-ins that
check what reaches them."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "include", "hip")),
                    reason="needs g++ and the HIP headers")
def test_moe_validation_under_sanitizers(tmp_path):
    exe = str(tmp_path / "moe_san")
    build = subprocess.run(["g++", "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                            "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
                            os.path.join(ROOT, "tests", "sanitize", "moe_driver.cpp"),
                            os.path.join(ROOT, "moe_grouped_gemm_scaled_amd", "csrc", "moe_api.cpp"),
                            "-L", os.path.join(ROCM, "lib"), "-lamdhip64", "-Wl,-rpath," + os.path.join(ROCM, "lib"), "-o", exe],
                           capture_output=True, text=True, timeout=600)
    assert build.returncode == 0, build.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1", HIP_VISIBLE_DEVICES="")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "ok" in out and "runtime error" not in out, out
