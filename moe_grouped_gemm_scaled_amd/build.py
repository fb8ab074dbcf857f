"""Build libdg.so (the HIP library) in-tree with hipcc for gfx950.

    python -m moe_grouped_gemm_scaled_amd.build

Every source is compiled ahead of time (no JIT); the object files go to
_build/ next to this file and the shared library to libdg.so beside it, with
_args.so, the native argument checks of the Python binding.  libdg.so needs
hipcc alone; _args.so needs g++ and torch's headers, and where it cannot be
built the binding makes the same checks in Python (some 350 ns a tensor
instead of 30): a warning says so.
"""
import os
import subprocess
import sys
import time

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libdg.so")
ARGS = os.path.join(HERE, "_args.so")     # the binding's argument checks, a Python extension module
SOURCES = ["api.cpp", "quant.hip", "gemm.hip", "decode.hip", "pipelined.hip", "persistent.hip", "mqa.hip", "noalloc.hip", "stream.hip",
           "layer_api.cpp", "norm.hip", "gated.hip", "gated_small.hip", "gated_bwd.hip"]
ARCH = "gfx950"

# -packed-fp32-ops: no v_pk_{add,mul,fma}_f32 from the compiler.
COMMON = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-Wall", "-Wno-unused-function",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-I", os.path.join(HERE, "..", "include")]


def _hipcc():
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    path = os.path.join(rocm, "bin", "hipcc")
    return path if os.path.exists(path) else "hipcc"


def _args_command():
    """Compiles the binding's argument checks (csrc/py_args.cpp, host code against torch's headers)."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = cpp_extension.include_paths() + [sysconfig.get_paths()["include"]]
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
            + [a for i in inc for a in ("-isystem", i)]
            + [os.path.join(CSRC, "py_args.cpp"), "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10",
               "-Wl,-rpath," + lib, "-o", ARGS + ".tmp"])


def _start_args():
    """The running compilation, or what kept it from starting."""
    try:
        return subprocess.Popen(_args_command(), stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    except (ImportError, OSError) as e:
        return e


def _finish_args(proc):
    why = proc
    if isinstance(proc, subprocess.Popen):
        out, _ = proc.communicate()
        if proc.returncode == 0:
            os.replace(ARGS + ".tmp", ARGS)
            return
        why = out.decode(errors="replace")
    if os.path.exists(ARGS):                  # of an older source
        os.remove(ARGS)
    print(f"{why}\n{os.path.basename(ARGS)} was not built: the binding checks arguments in Python", file=sys.stderr)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hipcc = _hipcc()
    procs = []
    objs = []
    t0 = time.time()
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        if not os.path.exists(path):
            continue
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        objs.append(obj)
        lang = ["-x", "hip"] if src.endswith(".hip") else []
        cmd = [hipcc] + COMMON + lang + ["-c", path, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    args = _start_args()
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        # hipcc's host pass does not know the packed-fp32 feature: harmless noise
        text = "\n".join(l for l in text.splitlines() if "packed-fp32-ops" not in l and
                         "is not a recognized feature for this target" not in l)
        if p.returncode != 0:
            failed.append(src)
            print(text, file=sys.stderr)
        elif verbose and text.strip():
            print(text, file=sys.stderr)
    if failed:
        raise RuntimeError(f"hipcc failed for {failed}")
    tmp = LIB + ".tmp"
    cmd = [hipcc, "-shared", "-fPIC", f"--offload-arch={ARCH}"] + objs + ["-o", tmp]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    _finish_args(args)
    if verbose:
        print(f"built {LIB} in {time.time() - t0:.1f}s", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build(verbose="-q" not in sys.argv)
