"""Build libfgb.so (the HIP kernels and their C ABI) for gfx950, in-tree.

Every .hip file under csrc/ is compiled with hipcc to an object, then linked
into fine_grained_blockwise_amd/libfgb.so.  Packed-FP32 VALU ops are disabled
and floating-point contraction is off, so every fp32 operation rounds where
the source says it does.  Beside it _tensors, the binding's extension module for
lists of tensors, is compiled against the installed torch and Python, whose
versions it carries (host code only).
"""
import concurrent.futures as cf
import glob
import importlib.util
import os
import runpy
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfgb.so")
TENSORS = os.path.join(HERE, "_tensors" + sysconfig.get_config_var("EXT_SUFFIX"))  # (another Python does not see it)
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

CFLAGS = [
    "-std=c++17", "-O3", "-fPIC", f"--offload-arch={ARCH}", "-ffp-contract=off",
    "-fno-gpu-rdc", "-Wall", "-Wno-unused-function",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(os.path.dirname(HERE), "include"),
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


def _compile(src):
    obj = os.path.join(BUILD, os.path.basename(src)[:-4] + ".o")
    cmd = [HIPCC] + CFLAGS + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj, r.stderr


def _build_tensors():
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    version = runpy.run_path(os.path.join(torch, "version.py"))["__version__"]
    tmp = TENSORS + ".tmp"
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", f'-DFGB_TORCH="{version}"', "-I", os.path.join(torch, "include"),
           "-I", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], os.path.join(CSRC, "tensor_list.cpp"),
           "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for tensor_list.cpp:\n{r.stderr}")
    os.replace(tmp, TENSORS)


def build(jobs=8, verbose=False):
    """Compile every HIP source and link libfgb.so, and _tensors; returns the library path."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(jobs, len(srcs) + 1)) as ex:
        tensors = ex.submit(_build_tensors)
        results = list(ex.map(_compile, srcs))
        tensors.result()
    if verbose:
        for obj, err in results:
            if err.strip():
                print(err)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp"
    subprocess.run([HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}", "-o", tmp] + objs,
                   check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
