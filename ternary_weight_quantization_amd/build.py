"""Build libbitnet.so (gfx950) in-tree with hipcc, and the torch autograd
functions over it.

    python -m ternary_weight_quantization_amd.build

Compiles every ``csrc/*.hip`` for gfx950 only, links one shared library next
to this file, and prints its path. Packed-FP32 instruction selection is
disabled for all device code. ``csrc/host/torch_ops.cpp`` (host code only, no
kernels) becomes the Python extension ``_bitnet_ops.so`` in the same place,
linked to it and to torch.
"""

import concurrent.futures
import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libbitnet.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
BUILD_DIR = os.path.join(ROOT, "_build")
OPS_SRC = os.path.join(CSRC, "host", "torch_ops.cpp")
OPS_PATH = os.path.join(HERE, "_bitnet_ops.so")
ARCH = "gfx950"

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
COMMON_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    "-Wno-unused-function",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    f"-I{INCLUDE}",
    f"-I{CSRC}",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


def _compile(src, extra):
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [HIPCC, *COMMON_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")


def _compile_ops():
    """The object of torch_ops.cpp, by the host compiler against torch's
    headers."""
    import torch
    from torch.utils import cpp_extension

    obj = os.path.join(BUILD_DIR, "torch_ops.cpp.o")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__",
          "-DUSE_ROCM", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *[f for p in cpp_extension.include_paths() for f in ("-isystem", p)], "-isystem", f"{rocm}/include",
          "-isystem", sysconfig.get_paths()["include"], f"-I{INCLUDE}", "-c", OPS_SRC, "-o", obj],
         f"compiling {OPS_SRC}")
    return obj


def _link_ops(obj):
    """Linked to libbitnet.so beside it; torch's libraries are the loaded
    process's own."""
    from torch.utils import cpp_extension

    tmp = OPS_PATH + ".tmp"
    _run([os.environ.get("CXX", "g++"), "-shared", "-fPIC", obj, "-o", tmp, f"-L{HERE}", f"-l:{LIB_NAME}",
          *[f"-L{p}" for p in cpp_extension.library_paths()], "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python",
          "-Wl,-rpath,$ORIGIN"], "linking the torch functions")
    os.replace(tmp, OPS_PATH)


def build(verbose=False, extra_flags=()):
    """Compile all sources and link LIB_PATH and OPS_PATH. Always rebuilds."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        ops = ex.submit(_compile_ops)
        objs = list(ex.map(lambda s: _compile(s, list(extra_flags)), srcs))
        ops_obj = ops.result()
    tmp = LIB_PATH + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp,
           "-Wl,-rpath,/opt/rocm/lib"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    _link_ops(ops_obj)
    if verbose:
        print(LIB_PATH)
        print(OPS_PATH)
    return LIB_PATH


if __name__ == "__main__":
    build(verbose=True, extra_flags=sys.argv[1:])
