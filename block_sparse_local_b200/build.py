"""Builds libsta.so (release) and libsta_debug.so (device bounds checks,
STA_DEBUG=1) in-tree for sm_100a with nvcc.

    python -m block_sparse_local_b200.build [--verbose]

The library is one translation unit (csrc/sta_lib.cu includes the kernel
headers) compiled with -gencode arch=compute_100a,code=sm_100a.  _kv_torch.so
(csrc/kv_torch.cpp, g++) is the native half of the Python cache calls.
"""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB_PATH = os.path.join(HERE, "libsta.so")
DEBUG_LIB_PATH = os.path.join(HERE, "libsta_debug.so")
KV_TORCH_PATH = os.path.join(HERE, "_kv_torch.so")
KV_TORCH_SOURCE = os.path.join(HERE, "csrc", "kv_torch.cpp")
SOURCES = [os.path.join(HERE, "csrc", "sta_lib.cu")]
DEPENDS = SOURCES + [os.path.join(HERE, "csrc", f) for f in
                     ("device_ptx.cuh", "reorder.cuh", "tile_lists.cuh",
                      "attn_fwd.cuh", "attn_fwd_pair.cuh", "attn_bwd.cuh", "attn_bwd_dq.cuh",
                      "hilbert.cuh", "kv_cache.cuh", "kv_split.cuh", "kv_decode.cuh", "kv_chunk.cuh")] + \
    [os.path.join(ROOT, "include", "sta.h")]


def nvcc_path():
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    p = os.path.join(cuda, "bin", "nvcc")
    return p if os.path.exists(p) else "nvcc"


def command(out=LIB_PATH, extra=()):
    return [nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-O3",
            "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-shared",
            "-I" + os.path.join(ROOT, "include"), *extra, "-o", out, *SOURCES]


def kv_torch_built_for():
    """What _kv_torch.so depends on besides its source: it uses the C++ interface
    of the installed torch and Python, and holds this text."""
    import torch

    return f"built for torch {torch.__version__}, Python {sys.version_info[0]}.{sys.version_info[1]};"


def kv_torch_matches(path=KV_TORCH_PATH):
    """Whether the file was built for the running torch and Python."""
    with open(path, "rb") as f:
        return kv_torch_built_for().encode() in f.read()


def kv_torch_command():
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    inc = [*cpp_extension.include_paths(), sysconfig.get_path("include"),
           os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            f'-DKV_TORCH_BUILT_FOR="{kv_torch_built_for()}"',
            *(x for d in inc for x in ("-isystem", d)), "-o", KV_TORCH_PATH, KV_TORCH_SOURCE,
            "-L" + libs, "-Wl,-rpath," + libs, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
            "-lc10_cuda", "-ldl"]


def up_to_date(path=LIB_PATH, depends=DEPENDS):
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(f) <= t for f in depends)


def build(force=False, verbose=False, debug=True):
    """Builds libsta.so, _kv_torch.so and (debug=True) libsta_debug.so, in parallel."""
    jobs = [(LIB_PATH, ())]
    if debug:
        jobs.append((DEBUG_LIB_PATH, ("-DSTA_DEBUG=1",)))
    procs = []

    def start(path, cmd):
        procs.append((path, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                             stderr=subprocess.PIPE, text=True)))

    for path, defs in jobs:
        if force or not up_to_date(path):
            extra = tuple(defs) + (("-Xptxas", "-v") if verbose else ())
            start(path, command(out=path, extra=extra))
    if force or not up_to_date(KV_TORCH_PATH, [KV_TORCH_SOURCE]) or not kv_torch_matches():
        start(KV_TORCH_PATH, kv_torch_command())
    for path, proc in procs:
        out, err = proc.communicate()
        if verbose or proc.returncode != 0:
            sys.stderr.write(out + err)
        if proc.returncode != 0:
            raise RuntimeError(f"the compiler failed building {os.path.basename(path)}")
    return LIB_PATH


if __name__ == "__main__":
    build(force=True, verbose="--verbose" in sys.argv)
    print(LIB_PATH)
