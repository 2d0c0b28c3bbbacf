"""Ahead-of-time build of libmpgemm.so for gfx950 with hipcc.

Every source is compiled for gfx950 only, with packed-fp32 instruction
selection disabled (-packed-fp32-ops), then linked into one shared library in
this package directory, next to the Python binding that loads it. The compiled
torch-facing calls (host code only) become a second one beside it, where torch is
there to compile them against; the library needs neither it nor them.
"""
import concurrent.futures as cf
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmpgemm.so")
CALLS = os.path.join(HERE, "_torch_calls.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CXX = os.environ.get("CXX", "g++")
SOURCES = ["api.cpp", "gemm_tile.hip", "w4a16.hip", "quantize.hip", "noalloc.hip", "stream_read.hip", "lowrank.hip",
           "api_mxfp4.cpp", "mxfp4_quantize.hip", "mxfp4_gemm.hip", "newton_schulz.hip"]
TORCH_SOURCE = "torch_calls.cpp"

FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-Wno-unused-command-line-argument",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _torch_flags():
    """Compile and link flags of the torch-facing calls."""
    import torch
    from torch.utils import cpp_extension
    inc = cpp_extension.include_paths() + ["/opt/rocm/include", sysconfig.get_path("include")]
    comp = ["-w"] + [f for i in inc for f in ("-isystem", i)] \
        + [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1"]
    link = ["-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_hip",
            "-ltorch_python", "-L", HERE, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
    return comp, link


def build(verbose: bool = False, jobs: int = 6) -> str:
    objdir = os.path.join(ROOT, "_build", "mpgemm")
    os.makedirs(objdir, exist_ok=True)
    try:
        torch_comp, torch_link = _torch_flags()
    except ImportError as e:   # (the C library needs no torch)
        print(f"{os.path.basename(CALLS)} is not built, torch is not there: {e}", file=sys.stderr)
        torch_comp = None

    def shown(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        return cmd

    def compile_one(src):
        obj = os.path.join(objdir, src + ".o")
        if src == TORCH_SOURCE:   # (host code: no kernels in it)
            cmd = [CXX, "-O2", "-std=c++17", "-fPIC"] + torch_comp + ["-I", os.path.join(ROOT, "include")]
        else:
            cmd = [HIPCC] + FLAGS
        r = subprocess.run(shown(cmd + ["-c", os.path.join(CSRC, src), "-o", obj]), capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"compiling {src} failed:\n{r.stdout}\n{r.stderr}")
        return obj

    def link(cmd, to):
        subprocess.run(shown(cmd), check=True)
        os.replace(to + ".tmp", to)

    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        torch_obj = ex.submit(compile_one, TORCH_SOURCE) if torch_comp is not None else None
        objs = list(ex.map(compile_one, SOURCES))
    link([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", LIB + ".tmp"] + objs, LIB)
    if torch_obj is not None:   # (an error in these is raised once the library is there)
        link([CXX, "-shared", "-o", CALLS + ".tmp", torch_obj.result()] + torch_link, CALLS)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
