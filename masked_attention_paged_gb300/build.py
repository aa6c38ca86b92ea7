"""Build libattn.so in-tree with nvcc for sm_103a (GB300).

Each .cu under csrc/ is compiled in parallel to an object file, then linked
into ``_build/libattn_<machine>.so``.  No CMake, no torch extension machinery:
the library is a plain C-ABI shared object.  marshal.cpp, which makes the
binding's calls in one step, is a Python module of its own beside it (g++, torch's
headers); the binding works without it, at a higher cost per call.
"""
from __future__ import annotations

import os
import platform
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB_NAME = f"libattn_{platform.machine()}.so"
LIB_PATH = os.path.join(BUILD, LIB_NAME)

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
    "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC,
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (CUDA toolkit required to build libattn)")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    deps = [src] + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    deps.append(os.path.join(INCLUDE, "libattn.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def marshal_path() -> str:
    """The binding's compiled module, per machine, version of torch and ABI of the
    interpreter: it is compiled against Python's object layouts, which nothing
    checks when it is loaded."""
    import torch
    abi = sysconfig.get_config_var("SOABI") or sys.implementation.cache_tag
    return os.path.join(BUILD, f"_marshal_{platform.machine()}_{torch.__version__.replace('+', '_')}_{abi}.so")


def _marshal_command(out: str) -> list[str]:
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [INCLUDE, os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
           os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"]]
    return ["g++", "-O1", "-std=c++17", "-fPIC", "-shared", *[x for p in inc for x in ("-I", p)],
            os.path.join(CSRC, "marshal.cpp"), "-o", out, "-L", os.path.join(root, "lib"), "-ltorch_python",
            "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{os.path.join(root, 'lib')}"]


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    exe = nvcc()
    flags = NVCC_FLAGS + list(extra_flags or [])
    objs = []
    jobs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + f".{platform.machine()}.o")
        objs.append(obj)
        if force or _stale(obj, src):
            jobs.append([exe, *flags, "-c", src, "-o", obj])

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr, file=sys.stderr)
        return r

    marshal = marshal_path()
    if force or _stale(marshal, os.path.join(CSRC, "marshal.cpp")):
        tmp = marshal + f".tmp{os.getpid()}"

        def build_marshal(cmd=_marshal_command(tmp)):
            try:
                run(cmd)
                os.replace(tmp, marshal)
            except (RuntimeError, OSError) as e:
                if os.path.exists(marshal):  # of other declarations
                    os.remove(marshal)
                print(f"marshal.cpp was not built, calls take longer on the host: {e}", file=sys.stderr)

        jobs.append(build_marshal)
    cu_jobs = any(not callable(j) for j in jobs)
    if jobs:
        with ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            list(ex.map(lambda j: j() if callable(j) else run(j), jobs))
    if force or cu_jobs or not os.path.exists(LIB_PATH):
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        run([exe, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
