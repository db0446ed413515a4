"""Builds libpd.so (the C-ABI library) in-tree for sm_103a with nvcc, and the
Python binding's extension module with g++.

Each .cu translation unit is compiled in parallel, then linked into
``decode_ragged_paged_gb300/libpd.so``; ``csrc/pd_bind.cpp`` becomes the
package's extension module ``_pd_bind``, named and stamped with the Python and
the torch that it was compiled against. Re-running is cheap: objects newer than
their sources and headers are reused.

    python -m decode_ragged_paged_gb300.build [--force] [--verbose-ptxas] [--no-bind]

--no-bind leaves the module out (for programs that call libpd.so from C: it takes
nvcc alone, and neither Python's nor torch's headers).
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpd.so")
BIND = os.path.join(HERE, "_pd_bind" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpd.so")


def _deps() -> list[str]:
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(ROOT, "include", "pd.h")]


def _stale(target: str, sources: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in sources)


def _compile(src: str, verbose_ptxas: bool) -> tuple[str, str]:
    obj = os.path.join(OBJ, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
    return obj, r.stderr


def _host_stamp() -> str:
    import platform
    return f"{platform.machine()} {nvcc()}"


def _bind() -> None:
    """Compiles the binding module (csrc/pd_bind.cpp) with g++ against torch's headers."""
    import torch
    home = os.path.dirname(torch.__file__)
    tmp = BIND + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DPD_TORCH="{torch.__version__}"',
           "-isystem", os.path.join(home, "include"),
           "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "pd_bind.cpp"), "-o", tmp,
           "-L", os.path.join(home, "lib"), f"-Wl,-rpath,{os.path.join(home, 'lib')}", "-ltorch_python", "-ltorch_cpu",
           "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on pd_bind.cpp:\n{r.stderr}")
    os.replace(tmp, BIND)
    plain = os.path.join(HERE, "_pd_bind.so")  # (an untagged module, which any Python would load)
    if os.path.exists(plain):
        os.remove(plain)
    with open(BIND_STAMP, "w") as f:
        f.write(_bind_stamp())


BIND_STAMP = os.path.join(OBJ, "bind.txt")


def _bind_stamp() -> str:
    """What the module's code takes for granted: it reads torch's and Python's objects in place."""
    import torch
    return f"{torch.__version__} {int(torch._C._GLIBCXX_USE_CXX11_ABI)} {sysconfig.get_config_var('SOABI')}"


def _bind_stale() -> bool:
    if not os.path.exists(BIND_STAMP) or open(BIND_STAMP).read() != _bind_stamp():
        return True
    return _stale(BIND, [os.path.join(CSRC, "pd_bind.cpp"), *_deps()])


def build(force: bool = False, verbose_ptxas: bool = False, jobs: int | None = None, bind: bool = True) -> str:
    """Compile every kernel and the C ABI into libpd.so, and (`bind`) the binding module; returns the library's path."""
    os.makedirs(OBJ, exist_ok=True)
    stamp = os.path.join(OBJ, "host.txt")
    # objects and the library built on another host (another CPU architecture) are never reused
    if not os.path.exists(stamp) or open(stamp).read() != _host_stamp() or not os.path.exists(LIB):
        force = True
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = _deps()
    todo = [s for s in sources
            if force or verbose_ptxas or _stale(os.path.join(OBJ, os.path.basename(s) + ".o"), [s, *deps])]
    bind = bind and (force or _bind_stale())
    logs = []
    if todo or bind:
        with cf.ThreadPoolExecutor(max_workers=jobs or min(len(todo) + 1, os.cpu_count() or 4)) as ex:
            if bind:
                bound = ex.submit(_bind)
            for obj, log in ex.map(lambda s: _compile(s, verbose_ptxas), todo):
                logs.append(log)
    objs = [os.path.join(OBJ, os.path.basename(s) + ".o") for s in sources]
    if force or todo or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, LIB)
    with open(stamp, "w") as f:
        f.write(_host_stamp())
    if bind:
        bound.result()  # after the library, which does not need it
    if verbose_ptxas:
        sys.stderr.write("".join(logs))
    return LIB


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    ap.add_argument("--no-bind", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose_ptxas=a.verbose_ptxas, bind=not a.no_bind))


if __name__ == "__main__":
    main()
