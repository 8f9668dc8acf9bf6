"""Builds the CUDA library of the indexer for sm_100a (nvcc; no GPU needed).

    python -m sparse_attention_token_02_b200.build [--jobs N] [--verbose]

Compiles every ``csrc/*.cu`` to an object with
``-gencode arch=compute_100a,code=sm_100a -lineinfo -O3`` and links them into
``libdsa_indexer.so`` next to this file (static CUDA runtime, so loading the
library needs only the driver; only the ``dsa_*`` C symbols are exported).
``csrc/layer_calls.cpp`` becomes the module ``_layer_calls``, the torch side of the
layer's calls (g++, torch's headers), for this Python and this torch; the package does
without it where it cannot be built.  Objects are rebuilt when a source or header is
newer, the module also when its command (torch's version and place are in it) changes.
"""

from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libdsa_indexer.so")
CALLS = os.path.join(PKG, "_layer_calls" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
CALLS_COMMAND = os.path.join(BUILD, "layer_calls.command")   # what CALLS was built with

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
          "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _headers() -> list[str]:
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch() -> tuple[str, str] | None:
    """Where torch is and its version, without importing it."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    place = spec.submodule_search_locations[0]
    if not os.path.exists(os.path.join(place, "version.py")):
        return None
    with open(os.path.join(place, "version.py")) as f:
        version = re.search(r"^__version__ = ['\"](.+?)['\"]", f.read(), re.M)
    return (place, version.group(1)) if version else None


def _calls_command(src: str) -> list[str] | None:
    """None where torch or Python's headers are not there."""
    found, python = _torch(), sysconfig.get_paths()["include"]
    if found is None or not os.path.exists(os.path.join(python, "Python.h")):
        return None
    torch, version = found
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    dirs = [INCLUDE, os.path.join(torch, "include"), os.path.join(torch, "include/torch/csrc/api/include"),
            os.path.join(cuda, "include"), python]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", f'-DTORCH_BUILT_FOR="{version}"',
            *(f"-I{d}" for d in dirs), src, "-o", CALLS,
            "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]


def _build_calls(run) -> None:
    """The compiled calls, where they can be had: a module that no longer fits is taken away before it is built anew."""
    src = os.path.join(CSRC, "layer_calls.cpp")
    command = _calls_command(src)
    wanted = " ".join(command or [])
    if os.path.exists(CALLS_COMMAND) and not _stale(CALLS, [src] + _headers()):
        with open(CALLS_COMMAND) as f:
            if f.read() == wanted:
                return
    for old in (CALLS, CALLS_COMMAND):
        if os.path.exists(old):
            os.remove(old)
    if command is None:
        return
    try:
        run(command)
    except (RuntimeError, OSError) as e:                     # no g++, a torch without CUDA, ...
        print(f"the layer's compiled calls could not be built, its Python forms serve instead: {e}", file=sys.stderr)
        return
    with open(CALLS_COMMAND, "w") as f:
        f.write(wanted)


def build(jobs: int = 8, verbose: bool = False, extra: list[str] | None = None, out_dir: str | None = None) -> str:
    """Build the library; `extra` nvcc flags and `out_dir` (objects and .so) serve tuning builds."""
    build_dir = os.path.join(out_dir, "_build") if out_dir else BUILD
    lib_path = os.path.join(out_dir, "libdsa_indexer.so") if out_dir else LIB
    os.makedirs(build_dir, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = _headers()
    cmds = []
    objs = []
    for src in sources:
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if _stale(obj, [src] + headers):
            cmds.append([nvcc(), *ARCH, *CFLAGS, *(extra or []), "-c", src, "-o", obj])

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr, flush=True)

    with cf.ThreadPoolExecutor(max_workers=max(1, jobs)) as ex:
        calls = None if out_dir else ex.submit(_build_calls, run)
        list(ex.map(run, cmds))
        if calls is not None:
            calls.result()
    if cmds or _stale(lib_path, objs):
        run([nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", lib_path, *objs])
    return lib_path


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--jobs", type=int, default=8)
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers / shared memory per kernel")
    a = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if a.ptxas_info else None
    if extra:
        for f in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(f)
    print(build(a.jobs, a.verbose or a.ptxas_info, extra))
    return 0


if __name__ == "__main__":
    sys.exit(main())
