"""Build the CUDA library in-tree: csrc/*.cu -> libsgemm_gb300.so (sm_103a only),
and the extension module that marshals torch tensors for fp8.py
(csrc/fp8_torch.cpp -> _fp8_torch.so, host code).

Each translation unit is compiled by nvcc in parallel (one -gencode for
compute capability 10.3a), objects go to ``_build/`` and are relinked only when
a source or header changed.  The CUDA runtime is linked statically, so the
library depends on nothing but the driver at run time.
"""
import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libsgemm_gb300.so")
TORCH_EXT = os.path.join(HERE, "_fp8_torch.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xptxas", "-v",
              "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; set NVCC or put the CUDA toolkit on PATH")
    return cand


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _compile(nvcc, src, obj, log, defines=()):
    cmd = [nvcc, *NVCC_FLAGS, *("-D" + d for d in defines), "-c", src, "-o", obj + ".tmp"]
    proc = subprocess.run(cmd, capture_output=True, text=True)
    with open(log, "w") as f:
        f.write(" ".join(cmd) + "\n" + proc.stdout + proc.stderr)
    if proc.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{proc.stderr[-4000:]}")
    os.replace(obj + ".tmp", obj)
    return obj


def _torch_target(spec) -> str:
    """What the extension module is built for: torch's version (as its version.py has it) and the interpreter."""
    with open(os.path.join(os.path.dirname(spec.origin), "version.py")) as f:
        version = re.search(r"__version__\s*=\s*['\"]([^'\"]+)", f.read())
    return f"torch {version.group(1) if version else '?'}, {sysconfig.get_config_var('SOABI')}"


def _torch_extension(force: bool):
    """Compile csrc/fp8_torch.cpp against the installed torch if it is out of date, or was built for another torch or
    interpreter.  Without torch there is nothing to marshal for.  The module saves time in fp8.py, which also does
    without it: where it cannot be built (no compiler, a torch without CUDA) that is a warning."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    src, log = os.path.join(CSRC, "fp8_torch.cpp"), os.path.join(BUILD, "fp8_torch.log")
    torch_dir, target, stamp = os.path.dirname(spec.origin), _torch_target(spec), os.path.join(BUILD, "fp8_torch.target")
    newest = max([os.path.getmtime(src), *(os.path.getmtime(h) for h in glob.glob(os.path.join(INCLUDE, "*.h")))])
    if not force and os.path.exists(TORCH_EXT) and os.path.getmtime(TORCH_EXT) >= newest and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read() == target:
                return TORCH_EXT
    cuda_include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    tmp = TORCH_EXT + ".tmp.%d" % os.getpid()
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-I", INCLUDE, "-I", os.path.join(torch_dir, "include"),
           "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-isystem", cuda_include, src, "-o", tmp,
           "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    try:
        proc = subprocess.run(cmd, capture_output=True, text=True)
        failed, said = proc.returncode != 0, proc.stdout + proc.stderr
    except OSError as e:
        failed, said = True, str(e)
    with open(log, "w") as f:
        f.write(" ".join(cmd) + "\n" + said)
    if failed:
        if os.path.exists(TORCH_EXT):   # of another torch, or of other entry points
            os.remove(TORCH_EXT)
        warnings.warn(f"the extension module of fp8.py was not built (see {log}); its calls take some 8 us longer:\n"
                      + said[-1000:])
        return None
    os.replace(tmp, TORCH_EXT)
    with open(stamp, "w") as f:
        f.write(target)
    return TORCH_EXT


def build(force: bool = False, jobs: int = None, verbose: bool = False, defines=(),
          out: str = None) -> str:
    """Compile and link if anything is out of date; return the library path.

    ``defines`` (e.g. ``["SG_SIMT_KC_UNROLL=4"]``) select compile-time kernel
    options; a build with defines needs its own ``out`` path and object dir.
    """
    nvcc = _nvcc()
    defines = list(defines)
    if defines and not out:
        raise ValueError("a build with defines needs its own output path")
    lib = out or LIB
    build_dir = BUILD if not out else os.path.join(BUILD, "variant_" + os.path.basename(out).replace(".so", ""))
    os.makedirs(build_dir, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    newest_header = max((os.path.getmtime(h) for h in _headers()), default=0.0)
    todo, objs = [], []
    for src in sources:
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        stale = force or not os.path.exists(obj) or \
            os.path.getmtime(obj) < max(os.path.getmtime(src), newest_header)
        if stale:
            todo.append((src, obj, obj[:-2] + ".log"))
    jobs = jobs or min(len(todo) + 1, os.cpu_count() or 4)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        extension = None if out else ex.submit(_torch_extension, force)
        list(ex.map(lambda t: _compile(nvcc, *t, defines=defines), todo))
    relink = force or bool(todo) or not os.path.exists(lib) or \
        os.path.getmtime(lib) < max(os.path.getmtime(o) for o in objs)
    if relink:
        tmp = lib + ".tmp.%d" % os.getpid()
        cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs, "-ldl", "-lpthread", "-lrt"]
        proc = subprocess.run(cmd, capture_output=True, text=True)
        if proc.returncode != 0:
            raise RuntimeError("link failed:\n" + proc.stderr[-4000:])
        os.replace(tmp, lib)
    if extension is not None:
        extension.result()
    if verbose:
        for _, obj, log in todo:
            sys.stdout.write(open(log).read())
    return lib


def ptxas_report() -> str:
    """The -Xptxas -v lines (registers, spills, shared memory) of the last build."""
    out = []
    for log in sorted(glob.glob(os.path.join(BUILD, "*.log"))):
        out.append(f"== {os.path.basename(log)[:-4]}")
        out += [ln for ln in open(log).read().splitlines()
                if "Compiling entry" in ln or "registers" in ln or "spill" in ln]
    return "\n".join(out)


if __name__ == "__main__":
    import argparse
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", action="store_true")
    ap.add_argument("--define", "-D", action="append", default=[])
    ap.add_argument("--out", default=None)
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.v, defines=a.define, out=a.out))
