"""Build libfftconv_b200.so in-tree with nvcc for sm_100a.

``python -m fft_long_convolution_causal_b200.build`` (or build()) compiles
every .cu file under csrc/ into one shared library next to this file.  The
library is rebuilt when any source or header is newer than it or when it was
built by other commands or another nvcc, from the objects of which neither the
commands nor the source and included files have changed.  A file <output>.key
beside the library and each object says what built it.
"""
import functools
import glob
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libfftconv_b200.so")
BUILD_DIR = os.path.join(ROOT, "_build")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]
LINK = ["-lcudart_static", "-lrt", "-lpthread", "-ldl"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


@functools.lru_cache(maxsize=None)
def _version(nvcc: str) -> str:
    try:
        return subprocess.run([nvcc, "--version"], capture_output=True, text=True).stdout
    except OSError:
        return ""


def _key() -> str:
    """What the objects and the library depend on beside their sources; wherever the tree is."""
    return "\n".join([NVCC, *ARCH, *FLAGS, *LINK]).replace(ROOT, ".") + "\n" + _version(NVCC)


def _built_alike(output: str) -> bool:
    try:
        with open(output + ".key") as f:
            return f.read() == _key()
    except OSError:
        return False


def _say_built(output: str):
    with open(output + ".key", "w") as f:
        f.write(_key())


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not (_built_alike(LIB) or not _version(NVCC)):  # without a compiler: by the times alone
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _deps())


def _fresh(obj) -> bool:
    """The object was compiled alike and is newer than every file its compilation read."""
    try:
        t = os.path.getmtime(obj)
        with open(obj + ".d") as f:
            deps = f.read().split(":", 1)[1].replace("\\\n", " ").split()
        return _built_alike(obj) and bool(deps) and all(os.path.getmtime(f) <= t for f in deps)
    except (OSError, IndexError):
        return False


def _compile(src, verbose, force=True):
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    if not force and not verbose and _fresh(obj):
        return obj, ""
    if os.path.exists(obj + ".key"):  # a compilation that is cut short leaves no key
        os.remove(obj + ".key")
    cmd = [NVCC, *ARCH, *FLAGS, "-MD", "-MF", obj + ".d", "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    _say_built(obj)
    return obj, r.stderr


def build(force: bool = False, verbose: bool = False, jobs: int = 0) -> str:
    """Compile the CUDA library for sm_100a; returns the library path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = _sources()
    jobs = jobs or min(len(srcs), os.cpu_count() or 1)
    with ThreadPoolExecutor(max_workers=jobs) as ex:
        results = list(ex.map(lambda s: _compile(s, verbose, force), srcs))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp"
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs, *LINK]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _say_built(LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
