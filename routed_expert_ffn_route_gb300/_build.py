"""Build the CUDA library in-tree: every csrc/*.cu compiled for sm_103a in parallel, then
linked into libmoe_gb300.so next to this file, and the token operators' Python entry points
(csrc/tokens_py.cpp, which reads tensors through torch's headers).  No cmake; nvcc and a C++
host compiler only."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmoe_gb300.so")
# Python entry points of the token operators, for this interpreter (its ABI is in the name)
PY_EXT = os.path.join(HERE, "_tokens_native" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVFLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
           "-Xcompiler", "-O2", "-I", os.path.join(os.path.dirname(HERE), "include")]


def nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return p


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(os.path.dirname(HERE), "include", "*.h"))


def _compile(src: str, extra) -> str:
    obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
    newest_dep = max([os.path.getmtime(src)] + [os.path.getmtime(h) for h in _headers()])
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest_dep and not extra:
        return obj
    cmd = [nvcc(), *ARCH, *NVFLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, extra=()) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    if force:
        for o in glob.glob(os.path.join(OUT_DIR, "*.o")):
            os.remove(o)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(16, len(srcs) + 1)) as ex:
        entries = ex.submit(_entries_obj, force)
        objs = list(ex.map(lambda s: _compile(s, list(extra)), srcs))
    if (not os.path.exists(LIB) or force or extra
            or max(os.path.getmtime(o) for o in objs) > os.path.getmtime(LIB)):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, LIB)
    _link_entries(entries.result(), force)
    return LIB


def _entries_key(cmd) -> str:
    """What the entry points' object was made by and for: an interpreter, a torch, a command.
    File times do not say it: another environment's torch may be older than the object."""
    import torch
    return "\n".join([sys.version, str(torch.__version__), str(torch.version.cuda), *cmd])


def _entries_obj(force: bool):
    """Compile the token operators' Python entry points (torch's headers, a host compiler).
    None where they cannot be had, without torch, with a torch without CUDA or without Python's
    headers: the C library needs none of these, and a call of a token operator says so then."""
    try:
        import torch
    except ImportError:
        return None
    if torch.version.cuda is None or not os.path.exists(
            os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return None
    src = os.path.join(CSRC, "tokens_py.cpp")
    obj = os.path.join(OUT_DIR, "tokens_py.o")
    base = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    abi = int(torch.compiled_with_cxx11_abi())
    inc = [base, os.path.join(base, "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], cuda]
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={abi}", f'-DTOKENS_TORCH="{torch.__version__}"',
           *(a for i in inc for a in ("-isystem", i)), "-c", src, "-o", obj]
    key, made = _entries_key(cmd), obj + ".key"
    dep = max(os.path.getmtime(p) for p in [src, torch.__file__] + _headers())
    if os.path.exists(obj) and os.path.exists(made) and not force:
        with open(made) as f:
            if f.read() == key and os.path.getmtime(obj) >= dep:
                return obj
    if os.path.exists(made):
        os.remove(made)  # written again once the object stands
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for tokens_py.cpp:\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    with open(made, "w") as f:
        f.write(key)
    return obj


def _link_entries(obj, force: bool):
    """The extension module beside the library it calls; torch's libraries are loaded by torch."""
    if obj is None:
        return
    untagged = os.path.join(HERE, "_tokens_native.so")  # any interpreter would load it
    if os.path.exists(untagged) and untagged != PY_EXT:
        os.remove(untagged)
    if (os.path.exists(PY_EXT) and not force
            and os.path.getmtime(PY_EXT) >= max(os.path.getmtime(obj), os.path.getmtime(LIB))):
        return
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = PY_EXT + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "c++", "-shared", "-o", tmp, obj, "-L", HERE,
           "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN", "-L", lib, "-ltorch_python",
           "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed for tokens_py.cpp:\n{r.stderr}")
    os.replace(tmp, PY_EXT)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv))
