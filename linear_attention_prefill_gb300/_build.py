"""Build libgdn.so in-tree with nvcc for sm_103a (no torch extension machinery), and beside
it the Python extension that binds the layer operators (layer_binding.cpp, host C++).

libgdn.so needs nvcc only.  The extension is compiled against the installed torch; without
one (or with one that has no CUDA) it is left out, and where it does not compile libgdn.so
is in place before the error is raised.

Every .cu under csrc/ compiles to an object in parallel; the objects link into
linear_attention_prefill_gb300/libgdn.so with the static CUDA runtime, so the
library loads on a machine without a GPU driver (exported symbols can be
inspected; nothing runs until a call reaches CUDA).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgdn.so")
BINDING_SRC = os.path.join(CSRC, "layer_binding.cpp")
BINDING = os.path.join(PKG, "_layer_native.so")
BINDING_FOR = os.path.join(PKG, "_layer_native.txt")  # what it was compiled against, kept beside it
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgdn.so")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [
        os.path.join(os.path.dirname(PKG), "include", "gdn.h")]


def binding_key():
    """What the extension is compiled against: torch's version and Python's ABI; None without a
    torch that has CUDA."""
    try:
        import torch
    except ImportError:
        return None
    if not torch.version.cuda:
        return None
    return f"torch {torch.__version__} {torch.version.git_version} {sysconfig.get_config_var('SOABI')}"


def binding_built_for():
    """The binding_key() that the extension in place was compiled against, or None."""
    if not os.path.exists(BINDING) or not os.path.exists(BINDING_FOR):
        return None
    with open(BINDING_FOR) as f:
        return f.read()


def _build_binding(key: str) -> None:
    """Compile the layer operators' binding against the installed torch, whose key it is."""
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    tmp = BINDING + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", BINDING_SRC, "-o", tmp]
    cmd += [f"-I{d}" for d in (os.path.join(root, "include"),
                              os.path.join(root, "include", "torch", "csrc", "api", "include"),
                              sysconfig.get_paths()["include"], os.path.join(cuda, "include"))]
    cmd += [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f"-L{os.path.join(root, 'lib')}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
            "-lc10_cuda", "-ltorch_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{r.stderr}")
    if os.path.exists(BINDING_FOR):  # never a new extension beside the old one's key
        os.remove(BINDING_FOR)
    os.replace(tmp, BINDING)
    with open(BINDING_FOR, "w") as f:
        f.write(key)


def up_to_date() -> bool:
    built = [LIB]
    key = binding_key()
    if key is not None:
        if binding_built_for() != key:
            return False
        built.append(BINDING)
    if not all(os.path.exists(b) for b in built):
        return False
    t = min(os.path.getmtime(b) for b in built)
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile and link libgdn.so, and the binding; returns libgdn.so's path.  Raises on a compiler
    error, one in the binding once libgdn.so is in place."""
    if not force and up_to_date():
        return LIB
    nvcc = nvcc_path()
    os.makedirs(BUILD, exist_ok=True)
    flags = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                    "-I", os.path.join(os.path.dirname(PKG), "include")]
    if ptxas_verbose:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        key = binding_key()
        binding = ex.submit(_build_binding, key) if key is not None else None
        results = list(ex.map(compile_one, _sources()))
    logs = "".join(err for _, err in results)
    if verbose and logs:
        sys.stderr.write(logs)
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        f.write(logs)
    if binding is not None:
        binding.result()
    elif verbose:
        sys.stderr.write("no torch with CUDA: the layer operators' Python binding is left out\n")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv)
    print(LIB)
