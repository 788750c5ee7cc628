"""Build the in-tree CUDA library ``libw4a4.so`` for sm_103a with nvcc.

Each translation unit is compiled in parallel into ``_build/`` and linked into
``w4a4_quantized_gemm_gb300/libw4a4.so`` (static CUDA runtime, no torch).  The
Python entry of the decoder-layer operators, ``csrc/binding.cpp``, is compiled
with g++ against the installed torch into ``_binding.so``, which uses that library
(the library is built without it where that cannot be done).
Each is rebuilt only when a source or header of its own is newer, the binding also
for another Python or torch.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libw4a4.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(HERE, "_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
                     "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(ROOT, "include", "*.h"))


def _newer(target, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(d) <= os.path.getmtime(target) for d in deps)


def _library_up_to_date() -> bool:
    return _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + _headers())


def _built_for() -> str:
    """What the binding's machine code depends on beside its sources; kept in _build/binding.for."""
    try:
        import torch
    except ImportError:
        return ""
    return f"python {sys.version} torch {torch.__version__} {torch.__file__}\n"


def _binding_up_to_date() -> bool:
    kept = os.path.join(BUILD, "binding.for")
    if not _newer(BINDING, [BINDING_SRC] + _headers()) or not os.path.exists(kept):
        return False
    with open(kept) as f:
        return f.read() == _built_for()


def up_to_date() -> bool:
    return _library_up_to_date() and _binding_up_to_date()


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds what is older than its sources.  Where the binding cannot be built (no Python or torch headers) the
    library is all the same, with a warning; the operators that need the binding then raise ImportError."""
    library, binding = force or not _library_up_to_date(), force or not _binding_up_to_date()
    if not library and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *NVCC_FLAGS, "-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{res.stderr}")
        return obj, res.stderr

    def compile_binding():
        obj = os.path.join(BUILD, "binding.o")
        import torch
        import torch.utils.cpp_extension as ext
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-c", BINDING_SRC, "-o", obj,
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
               "-I", os.path.join(ROOT, "include"), "-I", os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include"),
               "-isystem", sysconfig.get_paths()["include"], *(x for p in ext.include_paths() for x in ("-isystem", p))]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"g++ failed for {BINDING_SRC}:\n{res.stderr}")
        return obj, [x for p in ext.library_paths() for x in ("-L" + p, "-Wl,-rpath," + p)]

    def link(cmd, target):
        tmp = target + f".tmp{os.getpid()}"
        res = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stderr}")
        os.replace(tmp, target)

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        binding_job = ex.submit(compile_binding) if binding else None
        results = list(ex.map(compile_one, sources())) if library else []
    if verbose:
        for obj, log in results:
            print(f"== {os.path.basename(obj)}\n{log}")
    if library:
        link([nvcc, *ARCH, "-shared", *[o for o, _ in results], "-Xcompiler", "-fPIC"], LIB)
    if binding:
        try:
            obj, torch_libs = binding_job.result()
            link(["g++", "-shared", obj, "-L" + HERE, "-l:libw4a4.so", "-Wl,-rpath,$ORIGIN", *torch_libs, "-ltorch_python",
                  "-ltorch_cpu", "-lc10_cuda", "-lc10"], BINDING)
            with open(os.path.join(BUILD, "binding.for"), "w") as f:
                f.write(_built_for())
        except (RuntimeError, ImportError, OSError) as e:
            if os.path.exists(BINDING):
                os.remove(BINDING)  # of other sources
            warnings.warn(f"the binding of the decoder-layer operators was not built: {e}", RuntimeWarning)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
