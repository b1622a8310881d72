"""Build libmxgemm.so in-tree: nvcc for sm_103a only, one object per source
compiled in parallel, then a shared link against the CUDA runtime; beside it
_attn_bind.so, the CPython module that calls the attention entry points.  The
library needs nvcc alone and is linked whatever becomes of the module, which
needs torch's headers; where torch is not installed it is left out (the package,
which loads it, needs torch too)."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmxgemm.so")
SOURCES = ["api.cu", "quant.cu", "gemm.cu", "attn_api.cu", "attn.cu", "attn_long.cu", "rope.cu", "index.cu"]
BIND = os.path.join(PKG, "_attn_bind.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def _cuda_lib_dir() -> str:
    return os.path.join(os.path.dirname(os.path.dirname(nvcc())), "lib64")


def _stale(out: str, deps: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _bind_flags() -> tuple[list[str], list[str], str] | None:
    """Compile and link flags of the CPython module (torch's headers and
    libraries) and what it is built for; None without torch."""
    import sys
    import sysconfig
    try:
        import torch
    except (ImportError, OSError):
        return None
    root = os.path.dirname(os.path.abspath(torch.__file__))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(_cuda_lib_dir()), "include"), sysconfig.get_paths()["include"], INCLUDE]
    cc = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"] + ["-I" + i for i in inc]
    lib = os.path.join(root, "lib")
    ld = ["-L" + lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath," + lib,
          "-L" + PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + _cuda_lib_dir()]
    made_for = f"torch {torch.__version__}, Python {sys.version}\n" + "\n".join(cc + ld)
    return cc, ld, made_for


def _run(cmd: list[str]) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]
    if verbose:
        flags += ["-Xptxas", "-v"]
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            jobs.append([nvcc(), *flags, "-c", s, "-o", o])

    # the module: also built anew for another torch or Python than its stamp names
    bind_src, bind_obj = os.path.join(CSRC, "bind.cpp"), os.path.join(BUILD, "bind.o")
    stamp = os.path.join(BUILD, "bind.stamp")
    flags_bind = _bind_flags()
    made = None
    if os.path.exists(stamp):
        with open(stamp) as f:
            made = f.read()
    bind_new = flags_bind is not None and (force or made != flags_bind[2] or _stale(BIND, [bind_src] + headers))

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        bind_job = ex.submit(_run, ["g++", *flags_bind[0], "-c", bind_src, "-o", bind_obj]) if bind_new else None
        for out in ex.map(_run, jobs):
            if verbose and out:
                print(out)
        if force or _stale(LIB, objs):
            tmp = LIB + f".tmp{os.getpid()}"
            _run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "shared",
                  "-Xlinker", "-rpath," + _cuda_lib_dir()])
            os.replace(tmp, LIB)
    if bind_job is not None:
        bind_job.result()
        tmp = BIND + f".tmp{os.getpid()}"
        _run(["g++", "-shared", "-o", tmp, bind_obj, *flags_bind[1]])
        os.replace(tmp, BIND)
        with open(stamp, "w") as f:
            f.write(flags_bind[2])
    elif flags_bind is None:
        print("torch is not installed: the library is built, its Python module for the attention entry points is not")
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
